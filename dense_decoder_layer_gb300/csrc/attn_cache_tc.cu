// Attention of drafted tokens over a cache when a kv head has many query rows
// (a tree of tens of tokens, a chunk of a prompt): the tcgen05 form of
// attn_cache.cu, same mathematics, same schedule of chunks.
//
// What bounds it: with R = T G query rows per cached row the products are
// 4 R hd flop against 2 hd bits/8 bytes, so beyond some 140 rows of an e4m3
// cache (280 of a bf16 one) the tensor pipe is the floor, below it HBM; in
// between stands the work per score -- exp2, packing, and for 8- and 4-bit rows
// the conversion to bf16 -- which needs every issue slot of the SM, so the
// kernel is built to keep all of these running at once.
//
// One block of 640 threads per SM, two streams of 128 query rows x 128 keys:
// with more than 128 rows the streams are two row tiles that share every K/V
// tile, else they are the even and the odd key tiles of one row tile.  While
// one stream's softmax runs, the tensor pipe works for the other.
//   warp 0       tcgen05.mma issuer: S = Q K^T into TMEM, O += P V with P read
//                from tensor memory (over its S) and V MN-major from its rows
//   warps 4-11   loaders: 16-byte asynchronous copies of cache rows; 8- and
//                4-bit codes land in slots private to their thread, which
//                turns them into the bf16 tile (no barrier in between)
//   warps 12-19  softmax, one thread per query row: a tile's 128 scores in four
//                pieces, exponentials against the row's reference maximum,
//                which moves only when a score exceeds it by 2^8 (the piece is
//                then done again), so nothing is exchanged between threads
// The key's scales are applied to the scores (K) and to P (V): the bf16 tiles
// hold the codes themselves, exactly.
//
// Every wait is bounded; a wait that gives up sets the status word and the
// block leaves in order.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <string>

#include "attn_cache.cuh"
#include "fastmath.cuh"
#include "sm100.cuh"
#include "tc.h"

namespace pds {
namespace {

using namespace cacheattn;

constexpr int kKeys = 128;             // keys per tile
constexpr int kTileRows = 128;         // query rows per stream
constexpr int kLoadWarps = 8, kLoadThreads = 32 * kLoadWarps;
constexpr int kFirstLoadWarp = 4, kFirstSoftmaxWarp = kFirstLoadWarp + kLoadWarps;
constexpr int kSoftmaxThreads = 256;
constexpr int kTileThreads = 32 * kFirstSoftmaxWarp + kSoftmaxThreads;
constexpr float kMoveLog2 = 8.0f;      // the reference maximum follows beyond a growth of 2^8
// registers per thread: 96 at launch; 384 threads give up 32 each for the 256
// softmax threads' 48 more
constexpr int kLeanRegs = 64, kSoftmaxRegs = 144;
static_assert(kTileThreads * 96 >= 384 * kLeanRegs + 256 * kSoftmaxRegs, "register split");

template <int FMT, int HD>
struct TileCfg {
  static constexpr bool kQuant = FMT != PDS_KV_BF16;
  static constexpr int kRow = FMT == PDS_KV_BF16 ? 2 * HD : FMT == PDS_KV_E4M3 ? HD : HD / 2;
  static constexpr uint32_t kTile = 128u * HD * 2u;        // bf16 tile of Q, K or V
  static constexpr uint32_t kUnit = 128u * kRow;           // a tile's cached bytes
  static constexpr int kPerRow = kRow / 16;                // 16-byte pieces of a row
  static constexpr int kPieces = 128 * kPerRow / kLoadThreads;  // of a thread, per tile
  // Stages: 8- and 4-bit tiles wait in their raw slots, so few converted ones
  // are needed; bf16 rows land in the tiles themselves.
  static constexpr int kKStages = HD == 64 ? 3 : kQuant ? 1 : 2;
  static constexpr int kVStages = HD == 64 ? 4 : 2;
  static constexpr int kRaw = HD == 64 ? 6 : FMT == PDS_KV_E4M3 ? 3 : 4;  // raw slots (tiles)
  // Tiles in flight.  A bf16 tile's copy waits for its stage, and the tiles in
  // flight ahead of it are handed over only after that: three ahead, V_{j+1}
  // waits for P V of tile j - 1 before V_j is handed over and K_{j+2} for S of
  // tile j before K_{j+1} is, and neither product needs those.
  static constexpr int kAhead = kQuant ? kRaw - 1 : HD == 64 ? 5 : 3;
  // Ring of scale words.  They are fetched with K, kAhead tiles' halves early,
  // after a K stage has come free kKStages tiles back, when the softmax is done
  // with the tile two before that one: at most kAhead / 2 + kKStages + 3 tiles
  // are in use.
  static constexpr int kWordTiles = HD == 64 ? 8 : 6;
  static_assert(!kQuant || kWordTiles >= kAhead / 2 + kKStages + 3, "scale words in use");
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = 2 * kTile;
  static constexpr uint32_t kV = kK + kKStages * kTile;
  static constexpr uint32_t kRawAt = kV + kVStages * kTile;
  static constexpr uint32_t kWords = kRawAt + (kQuant ? kRaw * kUnit : 0u);
  static constexpr uint32_t kZero = kWords + (kQuant ? kWordTiles * 1024u : 0u);  // int4: own words
  static constexpr uint32_t kMask = kZero + (FMT == PDS_KV_INT4 ? kRaw * kPieces * 1024u : 0u);
  static constexpr uint32_t kPar = kMask + kMaskWords * 256u * 4u;
  static constexpr uint32_t kMl = kPar + kMaxDraftTokens * 4u;
  static constexpr uint32_t kBar = kMl + 2u * 128u * 8u;
  static constexpr int kNumBars = 1 + 2 * (kKStages + kVStages) + 8;
  static constexpr uint32_t kMisc = kBar + 8u * kNumBars;
  static constexpr size_t kSmem = 1024 + kMisc + 96;
  static_assert(kSmem <= 232448, "shared memory per block");
  static constexpr uint32_t kTmS = 0, kTmO = 256, kTmemCols = 512;
};

__device__ __forceinline__ uint64_t kmajor_desc(uint32_t base, int kstep) {
  // 16 contraction elements: 32 bytes inside a 128-byte column block, 4 per block
  return sm100::smem_desc_sw128(base + static_cast<uint32_t>(kstep >> 2) * 16384u +
                                static_cast<uint32_t>(kstep & 3) * 32u);
}
// V tile [128 keys][HD] as the MN-major B operand: rows are keys (128 bytes of
// 64 channels), 8-row groups 1024 bytes apart, channels 64..127 16 KB on.
__device__ __forceinline__ uint64_t v_desc(uint32_t base, int kstep) {
  const uint32_t a = base + static_cast<uint32_t>(kstep) * 16u * 128u;
  return static_cast<uint64_t>((a >> 4) & 0x3FFFu) | static_cast<uint64_t>(16384u >> 4) << 16 |
         static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1) << 46 |
         static_cast<uint64_t>(2) << 61;
}
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? (1u << 16) : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Byte offset of 8-channel piece c of row r in a swizzled bf16 tile.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return static_cast<uint32_t>(c >> 3) * 16384u + r * 128u + (((c & 7) ^ (r & 7)) << 4);
}

// (a0, a1) * (b0, b1) + (c, c) and (a0, a1) * (b0, b1), packed.
__device__ __forceinline__ void fma2_pair(float& a0, float& a1, float b0, float b1, float c) {
  uint64_t a, b, cc, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(cc) : "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(cc));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(d));
}
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
  uint64_t a, b, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(d));
}
__device__ __forceinline__ float max32(const float* v) {
  float a[11];
#pragma unroll
  for (int i = 0; i < 10; ++i) a[i] = max3(v[3 * i], v[3 * i + 1], v[3 * i + 2]);
  a[10] = fmaxf(v[30], v[31]);
  const float b0 = max3(a[0], a[1], a[2]), b1 = max3(a[3], a[4], a[5]);
  const float b2 = max3(a[6], a[7], a[8]), b3 = fmaxf(a[9], a[10]);
  return fmaxf(max3(b0, b1, b2), b3);
}

// Which of the 32 keys from key0 on a query row sees.  `mask`: the row's ancestor
// bits (the window already applied), a word per 32 tokens, 256 words apart;
// `lo`: the first cached row within its window.
__device__ __forceinline__ uint32_t visible32(int key0, int len, int lo, const uint32_t* mask) {
  const int rel = key0 - len;
  uint32_t v;
  if (rel <= -32) {
    v = 0xffffffffu;
  } else if (rel < 0) {
    v = ((1u << -rel) - 1u) | (mask[0] << -rel);
  } else {
    const int w = rel >> 5;
    const uint32_t a = w < kMaskWords ? mask[w * 256] : 0u;
    const uint32_t b = w + 1 < kMaskWords ? mask[(w + 1) * 256] : 0u;
    v = __funnelshift_r(a, b, rel & 31);
  }
  const int cached = min(max(-rel, 0), 32);              // of the 32, rows of the prefix
  const int cut = min(max(lo - key0, 0), cached);        // of those, below the window
  return cut >= 32 ? 0u : v & ~((1u << cut) - 1u);
}

// Whether the tile of keys from key0 on holds rows that some query rows see
// and others do not (or rows past the end).
__device__ __forceinline__ bool tile_partial(const Args& a, int key0, int len) {
  return key0 + kKeys > len || (a.window > 0 && key0 < len + a.n_tokens - a.window);
}

template <int FMT, int HD, bool VAR>
__global__ void __launch_bounds__(kTileThreads, 1)
    cache_attn_tile_kernel(const __grid_constant__ Args a) {
  using namespace sm100;
  using C = TileCfg<FMT, HD>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_base);
  const uint32_t bar0 = sbase + C::kBar;
  const uint32_t bar_q = bar0;
  auto bar_k_full = [&](int st) { return bar0 + 8u * (1 + st); };
  auto bar_k_empty = [&](int st) { return bar0 + 8u * (1 + C::kKStages + st); };
  auto bar_v_full = [&](int st) { return bar0 + 8u * (1 + 2 * C::kKStages + st); };
  auto bar_v_empty = [&](int st) { return bar0 + 8u * (1 + 2 * C::kKStages + C::kVStages + st); };
  constexpr int kBar2 = 1 + 2 * (C::kKStages + C::kVStages);
  auto bar_s_full = [&](int s) { return bar0 + 8u * (kBar2 + s); };
  auto bar_p_full = [&](int s) { return bar0 + 8u * (kBar2 + 2 + s); };
  auto bar_done = [&](int s) { return bar0 + 8u * (kBar2 + 4 + s); };
  auto bar_pv = [&](int s) { return bar0 + 8u * (kBar2 + 6 + s); };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* poison = reinterpret_cast<volatile int*>(misc + 2);  // V of a partial tile held inf / NaN
  int* shared_ok = reinterpret_cast<int*>(misc + 3);
  Unit* shared_unit = reinterpret_cast<Unit*>(misc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = a.c.n_kv_heads * a.row_tiles;
  const int w = blockIdx.x / per, p = blockIdx.x - w * per;
  const int head = p % a.c.n_kv_heads, group_tile = p / a.c.n_kv_heads;
  const int rows = a.n_tokens * a.group, r0 = group_tile * a.tile_rows;
  const bool two_tiles = rows - r0 > kTileRows;  // the streams are row tiles, else key halves
  if (threadIdx.x == 0) {
    mbar_init(bar_q, kSoftmaxThreads / 32);
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(bar_k_full(i), kLoadWarps);
      mbar_init(bar_k_empty(i), two_tiles ? 2 : 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(bar_v_full(i), kLoadWarps);
      mbar_init(bar_v_empty(i), two_tiles ? 2 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_s_full(s), 1);
      mbar_init(bar_p_full(s), 4);  // one arrival per softmax warp
      mbar_init(bar_done(s), 1);
      mbar_init(bar_pv(s), 1);
    }
    *abort_flag = 0;
    *poison = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), C::kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();  // everything below reads what earlier kernels wrote
  grid_dep_launch();
  if (warp == 0) {
    Unit u{};
    const Lane mine = lane_steps(a, lane);
    const int c = chunk_steps(a, lane, mine);
    const bool ok = find_unit(a, c, w, 0, lane, mine, u);
    if (lane == 0) {
      *shared_unit = u;
      *shared_ok = ok;
    }
    if (blockIdx.x == 0) {  // report lengths that do not fit
      bool bad = false;
      for (int s = lane; s < a.c.n_seqs; s += 32) bad |= lane_steps(a, s).n == 0;
      if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kStatusBadLength);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const Unit u = *shared_unit;
  // (a block without a unit walks through with no tiles)
  const int n = *shared_ok ? u.n_steps : 0;
  const int len = u.len, end = len + a.n_tokens;
  const int n_tiles[2] = {two_tiles ? n : (n + 1) / 2, two_tiles ? n : n / 2};
  auto tile_of = [&](int s, int i) { return two_tiles ? i : 2 * i + s; };

  if (warp < kFirstLoadWarp) {
    setmaxnreg_dec<kLeanRegs>();
    if (warp == 0 && lane == 0 && n > 0) {
      constexpr uint32_t kIdS = idesc(128, kKeys, false);
      constexpr uint32_t kIdPV = idesc(128, HD, true);
      bool ok = mbar_wait(bar_q, 0, abort_flag, a.status);
      // Each stream alternates S_i, O += P_i V_i.  Whichever product has its
      // operands is issued next, so neither stream waits behind the other.  S
      // of tile i goes over P of tile i - 1, so it waits until that product has
      // been completed.  (Key halves take their tiles of K in order: a stage's
      // barrier is asked only for the phase after the last one seen.)
      int at[2] = {0, 0}, next_k = 0;
      bool pv_next[2] = {false, false};
      auto try_issue = [&](int s) {
        const int i = at[s], t = tile_of(s, i);
        if (!pv_next[s]) {
          const int st = t % C::kKStages;
          if (!two_tiles && t != next_k) return false;
          if (!mbar_test(bar_k_full(st), (t / C::kKStages) & 1)) return false;
          if (i > 0 && !mbar_test(bar_pv(s), (i - 1) & 1)) return false;
          tc_fence_after();
          const uint32_t q = sbase + C::kQ + (two_tiles ? s * C::kTile : 0u);
          const uint32_t k = sbase + C::kK + st * C::kTile;
#pragma unroll
          for (int x = 0; x < HD / 16; ++x)
            umma_bf16(tmem + C::kTmS + s * 128u, kmajor_desc(q, x), kmajor_desc(k, x), kIdS,
                      x > 0 ? 1u : 0u);
          umma_commit(bar_s_full(s));
          umma_commit(bar_k_empty(st));
          ++next_k;
          pv_next[s] = true;
        } else {
          const int st = t % C::kVStages;
          if (!mbar_test(bar_p_full(s), i & 1)) return false;
          if (!mbar_test(bar_v_full(st), (t / C::kVStages) & 1)) return false;
          tc_fence_after();
          const uint32_t v = sbase + C::kV + st * C::kTile;
#pragma unroll
          for (int x = 0; x < kKeys / 16; ++x)
            umma_bf16_ts(tmem + C::kTmO + s * 128u, tmem + C::kTmS + s * 128u + x * 8u,
                         v_desc(v, x), kIdPV, (i > 0 || x > 0) ? 1u : 0u);
          umma_commit(bar_pv(s));
          umma_commit(bar_v_empty(st));
          pv_next[s] = false;
          ++at[s];
        }
        return true;
      };
      uint64_t t0 = global_timer_ns();
      uint32_t idle = 0;
      while (ok && (at[0] < n_tiles[0] || at[1] < n_tiles[1])) {
        bool progress = false;
        for (int s = 0; s < 2; ++s)
          if (at[s] < n_tiles[s] && try_issue(s)) progress = true;
        if (progress) {
          idle = 0;
        } else if ((++idle & 63u) == 0) {  // bounded as the other waits are
          if (idle == 64u) t0 = global_timer_ns();
          if (*abort_flag) {
            ok = false;
          } else if (global_timer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            atomicOr(a.status, kStatusTimeout);
            ok = false;
          }
        }
      }
      umma_commit(bar_done(0));
      umma_commit(bar_done(1));
      int dummy = 0;
      mbar_wait(bar_done(0), 0, &dummy, a.status);
      mbar_wait(bar_done(1), 0, &dummy, a.status);
    }
  } else if (warp < kFirstSoftmaxWarp) {
    setmaxnreg_dec<kLeanRegs>();
    const int tid = threadIdx.x - 32 * kFirstLoadWarp;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = ok && mbar_wait(bar, parity, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
    };
    auto arrive = [&](uint32_t bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // this thread's pieces of a tile: rows row0 + i kRowStep, 16-byte column col
    constexpr int kRowStep = kLoadThreads / C::kPerRow;
    const int col = tid % C::kPerRow, row0 = tid / C::kPerRow;
    const int64_t at = u.seq * a.c.seq_stride + head * a.c.head_stride + col * 16;
    const char* k_src = a.c.k + at;
    const char* v_src = a.c.v + at;
    const int64_t word0 = (static_cast<int64_t>(u.seq) * a.c.n_kv_heads + head) * a.c.capacity;
    const int units = 2 * n;  // K_0, V_0, K_1, V_1, ...
    auto tile_base = [&](int un) {
      const int t = un >> 1;
      return un & 1 ? sbase + C::kV + (t % C::kVStages) * C::kTile
                    : sbase + C::kK + (t % C::kKStages) * C::kTile;
    };
    auto wait_free = [&](int un) {
      const int t = un >> 1;
      if (un & 1) {
        if (t >= C::kVStages) wait(bar_v_empty(t % C::kVStages), (t / C::kVStages - 1) & 1);
      } else {
        if (t >= C::kKStages) wait(bar_k_empty(t % C::kKStages), (t / C::kKStages - 1) & 1);
      }
    };
    auto full = [&](int un) {
      return un & 1 ? bar_v_full((un >> 1) % C::kVStages) : bar_k_full((un >> 1) % C::kKStages);
    };
    auto issue = [&](int un) {
      if (un < units) {
        if (!C::kQuant) wait_free(un);
        if (ok) {
          const int key0 = (u.first + (un >> 1)) * kKeys;
          const char* src = un & 1 ? v_src : k_src;
          const uint32_t dst = C::kQuant
                                   ? sbase + C::kRawAt + (un % C::kRaw) * C::kUnit + tid * 16u
                                   : tile_base(un);
#pragma unroll
          for (int i = 0; i < C::kPieces; ++i) {
            const int r = row0 + i * kRowStep;
            const bool live = key0 + r < end;
            // a row past the end is not read: its address is that of the last one
            const int64_t j = live ? key0 + r : end - 1;
            copy16(C::kQuant ? dst + i * 4096u : dst + tile_at(r, col), src + j * a.c.row_stride,
                   live);
            if constexpr (FMT == PDS_KV_INT4)
              copy4(sbase + C::kZero + ((un % C::kRaw) * C::kPieces + i) * 1024u + tid * 4u,
                    (un & 1 ? a.c.v_scale : a.c.k_scale) + word0 + j, live);
          }
          if (C::kQuant && !(un & 1)) {  // the tile's scale words: K's, then V's
            const int key = key0 + (tid & 127);
            copy4(sbase + C::kWords + ((un >> 1) % C::kWordTiles) * 1024u + tid * 4u,
                  (tid < 128 ? a.c.k_scale : a.c.v_scale) + word0 + (key < end ? key : end - 1),
                  key < end);
          }
        }
      }
      copies_commit();
    };
    for (int un = 0; un < C::kAhead; ++un) issue(un);
    for (int un = 0; un < units && ok; ++un) {
      if (C::kQuant) issue(un + C::kAhead);  // into the slot this thread emptied last
      copies_wait<C::kAhead - (C::kQuant ? 0 : 1)>();
      if constexpr (!C::kQuant) {
        if ((un & 1) && tile_partial(a, (u.first + (un >> 1)) * kKeys, len)) {
          // Rows that some query rows must not see: an infinity or a NaN would
          // reach them through a zero weight.  It is taken out here and added
          // to the rows that do see it at the end.
          for (int i = 0; i < C::kPieces; ++i) {
            const uint32_t d = tile_base(un) + tile_at(row0 + i * kRowStep, col);
            const uint4 x = lds128(d);
            uint32_t y[4] = {x.x, x.y, x.z, x.w};
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (!not_finite2(y[e])) continue;
              bad = true;
              if ((y[e] & 0x7f80u) == 0x7f80u) y[e] &= 0xffff0000u;
              if ((y[e] & 0x7f800000u) == 0x7f800000u) y[e] &= 0x0000ffffu;
            }
            if (bad) {
              st_shared_u4(d, y[0], y[1], y[2], y[3]);
              *poison = 1;
            }
          }
        }
      } else {
        wait_free(un);
        if (!ok) break;
        const uint32_t src = sbase + C::kRawAt + (un % C::kRaw) * C::kUnit + tid * 16u;
        const uint32_t dst = tile_base(un);
#pragma unroll
        for (int i = 0; i < C::kPieces; ++i) {
          const int r = row0 + i * kRowStep;
          const uint4 x = lds128(src + i * 4096u);
          const uint32_t c[4] = {x.x, x.y, x.z, x.w};
          if constexpr (FMT == PDS_KV_E4M3) {
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[2 * e] = e4m3_pair(__byte_perm(c[e], 0u, 0x1404));
              y[2 * e + 1] = e4m3_pair(__byte_perm(c[e], 0u, 0x3424));
            }
            // the two halves in an order that keeps the lanes of a row on different banks
            const bool swap = col & (C::kPerRow >> 1);
            const uint32_t d0 = dst + tile_at(r, 2 * col), d1 = dst + tile_at(r, 2 * col + 1);
            st_shared_u4(swap ? d1 : d0, swap ? y[4] : y[0], swap ? y[5] : y[1],
                         swap ? y[6] : y[2], swap ? y[7] : y[3]);
            st_shared_u4(swap ? d0 : d1, swap ? y[0] : y[4], swap ? y[1] : y[5],
                         swap ? y[2] : y[6], swap ? y[3] : y[7]);
          } else {
            const uint32_t z = lds32(sbase + C::kZero + ((un % C::kRaw) * C::kPieces + i) * 1024u +
                                     tid * 4u) & 15u;
            const uint32_t zz = 0x43004300u | z | z << 16;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t lo = c[e], hi = c[e] >> 4;
              st_shared_u4(dst + tile_at(r, 4 * col + e), int4_pair(__byte_perm(lo, hi, 0x0400), zz),
                           int4_pair(__byte_perm(lo, hi, 0x0501), zz),
                           int4_pair(__byte_perm(lo, hi, 0x0602), zz),
                           int4_pair(__byte_perm(lo, hi, 0x0703), zz));
            }
          }
        }
        if (!(un & 1)) {
          // the scale words as factors: of scores in powers of two, and of P
          float* word = reinterpret_cast<float*>(smem + C::kWords +
                                                 ((un >> 1) % C::kWordTiles) * 1024u) + tid;
          uint32_t bits = __float_as_uint(*word);
          if (FMT == PDS_KV_INT4) bits &= 0xffff0000u;
          *word = __uint_as_float(bits) * (tid < 128 ? a.scale_log2 : 1.0f);
        }
      }
      arrive(full(un));
      if (!C::kQuant) issue(un + C::kAhead);
    }
    copies_wait<0>();
  } else {
    setmaxnreg_inc<kSoftmaxRegs>();
    const int tid = threadIdx.x - 32 * kFirstSoftmaxWarp;
    const int s = tid >> 7;                       // stream
    const int r = tid & 127;                      // row of the stream's tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::kTmS + s * 128u;
    const uint32_t to = tmem + lane_off + C::kTmO + s * 128u;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = ok && mbar_wait(bar, parity, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) tc_fence_after();
    };
    // Q tiles: row x of both streams' tiles in rounds of 8-channel pieces
    if (n > 0) {
      constexpr int kPieces = HD / 8;
      const int tiles = two_tiles ? 2 : 1;
      for (int idx = tid; idx < tiles * 128 * kPieces; idx += kSoftmaxThreads) {
        const int row = idx / kPieces, c = idx - row * kPieces, R = r0 + row;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (R < rows) {
          const int t = R / a.group, i = R - t * a.group;
          x = *reinterpret_cast<const uint4*>(
              a.q + (static_cast<int64_t>(u.seq) * a.n_tokens + t) * a.q_stride +
              (head * a.group + i) * HD + c * 8);
        }
        st_shared_u4(sbase + C::kQ + (row >> 7) * C::kTile + tile_at(row & 127, c), x.x, x.y, x.z,
                     x.w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q);
    }
    // the row's token: its ancestors (within the window) as bits of its own
    // column of the mask table, and the first cached row it sees
    const int R = r0 + (two_tiles ? s * kTileRows : 0) + r;
    const bool row_live = R < rows;
    const int tok = row_live ? R / a.group : 0;
    int32_t* par = reinterpret_cast<int32_t*>(smem + C::kPar);
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + C::kMask) + tid;
    if (n > 0 && a.parents && tid < a.n_tokens)
      par[tid] = a.parents[static_cast<int64_t>(u.seq) * a.n_tokens + tid];
    named_bar_sync(1, kSoftmaxThreads);
    int depth = tok;
    if (n > 0 && a.parents) {
      depth = tree_depth(par, tok);
      if (depth == kBadParent && row_live) atomicOr(a.status, kStatusBadParent);
    }
    {
      uint32_t bits[kMaskWords];
#pragma unroll
      for (int i = 0; i < kMaskWords; ++i) bits[i] = 0u;
      if (n > 0 && depth >= 0) {
        int left = a.window > 0 ? a.window : kMaxDraftTokens;  // itself counts as one
        for (int x = tok; x >= 0 && left > 0; x = a.parents ? par[x] : x - 1, --left)
#pragma unroll
          for (int i = 0; i < kMaskWords; ++i)
            if ((x >> 5) == i) bits[i] |= 1u << (x & 31);
      }
#pragma unroll
      for (int i = 0; i < kMaskWords; ++i) mask[i * 256] = bits[i];
    }
    const int lo = VAR && a.window > 0 ? len + depth - a.window + 1 : 0;

    const bool warp_live = r0 + (two_tiles ? s * kTileRows : 0) + (warp & 3) * 32 < rows;
    const float sc = a.scale_log2, cap = VAR ? a.cap * a.scale_log2 : 0.f;  // powers of two
    float m_ref = -INFINITY, l = 0.f;
    for (int i = 0; i < n_tiles[s]; ++i) {
      wait(bar_s_full(s), i & 1);
      if (!ok) break;
      if (!warp_live) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full(s));
        continue;
      }
      const int t = tile_of(s, i);
      const int key0 = (u.first + t) * kKeys;
      const bool partial = tile_partial(a, key0, len);
      const uint32_t words = sbase + C::kWords + (t % C::kWordTiles) * 1024u;
      uint32_t pk[64];
      float sum = 0.f;
      // a second pass only where the first finds that a reference has to move
      for (int pass = 0; pass < 2; ++pass) {
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // masked scores give 0
        float mx = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float z[32];
          tmem_load32(ts + c * 32, z);
          if (VAR && cap > 0.f) {
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              float f = sc;
              if constexpr (C::kQuant) f = __uint_as_float(lds32(words + (c * 32 + x) * 4));
              // c tanh(z / c) = c - 2 c / (2^(2 log2(e) z / c) + 1)
              const float y = z[x] * f;
              const float e = exp2_fast(y * (2.0f * 1.4426950408889634f / cap));
              z[x] = cap - __fdividef(2.0f * cap, e + 1.0f) - m_use;
            }
          } else if constexpr (C::kQuant) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float4 f = ld_shared_f4(words + (c * 32 + 4 * x) * 4);
              fma2_pair(z[4 * x], z[4 * x + 1], f.x, f.y, -m_use);
              fma2_pair(z[4 * x + 2], z[4 * x + 3], f.z, f.w, -m_use);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) fma2(z[2 * x], z[2 * x + 1], sc, -m_use);
          }
          uint32_t vis = 0xffffffffu;
          if (partial) {
            vis = visible32(key0 + c * 32, len, lo, mask);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!((vis >> x) & 1u)) z[x] = -INFINITY;
          }
          mx = fmaxf(mx, max32(z));
#pragma unroll
          for (int x = 0; x < 32; ++x) z[x] = exp2_fast(z[x]);
          float part[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int x = 1; x < 8; ++x) {
            add2(part[0], part[1], z[4 * x], z[4 * x + 1]);
            add2(part[2], part[3], z[4 * x + 2], z[4 * x + 3]);
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
          if constexpr (C::kQuant) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float4 f = ld_shared_f4(words + 512u + (c * 32 + 4 * x) * 4);
              mul2(z[4 * x], z[4 * x + 1], f.x, f.y);
              mul2(z[4 * x + 2], z[4 * x + 3], f.z, f.w);
            }
            if (partial) {  // a hidden row may have any scale, a NaN too
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (!((vis >> x) & 1u)) z[x] = 0.f;
            }
          }
#pragma unroll
          for (int x = 0; x < 16; ++x) pk[c * 16 + x] = pack_bf16x2(z[2 * x], z[2 * x + 1]);
        }
        const bool move = m_ref == -INFINITY ? mx > -INFINITY : mx > kMoveLog2;
        if (pass == 1 || !__any_sync(0xffffffffu, move)) break;
        float alpha = 1.f;
        if (move) {
          const float m_new = m_use + mx;
          alpha = exp2f(m_ref - m_new);  // 0 from -inf
          m_ref = m_new;
          l *= alpha;
        }
        if (i > 0) {
          // S of this tile being there, the products issued before it are done: O is at rest
#pragma unroll
          for (int c = 0; c < HD / 16; ++c) {
            float o[16];
            tmem_load16(to + c * 16, o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] *= alpha;
            tmem_store16(to + c * 16, o);
          }
        }
      }
      l += sum;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float f[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) f[x] = __uint_as_float(pk[c * 16 + x]);
        tmem_store16_nowait(ts + c * 16, f);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p_full(s));
    }

    // ---- the rows' results
    if (n > 0) {
      wait(bar_done(0), 0);
      wait(bar_done(1), 0);
    }
    float inv_scale = 1.f, other = 0.f;  // this thread's O times the first, the other stream's the second
    int c0 = 0, c1 = HD;                 // its columns
    const uint32_t xch = sbase + C::kQ;  // (every product is done: Q's space is free)
    const uint32_t mine_at = static_cast<uint32_t>(r) * (HD * 2);
    auto xch_at = [&](int c4) {          // float4 c4 of this row's half, spread over the banks
      return mine_at + (static_cast<uint32_t>(c4 ^ (r & (HD / 8 - 1))) << 4);
    };
    if (!two_tiles) {
      // the streams hold the same rows over different keys: each takes half of
      // the columns, and gives the other half to the other stream's thread
      float2* ml = reinterpret_cast<float2*>(smem + C::kMl);
      ml[s * 128 + r] = make_float2(m_ref, l);
      if (ok && warp_live) {
        const int give = s == 0 ? HD / 2 : 0;
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) {
          float o[16];
          tmem_load16(to + give + c * 16, o);
          const bool none = n_tiles[s] == 0;  // its accumulator was never written
#pragma unroll
          for (int x = 0; x < 4; ++x)
            st_shared_f4(xch + s * (64u * HD * 4u) + xch_at(4 * c + x),
                         none ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
        }
      }
      named_bar_sync(1, kSoftmaxThreads);
      const float2 x = ml[(1 - s) * 128 + r];
      const float m = fmaxf(m_ref, x.x), mu = m == -INFINITY ? 0.f : m;
      inv_scale = exp2f(m_ref - mu);
      other = exp2f(x.x - mu);
      // the first stream's share first, whichever thread adds
      const float mine_l = l * inv_scale, other_l = x.y * other;
      l = s == 0 ? mine_l + other_l : other_l + mine_l;
      m_ref = m;
      c0 = s == 0 ? 0 : HD / 2;
      c1 = c0 + HD / 2;
    }
    if (ok && warp_live && n > 0) {
      const bool pad = depth < 0, whole = u.n_chunks == 1;
      const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row that sees nothing is zero
      const int i = R - tok * a.group;
      uint16_t* dst = a.o + (static_cast<int64_t>(u.seq) * a.n_tokens + tok) * a.o_stride +
                      (head * a.group + i) * HD;
      const int half = two_tiles ? s : 0;
      float4* part = reinterpret_cast<float4*>(a.o_part) +
                     (static_cast<int64_t>(blockIdx.x) * (a.tile_rows / 128) + half) * (HD / 4) * 128;
      for (int c = c0; c < c1; c += 16) {
        float o[16];
        tmem_load16(to + c, o);
        if (!two_tiles) {
          const bool none = n_tiles[s] == 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float4 y = ld_shared_f4(xch + (1 - s) * (64u * HD * 4u) + xch_at((c - c0) / 4 + x));
            const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float mine_o = none ? 0.f : o[4 * x + e] * inv_scale, other_o = v[e] * other;
              o[4 * x + e] = s == 0 ? mine_o + other_o : other_o + mine_o;
            }
          }
        }
        if constexpr (!C::kQuant) {
          if (*poison && row_live) {  // what the loaders took out, for the rows that see it
            for (int t = 0; t < n; ++t) {
              const int key0 = (u.first + t) * kKeys;
              if (!tile_partial(a, key0, len)) continue;
              for (int g = 0; g < 4; ++g) {
                uint32_t vis = visible32(key0 + 32 * g, len, lo, mask);
                while (vis) {
                  const int x = __ffs(vis) - 1;
                  vis &= vis - 1;
                  const uint16_t* v = reinterpret_cast<const uint16_t*>(
                      a.c.v + u.seq * a.c.seq_stride + head * a.c.head_stride +
                      (key0 + 32 * g + x) * a.c.row_stride) + c;
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    if ((v[e] & 0x7f80u) == 0x7f80u) o[e] += bf16_to_f32(v[e]);
                }
              }
            }
          }
        }
        if (!row_live) continue;
        if (whole) {
          uint32_t y[8];
#pragma unroll
          for (int x = 0; x < 8; ++x)
            y[x] = pad ? 0u : pack_bf16x2(o[2 * x] * inv, o[2 * x + 1] * inv);
          reinterpret_cast<uint4*>(dst + c)[0] = make_uint4(y[0], y[1], y[2], y[3]);
          reinterpret_cast<uint4*>(dst + c)[1] = make_uint4(y[4], y[5], y[6], y[7]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            part[(c / 4 + x) * 128 + r] =
                pad ? make_float4(0.f, 0.f, 0.f, 0.f)
                    : make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      }
      if (row_live && !whole && (two_tiles || s == 0))
        a.ml_part[static_cast<int64_t>(blockIdx.x) * a.tile_rows + half * 128 + r] =
            pad ? make_float2(-INFINITY, 0.f) : make_float2(m_ref, l);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the chunks in order.  A thread has 16 channels of one row; a warp's
// lanes are 32 rows, whose float4 pieces lie side by side.  Grid: (sequence x
// head x row tile, HD / 32, halves of 128 rows); its schedule is made while
// the chunks are still being computed.
template <int HD>
__global__ void __launch_bounds__(256) cache_join_tile_kernel(const __grid_constant__ Args a) {
  __shared__ Unit shared_unit;
  const int lane = threadIdx.x & 31;
  const int per = a.c.n_kv_heads * a.row_tiles;
  const int seq = blockIdx.x / per, p = blockIdx.x - seq * per;
  const int head = p % a.c.n_kv_heads, group_tile = p / a.c.n_kv_heads;
  if (threadIdx.x < 32) {
    Unit u{};
    const Lane mine = lane_steps(a, lane);
    find_unit(a, chunk_steps(a, lane, mine), -1, seq, lane, mine, u);
    if (lane == 0) shared_unit = u;
  }
  __syncthreads();
  const Unit u = shared_unit;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int r = threadIdx.x & 127, half = blockIdx.z;
  const int c4 = (blockIdx.y * 2 + (threadIdx.x >> 7)) * 4;  // of the row's float4 pieces
  const int R = group_tile * a.tile_rows + half * 128 + r, rows = a.n_tokens * a.group;
  if (u.n_chunks <= 1 || R >= rows) return;  // written by its block, or refused
  const int64_t unit0 = static_cast<int64_t>(u.base) * per + p;
  float m = -INFINITY;
  for (int x = 0; x < u.n_chunks; ++x)
    m = fmaxf(m, __ldcg(a.ml_part + (unit0 + static_cast<int64_t>(x) * per) * a.tile_rows +
                        half * 128 + r).x);
  const float mu = m == -INFINITY ? 0.f : m;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  float sum = 0.f;
#pragma unroll 2
  for (int x = 0; x < u.n_chunks; ++x) {
    const int64_t unit = unit0 + static_cast<int64_t>(x) * per;
    const float2 ml = __ldcg(a.ml_part + unit * a.tile_rows + half * 128 + r);
    const float4* src = reinterpret_cast<const float4*>(a.o_part) +
                        ((unit * (a.tile_rows / 128) + half) * (HD / 4) + c4) * 128 + r;
    const float f = exp2f(ml.x - mu);
    sum += ml.y * f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 y = __ldcg(src + i * 128);
      acc[4 * i] += y.x * f;
      acc[4 * i + 1] += y.y * f;
      acc[4 * i + 2] += y.z * f;
      acc[4 * i + 3] += y.w * f;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  const int t = R / a.group, i = R - t * a.group;
  uint16_t* dst = a.o + (static_cast<int64_t>(seq) * a.n_tokens + t) * a.o_stride +
                  (head * a.group + i) * HD + c4 * 4;
  uint32_t y[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) y[x] = pack_bf16x2(acc[2 * x] * inv, acc[2 * x + 1] * inv);
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
}

template <int FMT, int HD, bool VAR>
cudaError_t launch_tile(const Args& a, dim3 grid, cudaStream_t st) {
  using C = TileCfg<FMT, HD>;
  const cudaError_t ce =
      kernel_smem_attr(reinterpret_cast<const void*>(cache_attn_tile_kernel<FMT, HD, VAR>),
                       static_cast<int>(C::kSmem));
  if (ce != cudaSuccess) return ce;
  return launch_after(cache_attn_tile_kernel<FMT, HD, VAR>, grid, kTileThreads, C::kSmem, st, a);
}

template <int HD>
cudaError_t launch_tile_format(const Args& a, int format, dim3 grid, cudaStream_t st) {
  const bool var = a.cap > 0.f || a.window > 0;
  switch (format) {
    case PDS_KV_BF16:
      return var ? launch_tile<PDS_KV_BF16, HD, true>(a, grid, st)
                 : launch_tile<PDS_KV_BF16, HD, false>(a, grid, st);
    case PDS_KV_E4M3:
      return var ? launch_tile<PDS_KV_E4M3, HD, true>(a, grid, st)
                 : launch_tile<PDS_KV_E4M3, HD, false>(a, grid, st);
    default:
      return var ? launch_tile<PDS_KV_INT4, HD, true>(a, grid, st)
                 : launch_tile<PDS_KV_INT4, HD, false>(a, grid, st);
  }
}

}  // namespace

cudaError_t launch_tile_attention(const Args& a, int format, int hd, int64_t grid,
                                  cudaStream_t st) {
  const dim3 g(static_cast<unsigned>(grid));
  cudaError_t ce = hd == 128 ? launch_tile_format<128>(a, format, g, st)
                             : launch_tile_format<64>(a, format, g, st);
  if (ce != cudaSuccess || a.slots == 0) return ce;
  const dim3 jg(static_cast<unsigned>(a.c.n_seqs) * a.c.n_kv_heads * a.row_tiles, hd / 32,
                a.tile_rows / 128);
  return hd == 128 ? launch_after(cache_join_tile_kernel<128>, jg, 256, 0, st, a)
                   : launch_after(cache_join_tile_kernel<64>, jg, 256, 0, st, a);
}

}  // namespace pds
