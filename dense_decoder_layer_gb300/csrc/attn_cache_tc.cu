// Attention of drafted tokens over a cache when a kv head has many query rows
// (a tree of tens of tokens, a chunk of a prompt): the tcgen05 form of
// attn_cache.cu, same mathematics, same schedule of chunks.
//
// What bounds it: with R = T G query rows per cached row the products are
// 4 R hd flop against 2 hd bits/8 bytes, so beyond some 140 rows of an e4m3
// cache (280 of a bf16 one) the tensor pipe is the floor, below it HBM; in
// between stands the work per score -- exp2, packing, and for 8- and 4-bit rows
// the conversion to fp16 -- so the kernel is built to keep all of these running
// at once.
//
// Measured (replayed graphs): 256 tokens of 32/8 heads of 128 over 8192 bf16 rows
// 44.3 us (0.78 PFLOP/s), e4m3 56.5 (0.61); 64 tokens of 24/8 over 32768 4-bit rows
// 50.6 (0.51) as a chain, 3 more as a tree; 32 tokens of 4 sequences over 16384 bf16
// rows 50.8 (5.3 TB/s).  A tile of 64 keys for both streams takes ~1900 cycles with bf16 rows, ~2600 with
// codes.  With the softmax taken out it takes ~1500 (products with 64 columns
// read their 128 rows of Q from shared memory each time: 48 cycles where the
// multipliers need 32), with the products taken out nearly the whole time
// remains, so both must get shorter to gain.  16 softmax warps, two threads per
// row, were 2 to 4% slower; the streams half a tile apart made no difference;
// nor did longer or shorter chunks.  Some 10 us of each call are not the loop: Q's
// staging, the first tiles (fetching code), the epilogue and the join.
//
// One block of 640 threads per SM, two streams of 128 query rows, tiles of 64
// keys: with more than 128 rows the streams are two row tiles that share every
// K/V tile, else they are the even and the odd key tiles of one row tile.
// While one stream's softmax runs, the tensor pipe works for the other, and
// each stream has two score buffers.
//   warps 0, 1   tcgen05.mma issuers, one per stream: S = Q K^T into TMEM,
//                O += P V with P read from tensor memory (over its S) and V
//                MN-major from its rows
//   warps 4-7    K loaders, warps 8-11 V loaders (neither waits for the other's
//                stages): 16-byte asynchronous copies of cache rows; 8- and
//                4-bit codes land in slots private to their thread, which
//                turns them into the fp16 tile (no barrier in between)
//   warps 12-19  softmax, one thread per query row (so nothing is exchanged):
//                64 scores at a time, exponentials against the row's reference,
//                which moves only when a tile's weights sum to more than 2^8 (no
//                maximum is taken otherwise, and at most one per tile)
// The key's scales are applied to the scores (K) and to P (V): the tiles of 8-
// and 4-bit rows hold the codes themselves, in fp16.
//
// Every wait is bounded; a wait that gives up sets the status word and the
// block leaves in order.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "attn_cache.cuh"
#include "fastmath.cuh"
#include "sm100.cuh"
#include "tc.h"

namespace pds {
namespace {

using namespace cacheattn;

constexpr int kKeys = 64;              // keys per tile
constexpr int kTileRows = 128;         // query rows per stream
constexpr int kLoadWarps = 4, kLoadThreads = 32 * kLoadWarps;  // of K, and of V
constexpr int kFirstLoadWarp = 4, kFirstSoftmaxWarp = kFirstLoadWarp + 2 * kLoadWarps;
constexpr int kSoftmaxThreads = 256;   // 2 streams x 128 rows
constexpr int kTileThreads = 32 * kFirstSoftmaxWarp + kSoftmaxThreads;
constexpr uint32_t kAboveUnit = 256u, kFarFromUnit = 512u;  // beside a tile's unit
constexpr float kMoveSum = 256.0f;     // a tile's weights sum to more: the reference moves
// registers per thread: 96 at launch; 384 threads give up 32 each for the 256
// softmax threads' 48 more
constexpr int kLeanRegs = 64, kSoftmaxRegs = 144;
static_assert(kTileThreads * 96 >= 384 * kLeanRegs + kSoftmaxThreads * kSoftmaxRegs,
              "register split");

template <int FMT, int HD>
struct TileCfg {
  static constexpr bool kQuant = FMT != PDS_KV_BF16;
  static constexpr int kRow = FMT == PDS_KV_BF16 ? 2 * HD : FMT == PDS_KV_E4M3 ? HD : HD / 2;
  static constexpr uint32_t kQTile = 128u * HD * 2u;
  static constexpr uint32_t kTile = 64u * HD * 2u;         // bf16 tile of K or V
  static constexpr uint32_t kUnit = 64u * kRow;            // a tile's cached bytes
  static constexpr int kPerRow = kRow / 16;                // 16-byte pieces of a row
  static constexpr int kPieces = 64 * kPerRow / kLoadThreads;  // of a thread, per tile
  static_assert(kPieces >= 1, "every loader has a piece");
  // Stages of K and of V, and raw slots of each (8- and 4-bit tiles wait there).
  // Even numbers: streams over different key tiles then never share a stage,
  // so a stage's phases are waited for one after the other by one issuer.
  static constexpr int kKStages = 4;
  static constexpr int kVStages = HD == 64 ? 6 : kQuant ? 2 : 4;
  static_assert(kKStages % 2 == 0 && kVStages % 2 == 0, "stages of two streams");
  static constexpr int kRaw = FMT == PDS_KV_E4M3 && HD == 128 ? 3 : 4;
  // Ring of scale words, fetched with K's raw slots.  When K's tile j is turned
  // into its stage, S of tile j - kKStages is done, so (two score buffers, two
  // streams) the softmax is done with tile j - kKStages - 5; tile j + kRaw is
  // fetched next.
  static constexpr int kWordTiles = kKStages + kRaw + 5;
  // A tile's words: factors of K (64), of V (64), and O's unit they are for.
  static constexpr uint32_t kWordSlot = 528;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = 2 * kQTile;
  static constexpr uint32_t kV = kK + kKStages * kTile;
  static constexpr uint32_t kRawAt = kV + kVStages * kTile;   // K's slots, then V's
  static constexpr uint32_t kWords = kRawAt + (kQuant ? 2 * kRaw * kUnit : 0u);
  static constexpr uint32_t kZero = kWords + (kQuant ? kWordTiles * kWordSlot : 0u);  // int4: own words
  static constexpr uint32_t kZeroSlot = kPieces * kLoadThreads * 4u;
  static constexpr uint32_t kMask = kZero + (FMT == PDS_KV_INT4 ? 2 * kRaw * kZeroSlot : 0u);
  static constexpr uint32_t kPar = kMask + kMaskWords * 256u * 4u;
  static constexpr uint32_t kQMax = kPar + kMaxDraftTokens * 4u;  // Q's maximum per warp
  static constexpr uint32_t kQRow = kQMax + 64u;                  // exponents of rows of Q, bytes
  static constexpr uint32_t kUnitAt = kQRow + 256u;               // O's unit of each stream
  static constexpr uint32_t kBar = kUnitAt + 16u;
  static constexpr int kNumBars = 2 + 2 * (kKStages + kVStages) + 14;
  static constexpr uint32_t kMisc = kBar + 8u * kNumBars;
  static constexpr size_t kSmem = 1024 + kMisc + 96;
  static_assert(kSmem <= 232448, "shared memory per block");
  static constexpr uint32_t kTmS = 0, kTmO = 256, kTmemCols = 512;
};

// Matrix descriptors (128-byte swizzle): the high words are constants, the low
// ones an address in 16-byte units plus, for V, the leading offset.
//  * K-major operand of ROWS rows: 16 contraction elements are 32 bytes inside
//    a 128-byte column block, 4 per block, blocks ROWS x 128 bytes apart.
//  * V tile [64 keys][HD] as the MN-major B operand: rows are keys (128 bytes of
//    64 channels), 8-row groups 1024 bytes apart, channels 64..127 8 KB on.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kKMajorLo = 1u << 16, kVLo = (8192u >> 4) << 16;
template <int ROWS>
__host__ __device__ constexpr uint32_t kmajor_step(int x) {
  return (static_cast<uint32_t>(x >> 2) * (ROWS * 128u) + static_cast<uint32_t>(x & 3) * 32u) >> 4;
}
__host__ __device__ constexpr uint32_t v_step(int x) { return x * 16u * 128u >> 4; }

// Products and commits, by one elected thread of a converged warp (elect.sync
// picks the same one every time), with operands that the compiler knows to be
// the same in all lanes: they stay in uniform registers and a step costs an
// instruction or two.  Issued in a rolled loop from values it could not tell to
// be uniform, a step took ~110 cycles, and 256 rows over 8192 bf16 keys 52.3 us
// instead of 45.8.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
__device__ __forceinline__ int same_in_warp(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %4};\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(id), "r"(kDescHi), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t id,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(id), "r"(kDescHi), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// kind::f16 with both operands bf16 or both fp16, float32 accumulator.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn, bool bf16) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? (1u << 16) : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Byte offset of 8-channel piece c of row r in a swizzled bf16 tile of ROWS rows.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
  return static_cast<uint32_t>(c >> 3) * (ROWS * 128u) + r * 128u + (((c & 7) ^ (r & 7)) << 4);
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
// 64 consecutive float32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_load64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]),
        "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
        "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]),
        "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
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

// Whether the `keys` keys from key0 on hold rows that some query rows see
// and others do not (or rows past the end).
__device__ __forceinline__ bool part_hidden(const Args& a, int key0, int keys, int len) {
  return key0 + keys > len || (a.window > 0 && key0 < len + a.n_tokens - a.window);
}

// mbar_try_wait that may sleep up to `ns` (a hint) before it answers no: a warp
// that polls takes issue slots from those that work.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}
// The bounded wait of a converged warp; every lane returns the same.  Short on
// purpose: a block runs most of its code once and has to fetch it first, some
// hundred cycles per 128 bytes, and this appears in twenty places.
__device__ __forceinline__ bool warp_wait(bool ok, uint32_t bar, uint32_t parity,
                                          volatile int* abort_flag, uint32_t* status) {
  if (__all_sync(0xffffffffu, ok && sm100::mbar_try_wait(bar, parity))) return true;
  if (ok) {
    const uint64_t t0 = sm100::global_timer_ns();
    ok = false;
    do {
      if (mbar_try_wait_for(bar, parity, 100000u)) {
        ok = true;
        break;
      }
    } while (!*abort_flag && sm100::global_timer_ns() - t0 < sm100::kWaitLimitNs);
    if (!ok) {
      *abort_flag = 1;
      atomicOr(status, kStatusTimeout);
    }
  }
  return __all_sync(0xffffffffu, ok) != 0;
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
  const uint32_t bar_q_max = bar0 + 8u * (C::kNumBars - 1);  // (8- and 4-bit rows) Q's maximum
  constexpr int kBar2 = 1 + 2 * (C::kKStages + C::kVStages);
  // per stream s and score buffer b = i & 1 of its tile i, phase i >> 1: the
  // scores are there / P is there / O += P V has completed (a barrier per
  // buffer keeps every wait within one phase); per stream: all of it is done
  auto bar_s_full = [&](int s, int b) { return bar0 + 8u * (kBar2 + 2 * s + b); };
  auto bar_p_full = [&](int s, int b) { return bar0 + 8u * (kBar2 + 4 + 2 * s + b); };
  auto bar_pv = [&](int s, int b) { return bar0 + 8u * (kBar2 + 8 + 2 * s + b); };
  auto bar_done = [&](int s) { return bar0 + 8u * (kBar2 + 12 + s); };
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
  if (C::kQuant && threadIdx.x < 64) reinterpret_cast<uint32_t*>(smem + C::kQRow)[threadIdx.x] = 0u;
  if (threadIdx.x == 0) {
    mbar_init(bar_q, kSoftmaxThreads / 32);
    mbar_init(bar_q_max, kSoftmaxThreads / 32);
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(bar_k_full(i), kLoadWarps);
      mbar_init(bar_k_empty(i), two_tiles ? 2 : 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(bar_v_full(i), kLoadWarps);
      mbar_init(bar_v_empty(i), two_tiles ? 2 : 1);
    }
    for (int s = 0; s < 2; ++s) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(bar_s_full(s, b), 1);
        mbar_init(bar_p_full(s, b), 4);  // one arrival per softmax warp
        mbar_init(bar_pv(s, b), 1);
      }
      mbar_init(bar_done(s), 1);
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
  const bool many = a.slots > 0 && a.c.n_seqs > 1 && !a.fit;
  Share share{};
  if (many) share = block_share(a, smem + C::kK);  // (nothing is there yet)
  if (warp == 0) {
    Unit u{};
    bool ok;
    if (a.slots == 0 || (many && w < a.c.n_seqs)) {
      ok = many ? first_unit(a, share, w, u) : whole_unit(a, w, u);
      if (!ok && p == 0 && lane == 0) atomicOr(a.status, kStatusBadLength);
    } else if (many) {
      ok = later_unit(a, share, w - a.c.n_seqs, lane, u);
    } else if (a.c.n_seqs == 1) {
      ok = only_unit(a, w, u);
    } else {
      const Lane mine = lane_steps(a, lane);
      ok = find_unit(a, chunk_steps(a, lane, mine), w, 0, lane, mine, u);
    }
    if (lane == 0) {
      *shared_unit = u;
      *shared_ok = ok;
    }
    if (a.slots > 0 && !many && blockIdx.x == 0) {  // report lengths that do not fit
      bool bad = false;
#pragma unroll 1
      for (int s = lane; s < a.c.n_seqs; s += 32) bad |= lane_steps(a, s).n == 0;
      if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kStatusBadLength);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const struct { int seq, n_chunks, first, n_steps, len; } u = {
      shared_unit->seq, shared_unit->n_chunks, shared_unit->first, shared_unit->n_steps,
      shared_unit->len};
  // (a block without a unit walks through with no tiles)
  const int n = *shared_ok ? u.n_steps : 0;
  const int len = u.len, end = len + a.n_tokens;
  const int n_tiles0 = two_tiles ? n : (n + 1) / 2, n_tiles1 = two_tiles ? n : n / 2;
  auto tile_of = [&](int s, int i) { return two_tiles ? i : 2 * i + s; };

  if (warp < kFirstLoadWarp) {
    setmaxnreg_dec<kLeanRegs>();
    if (warp < 2 && n > 0) {
      // One issuer per stream: their products interleave on the tensor pipe, so
      // one's waits cost the other nothing.  Per tile: S_i into the buffer that
      // P_{i-2} has left, then O += P_{i-1} V_{i-1} once the softmax has made P.
      constexpr uint32_t kIdS = idesc(128, kKeys, false, !C::kQuant);
      constexpr uint32_t kIdPV = idesc(128, HD, true, !C::kQuant);
      const int s = same_in_warp(warp);
      const int tiles = same_in_warp(s == 0 ? n_tiles0 : n_tiles1);
      const int step = same_in_warp(two_tiles ? 1 : 2);
      const uint32_t tm = same_in_warp(tmem), sb = same_in_warp(sbase);
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return ok = warp_wait(ok, bar, parity, abort_flag, a.status);
      };
      const uint32_t q = ((sb + C::kQ + (step == 1 ? s * C::kQTile : 0u)) >> 4) | kKMajorLo;
      const uint32_t scores_at = tm + C::kTmS + s * 128u, o_at = tm + C::kTmO + s * 128u;
      // stages and phases of the tile whose S / P V comes next
      int k_st = step == 1 ? 0 : s, v_st = k_st;
      uint32_t k_phase = 0, v_phase = 0;
      wait(bar_q, 0);
      for (int i = 0; ok && i <= tiles; ++i) {
        const uint32_t b = i & 1;
        if (i < tiles) {
          if (i >= 2 && !wait(bar_pv(s, b), ((i >> 1) - 1) & 1)) break;
          if (!wait(bar_k_full(k_st), k_phase)) break;
          tc_fence_after();
          const uint32_t k = ((sb + C::kK + k_st * C::kTile) >> 4) | kKMajorLo;
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < HD / 16; ++x)
              mma_ss(scores_at + b * 64u, q + kmajor_step<128>(x), k + kmajor_step<64>(x), kIdS,
                     x > 0);
            mma_commit(bar_s_full(s, b));
            mma_commit(bar_k_empty(k_st));
          }
          __syncwarp();
          if ((k_st += step) >= C::kKStages) k_st -= C::kKStages, k_phase ^= 1u;
        }
        if (i >= 1) {
          const int e = i - 1;
          if (!wait(bar_v_full(v_st), v_phase)) break;
          if (!wait(bar_p_full(s, e & 1), (e >> 1) & 1)) break;
          tc_fence_after();
          const uint32_t v = ((sb + C::kV + v_st * C::kTile) >> 4) | kVLo;
          const uint32_t p_at = scores_at + (e & 1) * 64u;
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < kKeys / 16; ++x)
              mma_ts(o_at, p_at + x * 8u, v + v_step(x), kIdPV, e > 0 || x > 0);
            mma_commit(bar_pv(s, e & 1));
            mma_commit(bar_v_empty(v_st));
          }
          __syncwarp();
          if ((v_st += step) >= C::kVStages) v_st -= C::kVStages, v_phase ^= 1u;
        }
      }
      if (elect_one()) mma_commit(bar_done(s));
      __syncwarp();
      int dummy = 0;
      warp_wait(true, bar_done(s), 0, &dummy, a.status);
    }
  } else if (warp < kFirstSoftmaxWarp) {
    setmaxnreg_dec<kLeanRegs>();
    const bool is_v = warp >= kFirstLoadWarp + kLoadWarps;
    const int tid = (threadIdx.x - 32 * kFirstLoadWarp) & (kLoadThreads - 1);
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = warp_wait(ok, bar, parity, abort_flag, a.status);
    };
    auto arrive = [&](uint32_t bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // this thread's pieces of a tile: rows row0 + i kRowStep, 16-byte column col
    constexpr int kRowStep = kLoadThreads / C::kPerRow;
    const int col = tid % C::kPerRow, row0 = tid / C::kPerRow;
    const char* src0 = (is_v ? a.c.v : a.c.k) + u.seq * a.c.seq_stride + head * a.c.head_stride +
                       col * 16;
    const int64_t word0 = (static_cast<int64_t>(u.seq) * a.c.n_kv_heads + head) * a.c.capacity;
    const int stages = is_v ? C::kVStages : C::kKStages;
    const uint32_t tiles_at = sbase + (is_v ? C::kV : C::kK);
    const uint32_t full0 = is_v ? bar_v_full(0) : bar_k_full(0);
    const uint32_t empty0 = is_v ? bar_v_empty(0) : bar_k_empty(0);
    const uint32_t raw0 = sbase + C::kRawAt + (is_v ? C::kRaw * C::kUnit : 0u) + tid * 16u;
    const uint32_t zero0 = sbase + C::kZero + (is_v ? C::kRaw * C::kZeroSlot : 0u) + tid * 4u;
    // copy tile t: bf16 rows to their places in the tile at `dst`, codes to this
    // thread's slots from `dst` on
    static_assert(C::kQuant || kRowStep % 8 == 0, "a thread's pieces are swizzled alike");
    const uint32_t piece0 = C::kQuant ? 0u : tile_at<64>(row0, col);
    constexpr uint32_t kPieceStep = C::kQuant ? kLoadThreads * 16u : kRowStep * 128u;
    const int64_t row_step = kRowStep * a.c.row_stride;
    auto issue = [&](int t, uint32_t dst, int slot) {
      if (t < n && ok) {
        const int key0 = (u.first + t) * kKeys;
        const char* from = src0 + static_cast<int64_t>(key0 + row0) * a.c.row_stride;
        const uint32_t* word = (is_v ? a.c.v_scale : a.c.k_scale) + word0 + key0 + row0;
        const uint32_t zero = zero0 + slot * C::kZeroSlot;
        if (key0 + kKeys <= end) {
#pragma unroll
          for (int i = 0; i < C::kPieces; ++i) {
            copy16(dst + piece0 + i * kPieceStep, from, true);
            from += row_step;
            if constexpr (FMT == PDS_KV_INT4)
              copy4(zero + i * (kLoadThreads * 4u), word + i * kRowStep, true);
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < C::kPieces; ++i) {
            // a row past the end is not read: its address is the sequence's first
            const bool live = key0 + row0 + i * kRowStep < end;
            copy16(dst + piece0 + i * kPieceStep, live ? from : src0, live);
            from += row_step;
            if constexpr (FMT == PDS_KV_INT4)
              copy4(zero + i * (kLoadThreads * 4u),
                    live ? word + i * kRowStep : word - (key0 + row0), live);
          }
        }
        if (C::kQuant && !is_v) {  // the tile's scale words: K's by 64 threads, V's by 32
          const uint32_t at = sbase + C::kWords + (t % C::kWordTiles) * C::kWordSlot;
          const int key = key0 + (tid & 63);
          if (tid < 96)
            copy4(at + tid * 4u, (tid < 64 ? a.c.k_scale : a.c.v_scale) + word0 +
                                     (key < end ? key : end - 1), key < end);
          if (tid >= 64 && tid < 96) {
            const int next = key + 32;
            copy4(at + (tid + 32) * 4u, a.c.v_scale + word0 + (next < end ? next : end - 1),
                  next < end);
          }
        }
      }
      copies_commit();
    };
    if constexpr (!C::kQuant) {
      // a tile is handed over once the copies of the next two have been issued
      int st = 0, st_done = 0;
      uint32_t phase = 1;  // of the stage's release; the first round passes at once
      for (int t = 0; t <= n + 1 && ok; ++t) {
        if (t < n) {
          if (t >= stages) wait(empty0 + 8u * st, phase);
          issue(t, tiles_at + st * C::kTile, 0);
          if (++st == stages) st = 0, phase ^= 1u;
        } else {
          copies_commit();
        }
        if (t < 2) continue;
        copies_wait<2>();
        if (is_v && part_hidden(a, (u.first + t - 2) * kKeys, kKeys, len)) {
          // Rows that some query rows must not see: an infinity or a NaN would
          // reach them through a zero weight.  It is taken out here and added
          // to the rows that do see it at the end.
#pragma unroll 1
          for (int i = 0; i < C::kPieces; ++i) {
            const uint32_t d = tiles_at + st_done * C::kTile + tile_at<64>(row0 + i * kRowStep, col);
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
        arrive(full0 + 8u * st_done);
        if (++st_done == stages) st_done = 0;
      }
    } else {
#pragma unroll 1
      for (int t = 0; t < C::kRaw; ++t) issue(t, raw0 + t * C::kUnit, t);
      int st = 0, slot = 0;
      uint32_t phase = 1, v_exp = kMinScaleExp;
      float k_factor = a.scale_log2;
      if (!is_v && n > 0) {  // Q's multiplier, once its maximum is there
        wait(bar_q_max, 0);
        uint32_t top = 0u;
        const uint32_t* q_max = reinterpret_cast<const uint32_t*>(smem + C::kQMax);
#pragma unroll 1
        for (int x = 0; x < kSoftmaxThreads / 32; ++x) top = max(top, q_max[x]);
        k_factor *= q_inverse(q_block_exponent(top));
      }
      for (int t = 0; t < n && ok; ++t) {
        copies_wait<C::kRaw - 1>();
        if (t >= stages) wait(empty0 + 8u * st, phase);
        if (!ok) break;
        const uint32_t src = raw0 + slot * C::kUnit;
        const uint32_t dst = tiles_at + st * C::kTile;
        const int key0 = (u.first + t) * kKeys;
        const bool clean = FMT == PDS_KV_E4M3 && is_v && part_hidden(a, key0, kKeys, len);
#pragma unroll
        for (int i = 0; i < C::kPieces; ++i) {
          const int r = row0 + i * kRowStep;
          const uint4 x = lds128(src + i * (kLoadThreads * 16u));
          uint32_t c[4] = {x.x, x.y, x.z, x.w};
          if constexpr (FMT == PDS_KV_E4M3) {
            if (clean) {
#pragma unroll
              for (int e = 0; e < 4; ++e) c[e] = e4m3_finite(c[e]);
            }
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) e4m3_pairs(c[e], y[2 * e], y[2 * e + 1]);
            // the two halves in an order that keeps the lanes of a row on different banks
            const bool swap = col & (C::kPerRow >> 1);
            const uint32_t d0 = dst + tile_at<64>(r, 2 * col), d1 = dst + tile_at<64>(r, 2 * col + 1);
            st_shared_u4(swap ? d1 : d0, swap ? y[4] : y[0], swap ? y[5] : y[1],
                         swap ? y[6] : y[2], swap ? y[7] : y[3]);
            st_shared_u4(swap ? d0 : d1, swap ? y[0] : y[4], swap ? y[1] : y[5],
                         swap ? y[2] : y[6], swap ? y[3] : y[7]);
          } else {
            // a word's 8 channels in the order 0 4 1 5 2 6 3 7 (Q's and O's are the same)
            const uint32_t w = lds32(zero0 + slot * C::kZeroSlot + i * (kLoadThreads * 4u));
            const uint32_t z = int4_zero(w, w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              st_shared_u4(dst + tile_at<64>(r, 4 * col + e), int4_lo(c[e], z), int4_hi(c[e], z),
                           int4_lo(c[e] >> 8, z), int4_hi(c[e] >> 8, z));
          }
        }
        if (!is_v) {
          // the scale words as factors: of scores in powers of two, and of P in
          // O's unit, which grows with the largest V scale
          float* word = reinterpret_cast<float*>(smem + C::kWords +
                                                 (t % C::kWordTiles) * C::kWordSlot);
          auto scale = [&](int x) {
            const uint32_t bits = __float_as_uint(word[x]);
            return __uint_as_float(FMT == PDS_KV_INT4 ? bits & 0xffff0000u : bits);
          };
          if (tid < 64) {
            word[tid] = scale(tid) * k_factor;
          } else if (tid < 96) {
            const float v0 = scale(tid), v1 = scale(tid + 32);
            // (a padding token's row is not written: it may hold any scale)
            auto counts = [&](int key) {
              return key < len || (key < end && !(a.parents && a.parents[static_cast<int64_t>(u.seq) *
                                                                         a.n_tokens + key - len] < -1));
            };
            const bool c0 = counts(key0 + tid - 64), c1 = counts(key0 + tid - 32);
            const uint32_t e0 = finite_bits(v0) >> 23, e1 = finite_bits(v1) >> 23;
            const uint32_t most = __reduce_max_sync(0xffffffffu, max(c0 ? e0 : 0u, c1 ? e1 : 0u));
            const uint32_t least = __reduce_min_sync(0xffffffffu, min(c0 ? e0 : 255u, c1 ? e1 : 255u));
            v_exp = max(v_exp, min(most, kMaxScaleExp));
            // What the softmax has to look at: scales above the unit (in this tile), or
            // far from it (where it looks at this tile's maximum).
            const uint32_t flags = (most > v_exp ? kAboveUnit : 0u) |
                                   (most > v_exp || least + 4u < v_exp ? kFarFromUnit : 0u);
            const float f = v_multiplier(v_exp);
            word[tid] = v0 * f;
            word[tid + 32] = v1 * f;
            if (tid == 64) word[128] = __uint_as_float(v_exp | flags);
          }
        }
        arrive(full0 + 8u * st);
        issue(t + C::kRaw, src, slot);  // into the slot this thread has just emptied
        if (++st == stages) st = 0, phase ^= 1u;
        if (++slot == C::kRaw) slot = 0;
      }
    }
    copies_wait<0>();
  } else {
    setmaxnreg_inc<kSoftmaxRegs>();
    const int tid = threadIdx.x - 32 * kFirstSoftmaxWarp;
    const int s = tid >> 7;                       // stream
    const int r = tid & 127;                      // row of the stream's tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lane_off + C::kTmO + s * 128u;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = warp_wait(ok, bar, parity, abort_flag, a.status);
      if (ok) tc_fence_after();
    };
    // Q into its (one or two) tiles, in 8-channel pieces; fp16 where the rows are
    // codes: each thread then converts the pieces it has copied, in place.
    // (Loops rolled by four: this runs once, and fetching its code costs as
    // much as its latencies.)
    if (n > 0) {
      constexpr int kPieces = HD / 8;
      constexpr int kStep = kSoftmaxThreads / kPieces;  // rows from one piece of a thread to its next
      static_assert(kStep % 8 == 0, "a thread's pieces are swizzled alike");
      const int q_rows = two_tiles ? 256 : 128, row0 = tid / kPieces, col = tid % kPieces;
      const uint32_t at0 = sbase + C::kQ + tile_at<128>(row0, col);
      auto place = [&](int row) {  // of this thread's piece of row `row`
        return at0 + static_cast<uint32_t>(row >> 7) * C::kQTile +
               static_cast<uint32_t>((row & 127) - row0) * 128u;
      };
      const uint16_t* src = a.q + static_cast<int64_t>(u.seq) * a.n_tokens * a.q_stride +
                            head * a.group * HD + col * 8;
#pragma unroll 4
      for (int row = row0; row < q_rows; row += kStep) {
        const int R = r0 + row;
        const bool live = R < rows;  // rows past the last are zero
        const int t = live ? token_of(a, R) : 0, h = live ? R - t * a.group : 0;
        copy16(place(row), src + t * a.q_stride + h * HD, live);
      }
      copies_commit();
      copies_wait<0>();
      if constexpr (C::kQuant) {
        // bits of the largest |value|, two at a time; over again without the
        // infinities and NaN if there are any
        auto piece_max = [&](int row) -> uint32_t {
          const uint4 x = lds128(place(row));
          const uint32_t pair = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                         __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
          return max(pair & 0xffffu, pair >> 16);
        };
        auto finite_piece_max = [&](int row) -> uint32_t {
          const uint4 x = lds128(place(row));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          uint32_t most = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            most = max(most, max(finite_bits(__uint_as_float(w[e] << 16)),
                                 finite_bits(__uint_as_float(w[e] & 0xffff0000u))));
          return most >> 16;
        };
        uint32_t top = 0u, least = 0xffffu;  // of the pieces; the least that is not zero
#pragma unroll 4
        for (int row = row0; row < q_rows; row += kStep) {
          const uint32_t most = piece_max(row);
          top = max(top, most);
          least = min(least, most - 1u);  // (zero goes to the top)
        }
        if (__any_sync(0xffffffffu, top >= 0x7f80u)) {
          top = 0u;
#pragma unroll 1
          for (int row = row0; row < q_rows; row += kStep) top = max(top, finite_piece_max(row));
          least = 0u;
        }
        uint32_t* q_max = reinterpret_cast<uint32_t*>(smem + C::kQMax);
        top = __reduce_max_sync(0xffffffffu, top << 16);
        if (lane == 0) {
          q_max[warp - kFirstSoftmaxWarp] = top;
          mbar_arrive(bar_q_max);
        }
        named_bar_sync(1, kSoftmaxThreads);
#pragma unroll 1
        for (int c = 0; c < kSoftmaxThreads / 32; ++c) top = max(top, q_max[c]);
        const uint32_t block = q_block_exponent(top);
        // Rows that may not take the block's multiplier: some piece of theirs is far
        // below it, or the block's largest above it.  (A row's pieces are neighbouring
        // lanes of one warp.)
        uint8_t* q_row = smem + C::kQRow;  // exponents of such rows, else 0
        if (__any_sync(0xffffffffu, ((least + 1u) >> 7) + 8u < block || (top >> 23) > block)) {
#pragma unroll 1
          for (int row = row0; row < q_rows; row += kStep) {
            uint32_t most = finite_piece_max(row);
#pragma unroll
            for (int o = 1; o < kPieces; o <<= 1)
              most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
            const uint32_t e = q_row_exponent(most << 16, block);
            if (col == 0 && e != block) q_row[row] = static_cast<uint8_t>(e);
          }
          __syncwarp();
        }
        const float q_block = q_multiplier(block);
#pragma unroll 4
        for (int row = row0; row < q_rows; row += kStep) {
          const uint4 x = lds128(place(row));
          const uint32_t own = q_row[row];
          const float q_mul = own ? q_multiplier(own) : q_block;
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
          float f[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(w[e] << 16) * q_mul;
            f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * q_mul;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = FMT == PDS_KV_INT4 ? pack_f16x2(f[e], f[e + 4])
                                      : pack_f16x2(f[2 * e], f[2 * e + 1]);
          st_shared_u4(place(row), w[0], w[1], w[2], w[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q);
    }
    // the row's token: its ancestors (within the window) as bits of its own
    // column of the mask table, and the first cached row it sees
    const int R = r0 + (two_tiles ? s * kTileRows : 0) + r;
    const bool row_live = R < rows;
    const int tok = row_live ? token_of(a, R) : 0;
    int32_t* par = reinterpret_cast<int32_t*>(smem + C::kPar);
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + C::kMask) + s * 128 + r;
    if (n > 0 && a.parents && tid < a.n_tokens)
      par[tid] = a.parents[static_cast<int64_t>(u.seq) * a.n_tokens + tid];
    named_bar_sync(1, kSoftmaxThreads);
    // what the row's scores are multiplied by, besides the block's factor
    float q_ratio = 1.f;
    if constexpr (C::kQuant) {
      if (n > 0) {
        const uint32_t own = smem[C::kQRow + (two_tiles ? s * kTileRows : 0) + r];
        if (own) {
          uint32_t top = 0u;
          const uint32_t* q_max = reinterpret_cast<const uint32_t*>(smem + C::kQMax);
#pragma unroll 1
          for (int c = 0; c < kSoftmaxThreads / 32; ++c) top = max(top, q_max[c]);
          q_ratio = q_inverse(own) * q_multiplier(q_block_exponent(top));
        }
      }
    }
    const bool ratios = C::kQuant && __any_sync(0xffffffffu, q_ratio != 1.f);
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
        const int left = a.window > 0 ? min(a.window, depth + 1) : depth + 1;  // itself counts
        if (a.parents) {
          int x = tok;
          for (int e = 0; e < left; ++e, x = par[x])
#pragma unroll
            for (int i = 0; i < kMaskWords; ++i)
              if ((x >> 5) == i) bits[i] |= 1u << (x & 31);
        } else {  // tokens tok - left + 1 .. tok
#pragma unroll
          for (int i = 0; i < kMaskWords; ++i) {
            const int hi = tok - 32 * i, lo = hi - left + 1;
            if (hi >= 0 && lo < 32)
              bits[i] = (hi >= 31 ? 0xffffffffu : (2u << hi) - 1u) & ~(lo > 0 ? (1u << lo) - 1u : 0u);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kMaskWords; ++i) mask[i * 256] = bits[i];  // (read by this thread alone)
    }
    const int lo = VAR && a.window > 0 ? len + depth - a.window + 1 : 0;

    const bool warp_live = r0 + (two_tiles ? s * kTileRows : 0) + (warp & 3) * 32 < rows;
    const float sc = a.scale_log2;
    const SoftCap cap = soft_cap(VAR ? a.cap * a.scale_log2 : 0.f);  // (in powers of two)
    float m_ref = -INFINITY, l = 0.f;
    uint32_t v_exp = kMinScaleExp;  // O's unit: the exponent of the largest V scale so far
    const int n_mine = s == 0 ? n_tiles0 : n_tiles1;
    const int tile_step = two_tiles ? 1 : 2;
    int slot = two_tiles ? 0 : s;                     // of the tile's scale words
    int key0 = (u.first + slot) * kKeys;              // the tile's first key
    // tiles from a key below the one, or above the other, on hold rows that are
    // hidden from some
    const int hide_lo = VAR && a.window > 0 ? len + a.n_tokens - a.window : 0;
    const int hide_hi = len - kKeys;
    for (int i = 0; i < n_mine; ++i) {
      const int b = i & 1;
      const uint32_t words = sbase + C::kWords + slot * C::kWordSlot;
      const int key = key0;
      slot += tile_step;
      if (slot >= C::kWordTiles) slot -= C::kWordTiles;
      key0 += tile_step * kKeys;
      wait(bar_s_full(s, b), (i >> 1) & 1);
      if (!ok) break;
      if (!warp_live) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full(s, b));
        continue;
      }
      const uint32_t ts = tmem + lane_off + C::kTmS + s * 128u + b * 64u;
      const bool partial = key > hide_hi || key < hide_lo, special = partial || ratios;
      uint32_t vis[2] = {0xffffffffu, 0xffffffffu};
      if (partial) {
        vis[0] = visible32(key, len, lo, mask);
        vis[1] = visible32(key + 32, len, lo, mask);
      }
      uint32_t unit = v_exp;
      if constexpr (C::kQuant) unit = lds32(words + 512u);
      float z[kKeys];
      // Scores less the reference, in powers of two, and their exponentials.  The
      // maximum is only taken where the row has no reference yet, its weights have
      // outgrown the old one, which their sum tells, or V's unit has grown; at most once,
      // because what is multiplied behind it is bounded by construction: the reference
      // is the largest of the rounded scores (over codes, of their levels) and is
      // subtracted from these.  (The fused
      // difference of the first pass also holds what the product's rounding drops,
      // which from 2^28 on is above 8 now and then: as a measure of growth that
      // would never end, from 2^31 on as a weight it would be nothing or infinite.)
      bool move = __any_sync(0xffffffffu, m_ref == -INFINITY || (unit & ~kFarFromUnit) != v_exp);
      bool rounded = move;
      float grown, pk[kKeys / 2];
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {  // weights; the maximum; weights again
        const float less = rounded ? 0.f : m_ref;
        auto scores = [&](bool times_ratio) {
          tmem_load64(ts, z);
          if (times_ratio) {
#pragma unroll
            for (int x = 0; x < kKeys / 2; ++x) mul2(z[2 * x], z[2 * x + 1], q_ratio, q_ratio);
          }
          if (VAR && cap.c > 0.f) {
            auto apply = [&](auto&& one) {
#pragma unroll
              for (int x = 0; x < kKeys; ++x) {
                float f = sc;
                if constexpr (C::kQuant) f = __uint_as_float(lds32(words + x * 4));
                z[x] = one(z[x] * f, cap) - less;
              }
            };
            if (cap.wide())
              apply([](float y, const SoftCap& k) { return capped_wide(y, k); });
            else
              apply([](float y, const SoftCap& k) { return capped(y, k); });
          } else if constexpr (C::kQuant) {
#pragma unroll
            for (int x = 0; x < kKeys / 4; ++x) {
              const float4 f = ld_shared_f4(words + x * 16);
              fma2_pair(z[4 * x], z[4 * x + 1], f.x, f.y, -less);
              fma2_pair(z[4 * x + 2], z[4 * x + 3], f.z, f.w, -less);
            }
          } else {
#pragma unroll
            for (int x = 0; x < kKeys / 2; ++x) fma2(z[2 * x], z[2 * x + 1], sc, -less);
          }
        };
        scores(false);
        if (special) {
          if (C::kQuant && ratios) scores(true);  // (rarely: so the others do not ask twice)
#pragma unroll
          for (int x = 0; x < kKeys; ++x)
            if (!((vis[x >> 5] >> (x & 31)) & 1u)) z[x] = -INFINITY;
        }
        if (move) {
          float alpha = 1.f, mx;
          if constexpr (C::kQuant) {
            const uint32_t v_new = unit & 255u;
            const int d = static_cast<int>(v_new - v_exp), k = unit_shift(d, l);
            v_exp = v_new;
            alpha = exp2_fast(static_cast<float>(k - d));
            m_ref -= static_cast<float>(k);
            l *= exp2_fast(static_cast<float>(k));
          }
          if (!C::kQuant || !(unit & kFarFromUnit)) {
            mx = fmaxf(max32(z), max32(z + 32));
          } else {
            float level[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) level[x] = -INFINITY;
#pragma unroll
            for (int x = 0; x < kKeys / 4; ++x) {
              const float4 f = ld_shared_f4(words + 256u + x * 16);
              // (a factor is its scale over the unit, times 2^6)
              auto shift = [&](float v) { return level_shift(__float_as_uint(v) << 1 >> 24, 133u); };
              float* y = level + 4 * (x & 1);
              y[0] = fmaxf(y[0], z[4 * x] + shift(f.x));
              y[1] = fmaxf(y[1], z[4 * x + 1] + shift(f.y));
              y[2] = fmaxf(y[2], z[4 * x + 2] + shift(f.z));
              y[3] = fmaxf(y[3], z[4 * x + 3] + shift(f.w));
            }
            mx = fmaxf(max3(level[0], level[1], level[2]), max3(level[3], level[4], level[5]));
            mx = max3(mx, level[6], level[7]);
          }
          if (mx > m_ref) {
            const float f = exp2_fast(m_ref - mx);  // 0 from -inf
            m_ref = mx;
            l *= f;
            alpha *= f;
          }
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O at rest: the product of the tile before has completed
            wait(bar_pv(s, b ^ 1), ((i - 1) >> 1) & 1);
            if (!ok) break;
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {
              float o[16];
              tmem_load16(to + c * 16, o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] *= alpha;
              tmem_store16(to + c * 16, o);
            }
          }
          move = false;
          // (bf16 rows: held on from here beside O and P, the scores would not fit
          // the registers, so they are loaded again)
          if constexpr (!C::kQuant) continue;
        }
        if (rounded) {
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;  // masked scores give 0
#pragma unroll
          for (int x = 0; x < kKeys / 2; ++x) add2(z[2 * x], z[2 * x + 1], -m_use, -m_use);
        }
        float sum[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) sum[x] = 0.f;
#pragma unroll
        for (int x = 0; x < kKeys / 8; ++x) {
          float* y = z + 8 * x;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = exp2_fast(y[e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) add2(sum[2 * e], sum[2 * e + 1], y[2 * e], y[2 * e + 1]);
          if constexpr (!C::kQuant) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pk[4 * x + e] = __uint_as_float(pack_bf16x2(y[2 * e], y[2 * e + 1]));
          }
        }
        grown = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
        if (rounded) break;
        move = rounded = __any_sync(0xffffffffu, grown > kMoveSum);
        if (!move) break;
      }
      if (!ok) break;
      l += grown;
      if constexpr (C::kQuant) {
#pragma unroll
        for (int x = 0; x < kKeys / 4; ++x) {
          const float4 f = ld_shared_f4(words + 256u + x * 16);
          mul2(z[4 * x], z[4 * x + 1], f.x, f.y);
          mul2(z[4 * x + 2], z[4 * x + 3], f.z, f.w);
        }
        if (partial) {  // a hidden row may have any scale, a NaN too
#pragma unroll
          for (int x = 0; x < kKeys; ++x)
            if (!((vis[x >> 5] >> (x & 31)) & 1u)) z[x] = 0.f;
        }
#pragma unroll
        for (int x = 0; x < kKeys / 2; ++x)
          pk[x] = __uint_as_float(pack_f16x2(z[2 * x], z[2 * x + 1]));
      }
      tmem_store32(ts, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p_full(s, b));
    }

    // ---- the rows' results
    if (n > 0) {
      wait(bar_done(0), 0);
      wait(bar_done(1), 0);
    }
    // Where the streams hold the same rows over different keys, each takes half
    // of the columns and gives the other half away.  Every product is done: the
    // spaces of Q and K are free.
    float2* ml = reinterpret_cast<float2*>(smem + C::kK);  // [stream][row]
    ml[s * 128 + r] = make_float2(m_ref, l);
    // (a stream's warps all have the same unit, but for those without rows)
    float* unit_of = reinterpret_cast<float*>(smem + C::kUnitAt);
    const float my_unit = C::kQuant && n_mine > 0 ? v_inverse(v_exp) : 1.f;
    if (r == 0) unit_of[s] = my_unit;
    const uint32_t xch = sbase + C::kQ;
    const uint32_t mine_at = static_cast<uint32_t>(r) * (HD * 2);
    auto xch_at = [&](int c4) {  // float4 c4 of the row's given half, spread over the banks
      return mine_at + (static_cast<uint32_t>(c4 ^ (r & (HD / 8 - 1))) << 4);
    };
    if (!two_tiles && ok && warp_live) {
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        float o[16];
        tmem_load16(to + (s == 0 ? HD / 2 : 0) + c * 16, o);
        const bool none = n_mine == 0;  // its accumulator was never written
#pragma unroll
        for (int x = 0; x < 4; ++x)
          st_shared_f4(xch + s * (64u * HD * 4u) + xch_at(4 * c + x),
                       none ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
      }
    }
    named_bar_sync(1, kSoftmaxThreads);
    float mine_f = my_unit, other_f = 0.f;  // factors of this stream's O and of the other's
    int c0 = 0, c1 = HD;                    // this thread's columns
    if (!two_tiles) {
      const float2 x0 = ml[(1 - s) * 128 + r];
      const float m = fmaxf(m_ref, x0.x), mu = m == -INFINITY ? 0.f : m;
      mine_f = exp2_fast(m_ref - mu);
      other_f = exp2_fast(x0.x - mu);
      // the first stream's share first, whichever thread adds
      l = s == 0 ? l * mine_f + x0.y * other_f : x0.y * other_f + l * mine_f;
      mine_f *= my_unit;
      other_f *= unit_of[1 - s];
      m_ref = m;
      c0 = s * (HD / 2);
      c1 = c0 + HD / 2;
    }
    if (ok && warp_live && n > 0) {
      const bool pad = depth < 0, whole = u.n_chunks == 1;
      const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row that sees nothing is zero
      const int i = R - tok * a.group;
      uint16_t* dst = a.o + (static_cast<int64_t>(u.seq) * a.n_tokens + tok) * a.o_stride +
                      (head * a.group + i) * HD;
      const int half = two_tiles ? s : 0;
      float4* out = reinterpret_cast<float4*>(a.o_part) +
                    (static_cast<int64_t>(blockIdx.x) * (a.tile_rows / 128) + half) * (HD / 4) * 128;
#pragma unroll 1
      for (int c = c0; c < c1; c += 16) {
        float o[16];
        tmem_load16(to + c, o);
        if (!two_tiles) {
          const bool none = n_mine == 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float4 y = ld_shared_f4(xch + (1 - s) * (64u * HD * 4u) +
                                          xch_at((c - s * (HD / 2)) / 4 + x));
            const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float mine_o = none ? 0.f : o[4 * x + e] * mine_f, other_o = v[e] * other_f;
              o[4 * x + e] = s == 0 ? mine_o + other_o : other_o + mine_o;
            }
          }
        } else if (C::kQuant) {
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] *= mine_f;
        }
        if constexpr (FMT == PDS_KV_INT4) {  // the channels back in their order
          float y[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) y[x] = o[(x & 8) + ((x & 3) << 1) + ((x >> 2) & 1)];
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] = y[x];
        }
        if constexpr (!C::kQuant) {
          if (*poison && row_live) {  // what the loaders took out, for the rows that see it
            for (int t = 0; t < n; ++t) {
              const int key0 = (u.first + t) * kKeys;
              if (!part_hidden(a, key0, kKeys, len)) continue;
              for (int g = 0; g < 2; ++g) {
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
#pragma unroll
          for (int x = 0; x < 2; ++x)
            reinterpret_cast<uint4*>(dst + c)[x] =
                make_uint4(y[4 * x], y[4 * x + 1], y[4 * x + 2], y[4 * x + 3]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            out[(c / 4 + x) * 128 + r] =
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

// Joins the chunks in order.  A thread has 8 channels of one row; a warp's
// lanes are 32 rows, whose float4 pieces lie side by side.  Grid: (sequence x
// head x row tile, HD / 16, halves of 128 rows); its schedule is made while
// the chunks are still being computed.  Bound by latency and the L2: 1024 rows of
// four chunks, 17 MB, take 7.5 us alone.
template <int HD>
__global__ void __launch_bounds__(256) cache_join_tile_kernel(const __grid_constant__ Args a) {
  __shared__ Unit shared_unit;
  const int lane = threadIdx.x & 31;
  const int per = a.c.n_kv_heads * a.row_tiles;
  Share share{};
  if (a.c.n_seqs > 1 && !a.fit) {
    __shared__ unsigned long long scratch[kShareScratch / 8];
    share = block_share(a, scratch);
    if (!share.any) {  // (the wait still: what follows may count on the chunks too)
      sm100::grid_dep_wait();
      sm100::grid_dep_launch();
      return;
    }
  }
#pragma unroll 1
  for (int blk = blockIdx.x; blk < a.c.n_seqs * per; blk += gridDim.x) {
    const int seq = blk / per, p = blk - seq * per;
    const int head = p % a.c.n_kv_heads, group_tile = p / a.c.n_kv_heads;
    if (threadIdx.x < 32) {
      Unit u{};
      if (a.c.n_seqs == 1) {
        only_unit(a, -1, u);
      } else if (!a.fit) {
        chunks_of(a, share, seq, lane, u);
      } else {
        const Lane mine = lane_steps(a, lane);
        find_unit(a, chunk_steps(a, lane, mine), -1, seq, lane, mine, u);
      }
      if (lane == 0) shared_unit = u;
    }
    __syncthreads();
    const int n_chunks = shared_unit.n_chunks, base = shared_unit.base, more = shared_unit.more;
    __syncthreads();
    sm100::grid_dep_wait();
    sm100::grid_dep_launch();
    const int r = threadIdx.x & 127, half = blockIdx.z;
    const int c4 = (blockIdx.y * 2 + (threadIdx.x >> 7)) * 2;  // of the row's float4 pieces
    const int R = group_tile * a.tile_rows + half * 128 + r, rows = a.n_tokens * a.group;
    if (n_chunks <= 1 || R >= rows) continue;  // written by its block, or refused
    const float2* ml = a.ml_part + static_cast<int64_t>(p) * a.tile_rows + half * 128 + r;
    const float4* src = reinterpret_cast<const float4*>(a.o_part) +
                        ((static_cast<int64_t>(p) * (a.tile_rows / 128) + half) * (HD / 4) + c4) * 128 + r;
    const int64_t ml_step = static_cast<int64_t>(per) * a.tile_rows;
    const int64_t o_step = static_cast<int64_t>(per) * (a.tile_rows / 128) * (HD / 4) * 128;
    constexpr int kBatch = 6;  // chunks whose loads are in flight together
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    float sum = 0.f, m = -INFINITY;
    for (int x0 = 0; x0 < n_chunks; x0 += kBatch) {
      float2 v[kBatch];
      float4 y[kBatch][2];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int k = x0 + x < n_chunks ? x0 + x : x0;
        const int64_t at = k == 0 ? base : more + k;
        v[x] = __ldcg(ml + at * ml_step);
        y[x][0] = __ldcg(src + at * o_step);
        y[x][1] = __ldcg(src + at * o_step + 128);
      }
      float m_new = m;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) m_new = fmaxf(m_new, v[x].x);
      const float mu = m_new == -INFINITY ? 0.f : m_new;
      const float old = exp2_fast(m - mu);
      m = m_new;
      sum *= old;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] *= old;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (x0 + x >= n_chunks) break;
        const float f = exp2_fast(v[x].x - mu);
        sum += v[x].y * f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[4 * i] += y[x][i].x * f;
          acc[4 * i + 1] += y[x][i].y * f;
          acc[4 * i + 2] += y[x][i].z * f;
          acc[4 * i + 3] += y[x][i].w * f;
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    const int t = token_of(a, R), i = R - t * a.group;
    uint16_t* dst = a.o + (static_cast<int64_t>(seq) * a.n_tokens + t) * a.o_stride +
                    (head * a.group + i) * HD + c4 * 4;
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                   pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
  }
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

cudaError_t launch_tile_attention(const Args& a, int format, int hd, int64_t grid, int num_sms,
                                  cudaStream_t st) {
  const dim3 g(static_cast<unsigned>(grid));
  cudaError_t ce = hd == 128 ? launch_tile_format<128>(a, format, g, st)
                             : launch_tile_format<64>(a, format, g, st);
  if (ce != cudaSuccess || a.slots == 0) return ce;
  const int slices = hd / 16 * (a.tile_rows / 128);
  const dim3 jg(std::min(a.c.n_seqs * a.c.n_kv_heads * a.row_tiles,
                         std::max(1, 8 * num_sms / slices)), hd / 16, a.tile_rows / 128);
  return hd == 128 ? launch_after(cache_join_tile_kernel<128>, jg, 256, 0, st, a)
                   : launch_after(cache_join_tile_kernel<64>, jg, 256, 0, st, a);
}

}  // namespace pds
