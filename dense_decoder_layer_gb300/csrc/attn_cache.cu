// Attention of a few new tokens per sequence over a cache of bf16, e4m3 or
// 4-bit rows (pds_attention_tree).
//
// Mathematics.  Query row r = t G + i of a (sequence, kv head) is head
// kv_head G + i of token t (G = H / Hkv).  With the cached row of key j read
// as scale_j code_j,
//   z_rj = log2(e)/sqrt(hd) kscale_j (q_r . kcode_j)       (softcap on top)
//   o_r  = sum_j 2^(z_rj - m_r) vscale_j vcode_j / sum_j 2^(z_rj - m_r)
// over the keys j that token t sees: the scales stay out of the matrix
// products, so the codes go into them as they are (fp16 holds every one) and
// nothing is rounded on the way but P = 2^(z-m) vscale, to fp16, or to bf16 for
// a bf16 cache, as in the prefill attention (a weight's error averages out over
// the keys), and o (once).
//
// What bounds it: every cached row is used by T G query rows, one to a few
// dozen, so at T G flop per byte of bf16 the call is bound by reading the
// cache (HBM); few-row calls by latency.  Hence the split: the keys of a
// sequence are cut into chunks over all SMs, each block holds the T G rows
// of one kv head (up to 32) and its 8 warps walk the chunk's 16-key steps
// independently, each through its own ring of asynchronous copies, so no
// barrier stands between a warp and the memory.  The warp computes
// S^T = K Q^T with keys as the 16-row operand and 8 query rows per column
// tile (a decode step has 3 or 4: a query-major tile would be 3/4 empty), and
// O^T = V^T P^T the same way, P^T being S^T's fragments transposed inside the
// warp.  A key's scales are then one factor per accumulator row, and a running
// reference that moves only when a score exceeds it by 8 (a weight of 2^8) needs no
// reduction over keys until the end.
//
// Chunks write unnormalised rows and (maximum, sum) to the workspace; a second
// kernel joins them in chunk order.  The chunk length is made from the
// sequences' lengths on the device (they change between replays of a graph).
//
// Measured (32/8 heads of 128; replayed graphs, so without the host's part), one
// token of 16 sequences of 4096 rows: bf16 44.5 us (6.0 TB/s), e4m3 29.4 (4.7),
// 4-bit 31.1 (2.3): bf16 is bound by HBM, the others by the conversion's
// instructions (the ALU pipe is the busiest, 38% and 56%) on the SMs that hold
// two of the 256 blocks.  24/8 heads, one token over 2048 bf16 rows: 5.8 us, of
// which some 4 are a launch, fetching the code and one round of loads.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <string>

#include "attn_cache.cuh"
#include "common.cuh"
#include "kv.h"
#include "sm100.cuh"
#include "tc.h"

namespace pds {
namespace {

using namespace cacheattn;

constexpr int kStep = 16;        // keys of a warp's step
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr float kMoveLog2 = 8.0f;  // the reference maximum follows beyond a growth of 2^8
constexpr int kMaxTiles = 4;     // column tiles of 8 query rows per block

// ------------------------------------------------------------ instructions

// Four 8x8 blocks of 16-bit values, transposed: lane l gives the address of
// row l % 8 of block l / 8.
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
// An 8x8 block of 16-bit values held by the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// ------------------------------------------------------------ the formats

// Bytes of a head's row, and of one step's K (or V) slice.
template <int FMT, int HD>
struct Fmt {
  static constexpr bool kBf16 = FMT == PDS_KV_BF16;
  static constexpr int kRow = kBf16 ? 2 * HD : FMT == PDS_KV_E4M3 ? HD : HD / 2;
  static constexpr int kSlice = kStep * kRow;
  static constexpr int kChunks = kRow / 16;  // 16-byte chunks of a row
  static constexpr int kStage = 2 * kSlice + 128;  // K, V, 16 + 16 scale words
  static constexpr int kKSteps = HD / 16;   // contraction steps of S^T
  static constexpr int kMTiles = HD / 16;   // channel tiles of O^T

  // Where chunk c of the step's key row r is kept.  The chunks are permuted
  // within 128-byte lines so that the lanes that load together (K: two rows,
  // all four quarters; V: keys 0, 2, 4, 6 of a lane group, neighbouring chunks)
  // hit different banks.
  static __device__ __forceinline__ uint32_t k_at(int r, int c) {
    if constexpr (kRow >= 128) return r * kRow + ((c ^ ((r & 1) << 2)) << 4);
    return r * kRow + (c << 4);
  }
  static __device__ __forceinline__ uint32_t v_at(int r, int c) {
    if constexpr (FMT == PDS_KV_BF16) return r * kRow + ((c ^ (r & 7)) << 4);
    if constexpr (kRow == 128) return r * 128 + ((c ^ (((r >> 1) & 3) << 1)) << 4);
    if constexpr (kRow == 64)
      return (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (((r >> 1) & 3) << 1)) << 4);
    return (r >> 2) * 128 + ((((r & 3) * 2 + c) ^ (((r >> 2) & 1) << 1)) << 4);
  }

  // A step's copy: piece x of a lane is row kRowsPerPiece x + lane / kChunks, chunk
  // lane % kChunks.  From one piece to the next its place moves by a constant,
  // but for the bits of V's permutation that depend on x alone.
  static constexpr int kRowsPerPiece = 32 / kChunks;
  static constexpr int kPieces = kStep / kRowsPerPiece;
  static constexpr uint32_t kPieceBytes = kRowsPerPiece * kRow;
  static constexpr uint32_t v_piece_xor(int x) {
    return FMT == PDS_KV_BF16 ? (HD == 128 ? (x & 3) << 5 : (x & 1) << 6)
                              : kRow == 128 ? (x & 1) << 6 : 0;
  }

  // The contraction runs over the head's channels in an order that lets a lane
  // read its share of a key's row with wide loads: in step ks the lane's quarter
  // t4 has the channels ch .. ch + 3 from this one on (4-bit rows: ch, ch + 4
  // and ch + 1, ch + 5), two in each operand register.
  static __device__ __forceinline__ int q_channel(int ks, int t4) {
    if constexpr (FMT == PDS_KV_BF16) return 8 * (t4 + 4 * (ks >> 1)) + 4 * (ks & 1);
    if constexpr (FMT == PDS_KV_E4M3) return 16 * (t4 + 4 * (ks >> 2)) + 4 * (ks & 3);
    return (HD / 4) * t4 + 8 * (ks >> 1) + 2 * (ks & 1);
  }
  // Channel of row half hh (0: rows 0-7, 1: rows 8-15), lane group g, of
  // channel tile i of O^T.
  static __device__ __forceinline__ int o_channel(int i, int hh, int g) {
    return FMT == PDS_KV_BF16 ? 16 * i + 8 * hh + g : (HD / 8) * g + 2 * i + hh;
  }
};

// S^T (16 keys x 8 NT rows) of one step.
template <int FMT, int HD, int NT>
__device__ __forceinline__ void scores(uint32_t ks, uint32_t q_frag, int lane, uint32_t kz0,
                                       uint32_t kz1, float (&s)[NT][4]) {
  using F = Fmt<FMT, HD>;
  const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[n][i] = 0.f;
  auto step = [&](int k, const uint32_t (&a)[4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint2 b = lds64(q_frag + ((k * NT + n) * 32 + lane) * 8);
      mma<F::kBf16>(s[n], a, b.x, b.y);
    }
  };
  if constexpr (FMT == PDS_KV_BF16) {
#pragma unroll
    for (int c = 0; c < HD / 32; ++c) {
      const uint4 x = lds128(ks + F::k_at(g, t4 + 4 * c));
      const uint4 y = lds128(ks + F::k_at(g + 8, t4 + 4 * c));
      const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
      step(2 * c, a0);
      step(2 * c + 1, a1);
    }
  } else if constexpr (FMT == PDS_KV_E4M3) {
#pragma unroll
    for (int c = 0; c < HD / 64; ++c) {
      const uint4 xv = lds128(ks + F::k_at(g, t4 + 4 * c));
      const uint4 yv = lds128(ks + F::k_at(g + 8, t4 + 4 * c));
      const uint32_t x[4] = {xv.x, xv.y, xv.z, xv.w}, y[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a[4];
        e4m3_pairs(x[w], a[0], a[2]);
        e4m3_pairs(y[w], a[1], a[3]);
        step(4 * c + w, a);
      }
    }
  } else {
    constexpr int kWords = HD / 32;
    uint32_t x[4], y[4];
    if constexpr (HD == 128) {
      const uint4 xv = lds128(ks + F::k_at(g, t4)), yv = lds128(ks + F::k_at(g + 8, t4));
      x[0] = xv.x, x[1] = xv.y, x[2] = xv.z, x[3] = xv.w;
      y[0] = yv.x, y[1] = yv.y, y[2] = yv.z, y[3] = yv.w;
    } else {
      const uint2 xv = lds64(ks + F::k_at(g, t4 >> 1) + 8 * (t4 & 1));
      const uint2 yv = lds64(ks + F::k_at(g + 8, t4 >> 1) + 8 * (t4 & 1));
      x[0] = xv.x, x[1] = xv.y;
      y[0] = yv.x, y[1] = yv.y;
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const uint32_t a0[4] = {int4_lo(x[w], kz0), int4_lo(y[w], kz1), int4_hi(x[w], kz0),
                              int4_hi(y[w], kz1)};
      x[w] >>= 8, y[w] >>= 8;
      const uint32_t a1[4] = {int4_lo(x[w], kz0), int4_lo(y[w], kz1), int4_hi(x[w], kz0),
                              int4_hi(y[w], kz1)};
      step(2 * w, a0);
      step(2 * w + 1, a1);
    }
  }
}

// O^T += V^T P^T of one step; p: the B fragments of P^T (two registers per
// column tile); vz0, vz1: zero points of keys (2t, 2t+1) and (2t+8, 2t+9);
// clean: hidden rows may hold any code.
template <int FMT, int HD, int NT>
__device__ __forceinline__ void accumulate(uint32_t vs, int lane, uint32_t vz0, uint32_t vz1,
                                           bool clean,
                                           const uint32_t (&p)[NT][2],
                                           float (&o)[Fmt<FMT, HD>::kMTiles][NT][4]) {
  using F = Fmt<FMT, HD>;
  const int g = lane >> 2, t4 = lane & 3;
  if constexpr (FMT == PDS_KV_BF16) {
    const int key = (lane & 7) + ((lane >> 4) << 3), odd = (lane >> 3) & 1;
#pragma unroll
    for (int i = 0; i < F::kMTiles; ++i) {
      uint32_t a[4];
      ldsm4_t(vs + F::v_at(key, 2 * i + odd), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma<true>(o[i][n], a, p[n][0], p[n][1]);
    }
  } else {
    // this lane's channels of keys 2t, 2t+1, 2t+8, 2t+9
    constexpr int kBytes = F::kRow / 8;          // of one key
    constexpr int kW = kBytes <= 4 ? 1 : kBytes / 4;
    uint32_t w[4][kW];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = 2 * t4 + (i & 1) + 8 * (i >> 1);
      if constexpr (kBytes == 16) {
        const uint4 x = lds128(vs + F::v_at(key, g));
        w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
      } else if constexpr (kBytes == 8) {
        const uint2 x = lds64(vs + F::v_at(key, g >> 1) + 8 * (g & 1));
        w[i][0] = x.x, w[i][1] = x.y;
      } else {
        w[i][0] = lds32(vs + F::v_at(key, g >> 2) + 4 * (g & 3));
      }
    }
    if constexpr (FMT == PDS_KV_E4M3) {
      if (clean) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < kW; ++x) w[i][x] = e4m3_finite(w[i][x]);
      }
#pragma unroll
      for (int x = 0; x < kW; ++x)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // channel tile 2 x + half: bytes 2 half and + 1 of word x, paired over keys
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          uint32_t a[4];
          e4m3_pairs(__byte_perm(w[0][x], w[1][x], sel), a[0], a[1]);
          e4m3_pairs(__byte_perm(w[2][x], w[3][x], sel), a[2], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<false>(o[2 * x + half][n], a, p[n][0], p[n][1]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < F::kMTiles; ++i) {
        // channel tile i: the two nibbles of byte i % 4 of word i / 4
        const int x = i >> 2, b = i & 3;
        const uint32_t sel = b | (static_cast<uint32_t>(4 + b) << 8);  // into bytes 0 and 2
        const uint32_t r0 = __byte_perm(w[0][x], w[1][x], sel);
        const uint32_t r1 = __byte_perm(w[2][x], w[3][x], sel);
        const uint32_t a[4] = {int4_lo(r0, vz0), int4_hi(r0, vz0), int4_lo(r1, vz1),
                               int4_hi(r1, vz1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma<false>(o[i][n], a, p[n][0], p[n][1]);
      }
    }
  }
}

template <int FMT, int HD, int NT>
struct Cfg {
  using F = Fmt<FMT, HD>;
  static constexpr int kRows = 8 * NT;
  // one block per SM where its registers (32 rows) or its stages (16 KB per
  // warp in flight) fill it, else two
  static constexpr int kBlocks = NT == 4 || F::kStage > 8192 ? 1 : 2;
  static constexpr int kFit = (kBlocks == 1 ? 200 : 100) * 1024 / (kWarps * F::kStage);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static_assert(kStages >= 2, "a step is read while another is fetched");
  static constexpr int kQ = 0;  // B fragments of Q
  static constexpr int kQBytes = F::kKSteps * NT * 32 * 8;
  static constexpr int kMask = kQ + kQBytes;                  // ancestors of the tile's tokens
  static constexpr int kDepth = kMask + kRows * kMaskWords * 4;
  static constexpr int kParent = kDepth + kMaxDraftTokens * 2;
  static constexpr int kMl = kParent + kMaxDraftTokens * 4;   // per warp and row: (maximum, sum)
  static constexpr int kInv = kMl + kWarps * kRows * 8;       // per warp: O's unit
  static constexpr int kQMax = kInv + kWarps * 4;             // per warp: Q's maximum in 8 rows
  static constexpr int kQInv = kQMax + kWarps * 8 * 4;        // per row: the inverse of Q's multiplier
  static constexpr int kMisc = (kQInv + kRows * 4 + 15) / 16 * 16;
  static constexpr int kRing = (kMisc + 64 + 127) / 128 * 128;
  static constexpr int kRingBytes = kWarps * kStages * F::kStage;
  // the warps' O rows are joined in the space of the ring
  static constexpr int kJoinStride = HD + 4;
  static constexpr int kJoin = kWarps * kRows * kJoinStride * 4;
  // behind them, the block's rows for the other blocks of its cluster: O, (maximum, sum)
  static constexpr int kShare = kRing + kJoin;
  static constexpr int kShareMl = kShare + kRows * HD * 4;
  static constexpr int kJoinEnd = kShareMl + kRows * 8;
  static constexpr int kSmem = kRing + kRingBytes > kJoinEnd ? kRing + kRingBytes : kJoinEnd;
  static_assert(kSmem * kBlocks <= 228 * 1024 - 1024 * kBlocks, "shared memory per SM");
};

// VAR: the call has a softcap or a window.
template <int FMT, int HD, int NT, bool VAR>
__global__ void __launch_bounds__(kThreads, Cfg<FMT, HD, NT>::kBlocks)
    cache_attn_kernel(const __grid_constant__ Args a) {
  using F = Fmt<FMT, HD>;
  using C = Cfg<FMT, HD, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + C::kMask);
  int16_t* depth = reinterpret_cast<int16_t*>(smem + C::kDepth);
  int32_t* par = reinterpret_cast<int32_t*>(smem + C::kParent);
  float2* ml = reinterpret_cast<float2*>(smem + C::kMl);
  Unit* shared_unit = reinterpret_cast<Unit*>(smem + C::kMisc);
  int* shared_ok = reinterpret_cast<int*>(smem + C::kMisc + 48);

  const int per = a.c.n_kv_heads * a.row_tiles;
  const int chunk_unit = a.cluster > 1 ? blockIdx.x / a.cluster : blockIdx.x;
  const int w = chunk_unit / per, p = chunk_unit - w * per;
  const int head = p % a.c.n_kv_heads, tile = p / a.c.n_kv_heads;
  sm100::grid_dep_wait();  // everything below reads what earlier kernels wrote
  sm100::grid_dep_launch();
  Unit u{};
  if (a.cluster > 1) {  // sequence w, in as many chunks as the cluster has blocks
    int first;
    const int n = seq_steps(a, w, first, u.len);
    if (n == 0) {  // (all of the cluster's blocks leave)
      if (p == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadLength);
      return;
    }
    const int c = (n + a.cluster - 1) / a.cluster, rank = blockIdx.x - chunk_unit * a.cluster;
    u.seq = w;
    u.n_chunks = a.cluster;
    u.first = first + rank * c;
    u.n_steps = max(0, min(c, n - rank * c));
  } else if (a.slots == 0) {
    if (!whole_unit(a, w, u)) {
      if (p == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadLength);
      return;
    }
  } else if (a.c.n_seqs == 1) {
    const bool ok = only_unit(a, w, u);
    if (blockIdx.x == 0 && threadIdx.x == 0 && u.n_chunks == 0)
      atomicOr(a.status, kStatusBadLength);
    if (!ok) return;
  } else if (!a.fit) {
    const Share h = block_share(a, smem + C::kRing);  // (the ring is not in use yet)
    const bool ok = w < a.c.n_seqs ? first_unit(a, h, w, u)
                                   : later_unit(a, h, w - a.c.n_seqs, lane, u);
    if (!ok) {
      if (w < a.c.n_seqs && p == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadLength);
      return;
    }
    __syncthreads();  // the ring may be filled
  } else {
    if (warp == 0) {
      const Lane mine = lane_steps(a, lane);
      const int c = chunk_steps(a, lane, mine);
      const bool ok = find_unit(a, c, w, 0, lane, mine, u);
      if (lane == 0) {
        *shared_unit = u;
        *shared_ok = ok;
      }
      if (blockIdx.x == 0) {  // report lengths that do not fit
        bool bad = false;
#pragma unroll 1
        for (int s = lane; s < a.c.n_seqs; s += 32) bad |= lane_steps(a, s).n == 0;
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, kStatusBadLength);
      }
    }
    __syncthreads();
    if (!*shared_ok) return;
    u = *shared_unit;
  }
  const int r0 = tile * C::kRows;                        // first query row
  const int rows = a.n_tokens * a.group;
  const int end = u.len + a.n_tokens;                    // keys [.., end)

  // this warp's steps: u.first + warp, + kWarps, ...
  const uint32_t ring = smem_addr(smem) + C::kRing + warp * C::kStages * F::kStage;
  const int64_t word0 = (static_cast<int64_t>(u.seq) * a.c.n_kv_heads + head) * a.c.capacity;
  const int n_mine = u.n_steps > warp ? (u.n_steps - warp - 1) / kWarps + 1 : 0;
  // where this lane's pieces of the next step to fetch come from and go to
  int row = (u.first + warp) * kStep + lane / F::kChunks;
  const char* seq_k = a.c.k + u.seq * a.c.seq_stride + head * a.c.head_stride;
  const char* seq_v = a.c.v + u.seq * a.c.seq_stride + head * a.c.head_stride;
  int64_t off = row * a.c.row_stride + (lane % F::kChunks) * 16;
  const int64_t piece_off = F::kRowsPerPiece * a.c.row_stride;
  const uint32_t k_to = F::k_at(lane / F::kChunks, lane % F::kChunks);
  const uint32_t v_to = F::kSlice + F::v_at(lane / F::kChunks, lane % F::kChunks);
  int word_row = (u.first + warp) * kStep + (lane & 15);  // of this lane's scale word
  const uint32_t* words = (lane < 16 ? a.c.k_scale : a.c.v_scale) + word0;
  int fetched = 0;
  uint32_t fetch_to = ring;
  auto fetch = [&]() {  // the next step of this warp, into the next stage
    if (fetched < n_mine) {
      int64_t o = off;
#pragma unroll
      for (int x = 0; x < F::kPieces; ++x) {
        // a row past the end is not read: it is given the sequence's first address
        const bool live = row + x * F::kRowsPerPiece < end;
        const int64_t from = live ? o : 0;
        copy16(fetch_to + x * F::kPieceBytes + k_to, seq_k + from, live);
        copy16(fetch_to + x * F::kPieceBytes + (v_to ^ F::v_piece_xor(x)), seq_v + from, live);
        o += piece_off;
      }
      if constexpr (!F::kBf16) {
        const bool live = word_row < end;
        copy4(fetch_to + 2 * F::kSlice + lane * 4, words + (live ? word_row : 0), live);
        word_row += kWarps * kStep;
      }
      row += kWarps * kStep;
      off += kWarps * kStep * a.c.row_stride;
      ++fetched;
      fetch_to += F::kStage;
      if (fetch_to == ring + C::kStages * F::kStage) fetch_to = ring;
    }
    copies_commit();
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages - 1; ++i) fetch();

  // Q as B fragments, in the contraction's channel order; rows past the last are zero
  constexpr int kQFrags = F::kKSteps * NT * 32;
  constexpr int kQIters = (kQFrags + kThreads - 1) / kThreads;
  uint32_t* q_max = reinterpret_cast<uint32_t*>(smem + C::kQMax);
  static_assert(kWarps % NT == 0, "a thread's fragments are all of one row: 8 (warp % NT) + g");
  uint32_t qb[kQIters][2], q_top = 0u;
#pragma unroll
  for (int it = 0; it < kQIters; ++it) {
    const int idx = it * kThreads + threadIdx.x;
    const int l = idx & 31, n = (idx >> 5) % NT, ks = idx / (32 * NT);
    const int r = r0 + 8 * n + (l >> 2);
    qb[it][0] = qb[it][1] = 0u;
    if (idx < kQFrags && r < rows) {
      const int t = token_of(a, r), i = r - t * a.group;
      const uint16_t* src = a.q + (static_cast<int64_t>(u.seq) * a.n_tokens + t) * a.q_stride +
                            (head * a.group + i) * HD;
      const int ch = F::q_channel(ks, l & 3);
      if constexpr (FMT == PDS_KV_INT4) {  // channels (ch, ch + 4), (ch + 1, ch + 5)
        const uint32_t x = *reinterpret_cast<const uint32_t*>(src + ch);
        const uint32_t y = *reinterpret_cast<const uint32_t*>(src + ch + 4);
        qb[it][0] = __byte_perm(x, y, 0x5410);
        qb[it][1] = __byte_perm(x, y, 0x7632);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(src + ch);
        qb[it][0] = x.x;
        qb[it][1] = x.y;
      }
    }
    if constexpr (!F::kBf16) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        q_top = max(q_top, max(finite_bits(__uint_as_float(qb[it][e] << 16)),
                               finite_bits(__uint_as_float(qb[it][e] & 0xffff0000u))));
    }
  }
  if constexpr (!F::kBf16) {
    q_top = max(q_top, __shfl_xor_sync(0xffffffffu, q_top, 1));
    q_top = max(q_top, __shfl_xor_sync(0xffffffffu, q_top, 2));
    if (t4 == 0) q_max[warp * 8 + g] = q_top;
  }
  // a tree's depths, and the ancestor sets of this tile's tokens
  const int t_first = token_of(a, r0);
  if (a.parents && threadIdx.x < a.n_tokens)
    par[threadIdx.x] = a.parents[static_cast<int64_t>(u.seq) * a.n_tokens + threadIdx.x];
  __syncthreads();
  float* q_inv = reinterpret_cast<float*>(smem + C::kQInv);
  float q_mul = 1.f;
  if constexpr (!F::kBf16) {
#pragma unroll
    for (int x = warp % NT; x < kWarps; x += NT) q_top = max(q_top, q_max[x * 8 + g]);
    const uint32_t e = q_exponent(q_top);
    q_mul = q_multiplier(e);
    if (warp < NT && t4 == 0) q_inv[8 * warp + g] = q_inverse(e) * a.scale_log2;
  }
#pragma unroll
  for (int it = 0; it < kQIters; ++it) {
    const int idx = it * kThreads + threadIdx.x;
    if constexpr (!F::kBf16) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        qb[it][e] = pack_f16x2(__uint_as_float(qb[it][e] << 16) * q_mul,
                               __uint_as_float(qb[it][e] & 0xffff0000u) * q_mul);
    }
    if (idx < kQFrags)
      *reinterpret_cast<uint2*>(smem + C::kQ + idx * 8) = make_uint2(qb[it][0], qb[it][1]);
  }
  if (a.parents && threadIdx.x < a.n_tokens) {
    const int t = threadIdx.x, d = tree_depth(par, t), tl = t - t_first;
    depth[t] = static_cast<int16_t>(d);
    if (d == kBadParent) atomicOr(a.status, kStatusBadParent);
    if (tl >= 0 && tl < C::kRows) {
      uint32_t bits[kMaskWords];
#pragma unroll
      for (int i = 0; i < kMaskWords; ++i) bits[i] = 0u;
      int x = t;
      for (int e = 0; e <= d; ++e, x = par[x])
#pragma unroll
        for (int i = 0; i < kMaskWords; ++i)
          if ((x >> 5) == i) bits[i] |= 1u << (x & 31);
#pragma unroll
      for (int i = 0; i < kMaskWords; ++i) mask[tl * kMaskWords + i] = bits[i];
    }
  }
  __syncthreads();
  auto depth_of = [&](int t) -> int { return a.parents ? depth[t] : t; };

  // this lane's rows: 8 n + 2 t4 + {0, 1}; their tokens (within the tile) and positions
  int tok[NT][2], pos[NT][2];
  // What scores are multiplied by besides K's scales, to be in powers of two.  Kept in
  // registers where there are any left, else read anew for each step.
  constexpr bool kKeep = F::kBf16 || NT == 1 || (NT == 4 && HD == 64);
  float2 row_scale[kKeep ? NT : 1];
  int pos_hi = 0;  // windows of all rows of the tile start at or below pos_hi - window + 1
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + 8 * n + 2 * t4 + e;
      const int t = r < rows ? token_of(a, r) : -1;
      const int d = t < 0 ? -1 : depth_of(t);
      tok[n][e] = d < 0 ? -1 : t - t_first;
      pos[n][e] = u.len + d;
      pos_hi = max(pos_hi, pos[n][e]);
    }
  if (VAR) pos_hi = __reduce_max_sync(0xffffffffu, pos_hi);
  const uint32_t row_scales = smem_addr(smem) + C::kQInv + 8 * t4;
  if constexpr (!F::kBf16 && kKeep) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint2 w = lds64(row_scales + 32 * n);
      row_scale[n] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    }
  }

  float o[F::kMTiles][NT][4];
#pragma unroll
  for (int i = 0; i < F::kMTiles; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
  float m_ref[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) m_ref[n][e] = -INFINITY, l[n][e] = 0.f;

  const SoftCap cap = soft_cap(VAR ? a.cap * a.scale_log2 : 0.f);  // (in powers of two)
  uint32_t v_exp = kMinScaleExp;  // exponent of the largest V scale so far: O's unit
  const uint32_t q_frag = smem_addr(smem) + C::kQ;
  uint32_t st = ring;  // the step's stage
  int j0 = (u.first + warp) * kStep;
  for (int i = 0; i < n_mine; ++i, j0 += kWarps * kStep) {
    if (i > 0) st = st + F::kStage == ring + C::kStages * F::kStage ? ring : st + F::kStage;
    copies_wait<C::kStages - 2>();
    __syncwarp();
    fetch();  // into the stage that the step before has been read from

    // scale words of this lane's keys: g, g + 8 (rows of S^T), and the zero
    // points that the operands need
    float kscale[2] = {1.f, 1.f}, vscale[2] = {1.f, 1.f};
    uint32_t kz[2] = {0u, 0u}, vz[2] = {0u, 0u};
    if constexpr (FMT != PDS_KV_BF16) {
      const uint32_t sw = st + 2 * F::kSlice;
      uint32_t kw[2], vw[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        kw[e] = lds32(sw + (g + 8 * e) * 4);
        vw[e] = lds32(sw + 64 + (g + 8 * e) * 4);
        if constexpr (FMT == PDS_KV_INT4) {
          kz[e] = int4_zero(kw[e], kw[e]);
          kw[e] &= 0xffff0000u;
          vw[e] &= 0xffff0000u;
          const uint2 z = lds64(sw + 64 + (2 * t4 + 8 * e) * 4);
          vz[e] = int4_zero(z.x, z.y);
        }
        kscale[e] = __uint_as_float(kw[e]);
        vscale[e] = __uint_as_float(vw[e]);
      }
    }

    float s[NT][4];
    scores<FMT, HD, NT>(st, q_frag, lane, kz[0], kz[1], s);

    // scaled scores in powers of two
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float2 rs = make_float2(a.scale_log2, a.scale_log2);
      if constexpr (!F::kBf16 && kKeep) rs = row_scale[n];
      if constexpr (!kKeep) {
        const uint2 w = lds64(row_scales + 32 * n);
        rs = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = e & 1 ? rs.y : rs.x;
        s[n][e] *= F::kBf16 ? f : kscale[e >> 1] * f;
      }
    }
    if (VAR && cap.c > 0.f) {
      if (cap.wide()) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = capped_wide(s[n][e], cap);
      } else {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = capped(s[n][e], cap);
      }
    }
    // a step that holds new tokens, the end, or a window's lower edge
    bool masked = j0 + kStep > u.len;
    if (VAR && a.window > 0) masked |= j0 <= pos_hi - a.window;
    bool seen[2] = {true, true};  // whether one of this lane's rows sees its key
    if (masked) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + g + 8 * e, rel = j - u.len;
        const int key_pos = rel < 0 || rel >= a.n_tokens ? j : u.len + depth_of(rel);
        seen[e] = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int t = tok[n][x];
            bool see = t >= 0;
            if (see && rel >= 0)
              see = a.parents ? rel < a.n_tokens &&
                                    ((mask[t * kMaskWords + (rel >> 5)] >> (rel & 31)) & 1u)
                              : rel <= t + t_first;
            if (VAR && a.window > 0) see = see && key_pos > pos[n][x] - a.window;
            if (!see) s[n][2 * e + x] = -INFINITY;
            seen[e] |= see;
          }
      }
    }
    // move the references where a score is far above (by their difference: from 2^26 on
    // a reference and 8 more need not be a float32)
    bool far = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) far |= s[n][e] - m_ref[n][e & 1] > kMoveLog2;
    if constexpr (!F::kBf16) {
#pragma unroll
      for (int e = 0; e < 2; ++e) far |= seen[e] && finite_bits(vscale[e]) >> 23 > v_exp;
    }
    if (__any_sync(0xffffffffu, far)) {
      float shift[2] = {0.f, 0.f};
      if constexpr (!F::kBf16) {
        uint32_t v_top = v_exp;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (seen[e]) v_top = max(v_top, min(finite_bits(vscale[e]) >> 23, kMaxScaleExp));
        v_top = __reduce_max_sync(0xffffffffu, v_top);
        if (__builtin_expect(v_top > v_exp && i > 0, 0)) {
          float most = 0.f;  // (sums are not negative: they order as their bits do)
#pragma unroll
          for (int n = 0; n < NT; ++n) most = fmaxf(most, fmaxf(l[n][0], l[n][1]));
          most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          const int d = static_cast<int>(v_top - v_exp), k = unit_shift(d, most);
          const float up = exp2_fast(static_cast<float>(k)), down = exp2_fast(static_cast<float>(k - d));
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              m_ref[n][x] -= static_cast<float>(k);
              l[n][x] *= up;
            }
          if (k < d) {
#pragma unroll
            for (int t = 0; t < F::kMTiles; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][n][e] *= down;
          }
        }
        v_exp = v_top;
#pragma unroll
        for (int e = 0; e < 2; ++e) shift[e] = level_shift(finite_bits(vscale[e]) >> 23, v_exp);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float m = fmaxf(s[n][x] + shift[0], s[n][2 + x] + shift[1]);
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, sh));
          if (m - m_ref[n][x] > kMoveLog2) {
            const float alpha = exp2_fast(m_ref[n][x] - m);  // 0 from -inf
            m_ref[n][x] = m;
            l[n][x] *= alpha;
#pragma unroll
            for (int t = 0; t < F::kMTiles; ++t) {
              o[t][n][x] *= alpha;
              o[t][n][2 + x] *= alpha;
            }
          }
        }
    }
    // P, its row sums (float32, unrounded) and its transposed fragments
    if constexpr (!F::kBf16) {
#pragma unroll
      for (int e = 0; e < 2; ++e) vscale[e] *= v_multiplier(v_exp);
    }
    uint32_t pf[NT][2];
    float pv[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = m_ref[n][e & 1];
        const float pe = exp2_fast(s[n][e] - (m == -INFINITY ? 0.f : m));
        l[n][e & 1] += pe;
        pv[n][e] = pe;
        if constexpr (FMT != PDS_KV_BF16)  // a hidden row may have any scale, a NaN too
          pv[n][e] = masked && pe == 0.f ? 0.f : pe * vscale[e >> 1];
      }
      auto pack = [](float lo, float hi) {
        return F::kBf16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
      };
      pf[n][0] = transpose8(pack(pv[n][0], pv[n][1]));
      pf[n][1] = transpose8(pack(pv[n][2], pv[n][3]));
    }
    if constexpr (FMT == PDS_KV_BF16) {
      // A hidden row of a masked step may hold an infinity or a NaN, which a
      // zero weight would not keep out of the product: such a step is summed
      // element by element, over what each row sees.
      if (masked) {
        bool bad = false;
#pragma unroll
        for (int x = 0; x < F::kSlice / 512; ++x) {
          const uint4 v = lds128(st + F::kSlice + (x * 32 + lane) * 16);
          bad |= not_finite2(v.x) || not_finite2(v.y) || not_finite2(v.z) || not_finite2(v.w);
        }
        if (__any_sync(0xffffffffu, bad)) {
          for (int key = 0; key < kStep; ++key) {
            const int src = (key & 7) * 4 + t4;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const float lo0 = __shfl_sync(0xffffffffu, pv[n][0], src);
              const float lo1 = __shfl_sync(0xffffffffu, pv[n][1], src);
              const float hi0 = __shfl_sync(0xffffffffu, pv[n][2], src);
              const float hi1 = __shfl_sync(0xffffffffu, pv[n][3], src);
              const float p0 = key < 8 ? lo0 : hi0, p1 = key < 8 ? lo1 : hi1;
#pragma unroll
              for (int t = 0; t < F::kMTiles; ++t)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const int ch = F::o_channel(t, hh, g);
                  uint16_t b;
                  asm volatile("ld.shared.u16 %0, [%1];"
                               : "=h"(b)
                               : "r"(st + F::kSlice + F::v_at(key, ch >> 3) + (ch & 7) * 2));
                  const float v = bf16_to_f32(b);
                  if (p0 != 0.f) o[t][n][2 * hh] += p0 * v;
                  if (p1 != 0.f) o[t][n][2 * hh + 1] += p1 * v;
                }
            }
          }
          continue;
        }
      }
    }
    accumulate<FMT, HD, NT>(st + F::kSlice, lane, vz[0], vz[1], masked, pf, o);
  }
  copies_wait<0>();

  // Join the warps: sums over the lanes that share rows, then over the warps,
  // in warp order.
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], sh);
      if (g == 0) ml[warp * C::kRows + 8 * n + 2 * t4 + x] = make_float2(m_ref[n][x], l[n][x]);
    }
  float* unit = reinterpret_cast<float*>(smem + C::kInv);  // of the warps' O
  if (lane == 0) unit[warp] = F::kBf16 ? 1.f : v_inverse(v_exp);
  __syncthreads();  // every warp is done with the ring
  float* join = reinterpret_cast<float*>(smem + C::kRing);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float* dst = join + (warp * C::kRows + 8 * n + 2 * t4 + x) * C::kJoinStride;
#pragma unroll
      for (int t = 0; t < F::kMTiles; ++t) {
        if constexpr (FMT == PDS_KV_BF16) {
          dst[F::o_channel(t, 0, g)] = o[t][n][x];
          dst[F::o_channel(t, 1, g)] = o[t][n][2 + x];
        } else {
          *reinterpret_cast<float2*>(dst + F::o_channel(t, 0, g)) =
              make_float2(o[t][n][x], o[t][n][2 + x]);
        }
      }
    }
  __syncthreads();
  const bool whole = u.n_chunks == 1;
  for (int idx = threadIdx.x; idx < C::kRows * (HD / 4); idx += kThreads) {
    const int r = idx / (HD / 4), ch = (idx - r * (HD / 4)) * 4;
    if (r0 + r >= rows) break;
    const int t = token_of(a, r0 + r), i = r0 + r - t * a.group;
    float m = -INFINITY;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) m = fmaxf(m, ml[x * C::kRows + r].x);
    const float mu = m == -INFINITY ? 0.f : m;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float2 v = ml[x * C::kRows + r];
      const float f = exp2_fast(v.x - mu);  // 0 for a warp that saw none of the row's keys
      const float4 y = *reinterpret_cast<const float4*>(join + (x * C::kRows + r) * C::kJoinStride + ch);
      const float fo = f * unit[x];
      sum += v.y * f;
      acc.x += y.x * fo;
      acc.y += y.y * fo;
      acc.z += y.z * fo;
      acc.w += y.w * fo;
    }
    if (depth_of(t) < 0) {  // a padding token's rows went along with the others
      m = -INFINITY;
      sum = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (a.cluster > 1) {
      *reinterpret_cast<float4*>(smem + C::kShare + (r * HD + ch) * 4) = acc;
      if (ch == 0) *reinterpret_cast<float2*>(smem + C::kShareMl + r * 8) = make_float2(m, sum);
    } else if (whole) {
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // a row that sees nothing is zero
      uint16_t* dst = a.o + (static_cast<int64_t>(u.seq) * a.n_tokens + t) * a.o_stride +
                      (head * a.group + i) * HD + ch;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    } else {
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * C::kRows + r;
      *reinterpret_cast<float4*>(a.o_part + slot * HD + ch) = acc;
      if (ch == 0) a.ml_part[slot] = make_float2(m, sum);
    }
  }
  if (a.cluster <= 1) return;
  // The chunks of the cluster's blocks, in order: every block takes a share of
  // the rows' pieces and reads the others' over distributed shared memory.
  sm100::cluster_sync();
  const uint32_t share = smem_addr(smem) + C::kShare, share_ml = smem_addr(smem) + C::kShareMl;
  const int live_rows = min(rows - r0, C::kRows);
  for (int idx = (blockIdx.x - chunk_unit * a.cluster) * kThreads + threadIdx.x;
       idx < live_rows * (HD / 4); idx += a.cluster * kThreads) {
    const int r = idx / (HD / 4), ch = (idx - r * (HD / 4)) * 4;
    float m = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < a.cluster; ++x) {
      const float2 v = sm100::ld_cluster_f2(sm100::mapa_shared(share_ml + r * 8, x));
      const float4 y = sm100::ld_cluster_f4(sm100::mapa_shared(share + (r * HD + ch) * 4, x));
      const float m_new = fmaxf(m, v.x), mu = m_new == -INFINITY ? 0.f : m_new;
      const float old = exp2_fast(m - mu), f = exp2_fast(v.x - mu);
      m = m_new;
      sum = sum * old + v.y * f;
      acc.x = acc.x * old + y.x * f;
      acc.y = acc.y * old + y.y * f;
      acc.z = acc.z * old + y.z * f;
      acc.w = acc.w * old + y.w * f;
    }
    const int t = token_of(a, r0 + r), i = r0 + r - t * a.group;
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint16_t* dst = a.o + (static_cast<int64_t>(u.seq) * a.n_tokens + t) * a.o_stride +
                    (head * a.group + i) * HD + ch;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  }
  sm100::cluster_sync();  // nobody leaves while its rows may still be read
}

// Four warps per (sequence, token, head) row: warp i joins chunks i, i + 4, ...,
// and the first joins the four, in order.  The schedule is made while the
// chunks are still being computed (lens were complete before those began), the
// loads come after.  Bound by latency (lengths, schedule, one or two rounds of
// loads): 5 us alone for 24 rows of 19 chunks, of which 2 to 3 remain behind the chunks.
template <int HD>
__global__ void __launch_bounds__(256) cache_join_kernel(const __grid_constant__ Args a) {
  constexpr int kShare = 4;        // warps of a row
  constexpr int kPer = HD / 32;
  constexpr int kBatch = 8;        // chunks whose loads are in flight together
  __shared__ float part_o[8][HD];
  __shared__ float2 part_ml[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = a.n_tokens * a.n_heads;
  const int per = a.c.n_kv_heads * a.row_tiles;
  const int64_t stride = static_cast<int64_t>(per) * a.tile_rows;
  Share share{};
  const bool many = a.c.n_seqs > 1 && !a.fit;
  if (many) {
    __shared__ unsigned long long scratch[kShareScratch / 8];
    share = block_share(a, scratch);
    if (!share.any) {  // (the wait still: what follows may count on the chunks too)
      sm100::grid_dep_wait();
      sm100::grid_dep_launch();
      return;
    }
  }
  const int pairs = static_cast<int>((static_cast<int64_t>(a.c.n_seqs) * per_seq + 1) / 2);
#pragma unroll 1
  for (int blk = blockIdx.x; blk < pairs; blk += gridDim.x) {
    const int row = blk * (8 / kShare) + warp / kShare;
    const int seq = row / per_seq, rest = row - seq * per_seq;
    const int t = rest / a.n_heads, h = rest - t * a.n_heads;
    const int head = h / a.group, r = t * a.group + h - head * a.group;
    const int tile = r / a.tile_rows;
    Unit u{};
    if (a.c.n_seqs == 1) {
      only_unit(a, -1, u);
    } else if (many) {
      if (seq < a.c.n_seqs) chunks_of(a, share, seq, lane, u);
    } else if (seq < a.c.n_seqs) {
      const Lane mine = lane_steps(a, lane);
      find_unit(a, chunk_steps(a, lane, mine), -1, seq, lane, mine, u);
    }
    // written by its block, or refused, or no such row
    const bool live = seq < a.c.n_seqs && u.n_chunks > 1;
    const int n_chunks = live ? u.n_chunks : 0;
    // of chunk x: the first apart from the others where there are many sequences
    const int64_t slot0 = (static_cast<int64_t>(tile) * a.c.n_kv_heads + head) * a.tile_rows +
                          (r - tile * a.tile_rows);
    sm100::grid_dep_wait();
    sm100::grid_dep_launch();
    float acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    float sum = 0.f, m = -INFINITY;
#pragma unroll 1
    for (int x0 = warp % kShare; x0 < n_chunks; x0 += kBatch * kShare) {
      float2 v[kBatch];
      float y[kBatch][kPer];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int at = x0 + x * kShare;
        const bool have = at < n_chunks;
        const int64_t slot = slot0 + (at == 0 ? u.base : u.more + at) * stride;
        const float* src = a.o_part + slot * HD + lane * kPer;
        v[x] = have ? __ldcg(a.ml_part + slot) : make_float2(-INFINITY, 0.f);
        if constexpr (kPer == 4) {
          const float4 f = have ? __ldcg(reinterpret_cast<const float4*>(src))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
          y[x][0] = f.x, y[x][1] = f.y, y[x][2] = f.z, y[x][3] = f.w;
        } else {
          const float2 f = have ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
          y[x][0] = f.x, y[x][1] = f.y;
        }
      }
      float m_new = m;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) m_new = fmaxf(m_new, v[x].x);
      const float mu = m_new == -INFINITY ? 0.f : m_new;
      const float old = exp2_fast(m - mu);
      m = m_new;
      sum *= old;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] *= old;
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const float f = exp2_fast(v[x].x - mu);  // 0 where there is none
        sum += v[x].y * f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += y[x][i] * f;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) part_o[warp][lane * kPer + i] = acc[i];
    if (lane == 0) part_ml[warp] = make_float2(m, sum);
    __syncthreads();
    if (live && warp % kShare == 0) {
#pragma unroll
      for (int x = 0; x < kShare; ++x) m = fmaxf(m, part_ml[warp + x].x);
      const float mu = m == -INFINITY ? 0.f : m;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
#pragma unroll
      for (int x = 0; x < kShare; ++x) {
        const float2 v = part_ml[warp + x];
        const float f = exp2_fast(v.x - mu);
        sum += v.y * f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += part_o[warp + x][lane * kPer + i] * f;
      }
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      uint16_t* dst =
          a.o + (static_cast<int64_t>(seq) * a.n_tokens + t) * a.o_stride + h * HD + lane * kPer;
      if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                    pack_bf16x2(acc[2] * inv, acc[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ launch

int column_tiles(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : kMaxTiles; }
int blocks_per_sm(int format, int hd, int nt) {  // Cfg::kBlocks
  return nt == kMaxTiles || (format == PDS_KV_BF16 && hd == 128) ? 1 : 2;
}

// Few short ranges: their chunks are the blocks of a cluster, which join them over
// distributed shared memory, one launch instead of two and no workspace.  Up to
// this many blocks, and this many chunks of the shortest length between them:
// beyond, the two launches spread the keys over more SMs.  us with and without
// clusters: 1 token, bf16, 1000 keys 5.6/6.3, 2048 5.9/6.2, 4000 7.2/6.9 (but a
// launch less to issue), 8000 9.9/8.9; 4 sequences, int4, 1000 5.9/8.0, 4000 10.7/13.1.
constexpr int kMaxCluster = 8;
constexpr int kClusterChunks = 16;

// From this many query rows per kv head on, the tcgen05 kernel.  us here and there
// for 8 sequences of 4096 rows, 24 rows: bf16 33.9/32.2, e4m3 33.8/36.5, 4-bit
// 34.5/36.1; one sequence of 8192: 13.1/17.0, 13.3/18.8, 13.9/19.0.  36 rows (two
// row tiles here): 46.9/32.8, 49.4/37.3, 53.6/37.1.  (Several bf16 sequences alone would
// gain a twentieth from a limit of their own.)
constexpr int kTileMinRows = 33;

struct Shape {
  bool tiles;            // the tensor-core kernel
  int nt;                // the warp kernel's column tiles
  int step_shift, tile_rows;  // log2 of a step's keys, query rows of a block
  int row_tiles, per;    // blocks of rows per kv head, and per sequence
  int slots, fit;
};

// How a call's rows are tiled and over how many blocks its keys are spread.
Shape make_shape(int format, int hd, int n_seqs, int n_tokens, int n_heads, int n_kv_heads,
                 int num_sms) {
  Shape s{};
  const int rows = n_tokens * (n_heads / n_kv_heads);
  s.tiles = rows >= kTileMinRows;
  s.nt = column_tiles(rows);
  s.step_shift = s.tiles ? 6 : 4;
  s.tile_rows = s.tiles ? (rows <= 128 ? 128 : 256) : 8 * s.nt;
  s.row_tiles = (rows + s.tile_rows - 1) / s.tile_rows;
  s.per = n_kv_heads * s.row_tiles;
  const int64_t units = static_cast<int64_t>(n_seqs) * s.per;
  const int resident = num_sms * (s.tiles ? 1 : blocks_per_sm(format, hd, s.nt));
  // One wave where all (sequence, head, tile) fit at once.  Where they do not,
  // only what is longer than an average block's share is cut.  Shorter chunks
  // balance better but every block costs some microseconds of its own: 16
  // sequences of 4096 e4m3 rows take 29.8 us in one wave, 33.7 in two, 38.9 in
  // four; 64 sequences of 1024 (64-wide heads) 26.0 cut so, 33.4 cut in two waves.
  s.fit = units <= resident;
  s.slots = resident;
  return s;
}

int64_t max_units(const Shape& s, int n_seqs) {
  return s.fit ? s.slots : s.slots + static_cast<int64_t>(n_seqs) * s.per;
}

template <int FMT, int HD, int NT, bool VAR>
cudaError_t launch(const Args& a, int64_t grid, cudaStream_t st) {
  using C = Cfg<FMT, HD, NT>;
  static_assert(C::kBlocks == (NT == kMaxTiles || (FMT == PDS_KV_BF16 && HD == 128) ? 1 : 2),
                "blocks_per_sm() says how many blocks an SM holds");
  const cudaError_t ce = kernel_smem_attr(
      reinterpret_cast<const void*>(cache_attn_kernel<FMT, HD, NT, VAR>), C::kSmem);
  if (ce != cudaSuccess) return ce;
  return launch_after_cluster(cache_attn_kernel<FMT, HD, NT, VAR>,
                              dim3(static_cast<unsigned>(grid)), kThreads, C::kSmem, a.cluster, st, a);
}

template <int FMT, int HD>
cudaError_t launch_rows(const Args& a, int nt, int64_t grid, cudaStream_t st) {
  const bool var = a.cap > 0.f || a.window > 0;
  switch (nt) {
    case 1: return var ? launch<FMT, HD, 1, true>(a, grid, st) : launch<FMT, HD, 1, false>(a, grid, st);
    case 2: return var ? launch<FMT, HD, 2, true>(a, grid, st) : launch<FMT, HD, 2, false>(a, grid, st);
    default: return var ? launch<FMT, HD, 4, true>(a, grid, st) : launch<FMT, HD, 4, false>(a, grid, st);
  }
}

template <int HD>
cudaError_t launch_format(const Args& a, int format, int nt, int64_t grid, cudaStream_t st) {
  switch (format) {
    case PDS_KV_BF16: return launch_rows<PDS_KV_BF16, HD>(a, nt, grid, st);
    case PDS_KV_E4M3: return launch_rows<PDS_KV_E4M3, HD>(a, nt, grid, st);
    default: return launch_rows<PDS_KV_INT4, HD>(a, nt, grid, st);
  }
}

}  // namespace

size_t tree_attention_ws_bytes(int format, int hd, int n_seqs, int n_tokens, int n_heads,
                               int n_kv_heads, int num_sms) {
  const Shape s = make_shape(format, hd, n_seqs, n_tokens, n_heads, n_kv_heads, num_sms);
  return static_cast<size_t>(max_units(s, n_seqs)) * s.tile_rows * (hd * 4 + 8);
}

pds_status tree_attention(const TreeAttnCall& t, cudaStream_t st, std::string* err) {
  const CacheView& c = t.cache;
  const Shape s = make_shape(t.format, t.head_dim, c.n_seqs, t.n_tokens, t.n_heads, c.n_kv_heads,
                             t.num_sms);
  Args a{};
  a.c = c;
  a.q = t.q;
  a.o = t.o;
  a.q_stride = t.q_stride;
  a.o_stride = t.o_stride;
  a.parents = t.parents;
  a.n_tokens = t.n_tokens;
  a.n_heads = t.n_heads;
  a.group = t.n_heads / c.n_kv_heads;
  a.per_group = 1.0f / static_cast<float>(a.group);
  a.max_len = t.max_len;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(t.head_dim));
  a.cap = t.softcap > 0.f ? t.softcap * sqrtf(static_cast<float>(t.head_dim)) : 0.f;
  a.window = t.window;
  a.row_tiles = s.row_tiles;
  a.tile_rows = s.tile_rows;
  a.step_shift = s.step_shift;
  // Two steps per warp, four tiles: with half 8 x 600 4-bit rows take 8.7 us
  // instead of 7.0, with double one token over 600 e4m3 rows 5.8 instead of 4.8.
  a.min_steps = s.tiles ? 4 : 2 * kWarps;
  a.status = t.status;
  // a window's keys, with whole steps at both ends
  const int64_t prefix = t.window > 0 ? std::min<int64_t>(t.max_len, int64_t{t.window} + (2 << s.step_shift))
                                      : t.max_len;
  const int64_t span = prefix + t.n_tokens;
  const int64_t least = static_cast<int64_t>(a.min_steps) << a.step_shift;
  const int64_t most_chunks = (span + least - 1) / least;
  // One row tile's two streams take every other tile of keys: three each cost no
  // more than a second chunk and the join (us uncut/cut for 4 sequences of 16 tokens,
  // 32/8 heads of 64, over 350 rows: bf16 7.5/9.7, e4m3 9.1/10.8; over 550 10.2/10.2).
  const int64_t uncut = s.tiles && s.tile_rows == 128 ? least + least / 2 : least;
  const int64_t units = static_cast<int64_t>(c.n_seqs) * s.per;
  int64_t grid = units;
  int cluster = 1;
  while (cluster < kMaxCluster && cluster < most_chunks) cluster *= 2;
  a.cluster = 1;
  if (!s.tiles && cluster > 1 && most_chunks <= kClusterChunks && units * cluster <= s.slots) {
    a.cluster = cluster;
    grid = units * cluster;
  } else if (t.ws && span > uncut && s.per < s.slots) {  // (else a range per SM at least)
    a.slots = s.slots;
    a.fit = s.fit;
    a.per_chunk = 1.0f / static_cast<float>(s.slots / s.per);
    const int64_t most = max_units(s, c.n_seqs);
    grid = std::min(most, units * most_chunks);
    a.o_part = reinterpret_cast<float*>(t.ws);
    a.ml_part = reinterpret_cast<float2*>(t.ws + static_cast<size_t>(most) * a.tile_rows *
                                                     t.head_dim * 4);
  }
  cudaError_t ce = s.tiles ? launch_tile_attention(a, t.format, t.head_dim, grid, t.num_sms, st)
                   : t.head_dim == 128 ? launch_format<128>(a, t.format, s.nt, grid, st)
                                       : launch_format<64>(a, t.format, s.nt, grid, st);
  if (ce == cudaSuccess && a.slots > 0 && !s.tiles) {
    const int64_t rows = static_cast<int64_t>(c.n_seqs) * t.n_tokens * t.n_heads;
    const dim3 blocks(static_cast<unsigned>(std::min<int64_t>((rows + 1) / 2, 8 * t.num_sms)));
    ce = t.head_dim == 128 ? launch_after(cache_join_kernel<128>, blocks, 256, 0, st, a)
                           : launch_after(cache_join_kernel<64>, blocks, 256, 0, st, a);
  }
  if (ce != cudaSuccess) {
    *err = std::string("cache attention launch: ") + cudaGetErrorString(ce);
    return PDS_ELAUNCH;
  }
  return PDS_OK;
}

}  // namespace pds
