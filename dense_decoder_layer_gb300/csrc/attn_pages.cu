// Attention of one new token per sequence over a paged K/V cache, split over the
// cache's length and joined.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = 2^(x_j - m),   x_j = log2(e) q.k_j / sqrt(hd)
//
// (x_j capped first where a softcap is given).  A row of K and of V is read once for the
// G query heads of its kv head: 4 G hd operations for 2 hd values, far below what
// the tensor cores could do, so HBM bounds it, and everything between HBM and the
// products has to keep out of the way.
//
// Both products therefore take the cached rows as the 128-row operand of tcgen05.mma, as TMA
// lays them into shared memory, page by page, and the few query heads as its columns:
//   S[128 keys x heads]    = K[128 keys x hd] Q^T      (lane = key)
//   O[hd channels x heads] = V^T[hd x 128 keys] P      (lane = channel)
// A thread of the softmax has one key: its scale words are its own numbers, its weights
// 16-byte rows of P, and O needs no exchange either (a thread has one channel of every
// head, in registers, rescaled as the reference moves).  Rows of 8 bits enter the
// products as they are; 4-bit codes become bytes by a mask and a shift: the byte c < 16 is
// the e4m3 number c 2^-9, and the zero points come off as z sum(q), z sum(p).
//   * e4m3 products need the other operand in e4m3: Q as the sum of two pieces (the
//     second in sixteenths; exact for channels down to 2^-13 of the row's largest), P in
//     fp16 (2^-11 of a weight) as the sum of three, in columns of their own.
//   * bf16 rows: Q as it is, P as the sum of two bf16 pieces (2^-16).
// Over codes P is the weight times V's scale, against the largest such product met (to within
// the scale's mantissa); the sum of the weights is kept against the same number less
// the exponent of the unit's first V scale that is not 0, so it stays in range while scales lie within
// 2^80; a row of zeros takes part with 2^-80 of that scale.
//
// The tiles of all (sequence, kv head, group of heads) units, in this order, are cut into
// equal shares, one per block, whatever the lengths: a block works on the end of one unit, on
// whole ones and on the start of another.  Units cut so are joined by a second kernel from
// normalised float32 parts.  Few short units are a cluster's each instead, and joined in it.
//
// A block, two per SM: warps 0-3 softmax and O, warp 4 copies and the scale words, warp 5
// products, warp 7 Q of the next units; for e4m3 rows of 64 channels, whose copies one warp does
// not issue fast enough, warp 6 takes V's and the words.  With 4-bit rows warps 6 and 7 spread K's
// and V's codes, and warp 6 makes Q.  Every wait is bounded: one that gives up sets the abort flag and
// the status word; from then on no wait waits, nothing is copied or multiplied any more, and the
// block runs to its end in order.
//
// Measured in replayed graphs, us (and the bytes at a copy's rate, which a kernel that only reads may
// beat by a hundredth or two): 32 sequences of 8192 rows, 32/8 x 128, pages of 16: bf16 162 (158), e4m3 85 (81.5),
// 4 bits 77 (42; pages of 64: 72); 16 of 4096 rows 46 (39.5), 27 (20.4), 26 (10.5); one of 2048 rows, 24/8, bf16
// 6.9.  bf16 and e4m3 are bound by HBM.  4 bits are by the conversion (without it 59 of the 72), which reads codes from shared
// memory and writes bytes that the products read again, half of shared memory's cycles in all; and
// then, as e4m3 of 64 channels (52, HBM 42), by warp 5, which takes 1600 cycles for a tile's waits, products
// and commits.  Single tokens are a chain of latencies: length, table, page, scores, weights, O.
// More than eight query heads per kv head are units of their own, a length each: 64/4 heads over 16 sequences of 4096
// bf16 rows read 217 MB where the rows are 134, over 32 of 8192 164 us take twice the bytes' time (79).
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attn_cache.cuh"
#include "fastmath.cuh"
#include "kv_rows.cuh"
#include "pages.h"
#include "sm100.cuh"
#include "tc.h"

namespace pds {
namespace {

using cacheattn::capped;
using cacheattn::capped_wide;
using cacheattn::copy16;
using cacheattn::exp2_fast;
using cacheattn::soft_cap;
using cacheattn::SoftCap;

constexpr int kKeys = 128;
constexpr int kBlocksPerSm = 2;
constexpr int kMaxHeads = 8;  // query heads of a unit
constexpr int kMaxCluster = 8;

struct PagedArgs {
  PageView p;
  const int32_t* new_rows;
  const uint16_t* q;
  uint16_t* o;
  int64_t q_stride, o_stride;
  int n_heads, group;      // group: query heads per kv head
  int chunk, n_chunks;     // heads of a unit, units per kv head
  float scale_log2, cap_log2;
  int window;
  int whole_pages;         // a head's rows of a page lie side by side
  int cluster;             // > 1: a unit per cluster of so many blocks
  uint32_t* status;
  int4* desc;              // [blocks]: flags, sequence, unit of the sequence
  float2* ml;              // [2 blocks][kMaxHeads]: reference, sum
  float* part;             // [2 blocks][kMaxHeads][hd]: normalised
};
constexpr int kHasEnd = 1, kEndsUnit = 2, kHasStart = 4;  // desc flags

template <int FMT, int HD, int GT>
struct Cfg {
  static constexpr bool kCodes = FMT != PDS_KV_BF16, kInt4 = FMT == PDS_KV_INT4;
  static constexpr int kEl = kCodes ? 1 : 2;                  // bytes of an operand's element
  static constexpr int kOpRow = HD * kEl;                     // of an operand row
  static constexpr int kBlk = kOpRow < 128 ? kOpRow : 128;    // swizzled column block
  static constexpr int kBlks = kOpRow / kBlk;
  static constexpr uint32_t kTile = 128u * kOpRow;
  static constexpr int kRawRow = kInt4 ? HD / 2 : kOpRow;
  static constexpr uint32_t kHalf = 128u * kRawRow;           // a tile of K or V as it arrives
  // Stages: tile i's K is half 2 i, its V half 2 i + 1, half h in stage h % kRing.  A wait
  // tells phases of a stage apart by their parity, so whoever waits for a half has to know that
  // the one before it in its stage was there.  With an even number of stages K and V have stages of
  // their own, and one after the other suffices: each may have a copier, and a converter.  With
  // an odd one the copier has to be one, and whoever waits has to take them as they come.
  static constexpr int kRing = FMT == PDS_KV_BF16 ? (HD == 128 ? 3 : 6)
                               : kInt4            ? (HD == 64 ? 10 : 4)
                                                  : (HD == 64 ? 10 : GT > 4 ? 4 : 6);
  static_assert(kRing % 2 == 0 || FMT == PDS_KV_BF16, "converters wait for K's or V's halves only");
  static constexpr bool kTwoCopiers = FMT == PDS_KV_E4M3 && HD == 64;
  // (a tile's words are read until its weights are made, two tiles behind its scores)
  static constexpr int kWordSlots = kCodes ? kRing / 2 + 4 : 0;
  static constexpr int kQParts = kCodes ? 2 : 1, kPParts = kCodes ? 3 : 2;
  static constexpr int kSCols = kQParts * GT, kOCols = kPParts * GT;  // used columns
  static constexpr int kQRows = (kSCols + 7) / 8 * 8;
  static constexpr int kN = 16;                               // columns of S
  static constexpr int kNO = kOCols > 16 ? 32 : 16;           // of O
  static constexpr int kPGroups = kNO * kEl / 16;             // 16-byte groups of a key's row of P
  static constexpr uint32_t kQBlk = kQRows * kBlk, kQ = kQBlk * kBlks;
  static constexpr uint32_t kP = 2048u * kPGroups;
  static constexpr uint32_t kRingAt = 0;
  // 4 bits: the bytes of two tiles of K and of V (eight heads of 128 channels leave no room for two of V)
  static constexpr uint32_t kConvAt = (kRing * kHalf + 1023) / 1024 * 1024;
  static constexpr int kVBytes = HD == 128 && GT > 4 ? 1 : 2;
  static constexpr uint32_t kQAt = kConvAt + (kInt4 ? (2 + kVBytes) * kTile : 0u);
  static constexpr uint32_t kPAt = kQAt + 2 * kQ + 1024;      // (columns that nobody reads: past Q's rows)
  static constexpr uint32_t kWordsAt = kPAt + 2 * kP;
  static constexpr uint32_t kXchAt = kWordsAt + kWordSlots * 1024u;   // [2][GT][4] maxima
  static constexpr uint32_t kSumAt = kXchAt + 2 * GT * 16;            // [2][2 GT][4] sums
  static constexpr uint32_t kQMulAt = kSumAt + 2 * 2 * GT * 16;           // [4][2][GT]: factors, sums of Q
  static constexpr uint32_t kBar = kQMulAt + 4 * 2 * GT * 4;
  static constexpr int kNumBars = 2 * kRing + 2 * (kWordSlots > 0 ? kWordSlots : 1) + 2 + 2 + 2 + 2 + 2 + 8 + 1;
  static constexpr uint32_t kMisc = kBar + 8 * kNumBars;              // TMEM address, abort flag
  static constexpr uint32_t kSums = kMisc + 16;                       // tiles per 32 sequences
  static constexpr uint32_t kEndOf = kSums + 4 * (kMaxPagedSeqs / 32);
  static constexpr size_t kSmem = 1024 + kEndOf;
  static_assert(kSmem <= (233472 - 2048) / kBlocksPerSm, "two blocks per SM");
  static constexpr int kThreads = 256;
  static constexpr uint32_t kTmemCols = 128, kTmS = 0, kTmO = 32;
  static constexpr int kKeyStep = 32 / kEl;  // keys of a step of the second product
};

// ------------------------------------------------------------ instructions

__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
__device__ __forceinline__ bool try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns) {
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
// The bounded wait of a converged warp.  After an abort it does not wait.  What is seldom
// run is called, not inlined: a block that lives for a tile or two has to fetch its code first.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                     uint32_t* status) {
  const uint64_t t0 = sm100::global_timer_ns();
  while (!try_wait_for(bar, parity, 100000u)) {
    if (*abort_flag) return false;
    if (sm100::global_timer_ns() - t0 > sm100::kWaitLimitNs) {
      *abort_flag = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}
// Whether the phase was reached, the same in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          uint32_t* status) {
  const bool there = sm100::mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, there)) return true;
  return __all_sync(0xffffffffu, there || wait_on(bar, parity, abort_flag, status));
}
// The same for a block that leaves: not cut short by the abort flag.
__device__ __noinline__ void last_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = sm100::global_timer_ns();
  while (!try_wait_for(bar, parity, 100000u) && sm100::global_timer_ns() - t0 < sm100::kWaitLimitNs) {
  }
  __syncwarp();
}

// Products and commits come from one elected lane, with operands that the compiler knows to be the
// same in all: they stay in uniform registers.  a, b: low words of the matrices' descriptors.
__device__ __forceinline__ uint32_t same_in_warp(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
template <bool F8>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t id,
                                    bool accumulate) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\t"
        "mov.b64 db, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(id), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 da, {%1, %2};\n\t"
        "mov.b64 db, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(id), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// Shared-memory matrix descriptor: address and byte offset `lead` in the low word, byte offset
// `stride` and layout (0 none, 2 128-byte swizzle, 4 64-byte) in the high one.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3FFFu) | (lead >> 4) << 16;
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride, uint32_t layout) {
  return stride >> 4 | 1u << 14 | layout << 29;
}
// Instruction descriptor: float32 accumulator, both operands bf16 or both e4m3 (format 0), A and B
// MN-major or not.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// A box of a page: channels x, rows from y, kv head h, page p.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                         int h, int page, uint64_t hint) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(h), "r"(page), "r"(bar), "l"(hint)
      : "memory");
}
// This thread's copies so far arrive on `bar` (one of its count) when they are there.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void load_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
// Columns of this thread's lane: A from one address and B from another (either may be none), with the
// wait in the same statement, so that nothing touches the registers before they are there.
template <int A, int B>
__device__ __forceinline__ void tmem_read(uint32_t addr_a, float (&va)[A], uint32_t addr_b, float (&vb)[B]);
#define PDS_OUT4(v, i) "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
template <>
__device__ __forceinline__ void tmem_read<4, 8>(uint32_t a, float (&va)[4], uint32_t b, float (&vb)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%12];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%4, %5, %6, %7, %8, %9, %10, %11}, [%13];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : PDS_OUT4(va, 0), PDS_OUT4(vb, 0), PDS_OUT4(vb, 4)
      : "r"(a), "r"(b)
      : "memory");
}
template <>
__device__ __forceinline__ void tmem_read<8, 12>(uint32_t a, float (&va)[8], uint32_t b, float (&vb)[12]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%20];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%21];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%16, %17, %18, %19}, [%22];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : PDS_OUT4(va, 0), PDS_OUT4(va, 4), PDS_OUT4(vb, 0), PDS_OUT4(vb, 4), PDS_OUT4(vb, 8)
      : "r"(a), "r"(b), "r"(b + 8)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_read(uint32_t a, float (&v)[N]) {
  if constexpr (N == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PDS_OUT4(v, 0)
        : "r"(a)
        : "memory");
  } else if constexpr (N == 8) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PDS_OUT4(v, 0), PDS_OUT4(v, 4)
        : "r"(a)
        : "memory");
  } else if constexpr (N == 12) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%12];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%8, %9, %10, %11}, [%13];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PDS_OUT4(v, 0), PDS_OUT4(v, 4), PDS_OUT4(v, 8)
        : "r"(a), "r"(a + 8)
        : "memory");
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PDS_OUT4(v, 0), PDS_OUT4(v, 4), PDS_OUT4(v, 8), PDS_OUT4(v, 12)
        : "r"(a)
        : "memory");
  } else {
    static_assert(N == 24, "columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
        "%13, %14, %15}, [%24];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%25];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : PDS_OUT4(v, 0), PDS_OUT4(v, 4), PDS_OUT4(v, 8), PDS_OUT4(v, 12), PDS_OUT4(v, 16), PDS_OUT4(v, 20)
        : "r"(a), "r"(a + 16)
        : "memory");
  }
}
#undef PDS_OUT4
// An integer below 2^23 as a float, without the conversion pipe.
__device__ __forceinline__ float small_float(uint32_t x) {
  return __uint_as_float(x | 0x4b000000u) - 8388608.f;
}
__device__ __forceinline__ float warp_top(float x) {  // NaN is passed over
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Two numbers as e4m3 codes, the first in the low byte, and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}
__device__ __forceinline__ uint32_t to_e4m3x2(__half2 x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return d;
}
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return *reinterpret_cast<const __half2*>(&h);
}
__device__ __forceinline__ float ld_cluster(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(static_cast<uint16_t>(v)) : "memory");
}
__device__ __forceinline__ void sts8(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b8 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// ---------------------------------------------------------------- schedule

struct Rows {  // of a sequence: visible rows [lo, hi), the tiles that hold them
  int lo, hi, t0, tiles;
};
__device__ __forceinline__ Rows seq_rows(const PagedArgs& a, int s) {
  Rows r{0, 0, 0, 0};
  if (s >= a.p.n_seqs) return r;
  const int64_t end = rows_end(a.p, a.new_rows, s);
  if (end <= 0) return r;
  r.hi = static_cast<int>(end);
  r.lo = a.window > 0 ? max(r.hi - a.window, 0) : 0;
  r.t0 = r.lo / kKeys;
  r.tiles = (r.hi - 1) / kKeys + 1 - r.t0;
  return r;
}

// n / d for n >= 0, d > 0, without the long way round that the compiler takes: the quotient of the
// rounded numbers is off by 2^-21 of itself at most, that of what is left by less than one.
__device__ __forceinline__ int quotient(int n, int d) {
  const float per = __fdividef(1.0f, static_cast<float>(d));
  int q = static_cast<int>(static_cast<float>(n) * per);
  int r = n - q * d;
  q += static_cast<int>(floorf(static_cast<float>(r) * per));
  r = n - q * d;
  return r < 0 ? q - 1 : r >= d ? q + 1 : q;
}
__device__ __forceinline__ int warp_incl(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// One warp's walk over a block's tiles; every lane holds the rows of one of 32
// sequences, the walk's own numbers are the same in all lanes.
struct Walk {
  Rows mine;
  int base;               // first of the 32 sequences
  int s, unit, t;         // sequence, unit of it, tile of the unit
  int kvh, part;          // the unit's kv head, and which of its groups of heads
  Rows cur;
  __device__ __forceinline__ void take(int lane) {
    s = base + lane;
    cur.lo = __shfl_sync(0xffffffffu, mine.lo, lane);
    cur.hi = __shfl_sync(0xffffffffu, mine.hi, lane);
    cur.t0 = __shfl_sync(0xffffffffu, mine.t0, lane);
    cur.tiles = __shfl_sync(0xffffffffu, mine.tiles, lane);
  }
  // To tile b of all, b below the sum; sums: tiles of one unit each per 32 sequences (not used
  // for 32 sequences or fewer, whose rows `mine` holds already).
  __device__ __forceinline__ void start(const PagedArgs& a, const int* sums, int units, int b) {
    const int lane = threadIdx.x & 31;
    int from = 0, c = 0;
    const int chunks = (a.p.n_seqs + 31) >> 5;
    for (int c0 = 0; chunks > 1; c0 += 32) {
      const int n = c0 + lane < chunks ? sums[c0 + lane] * units : 0;
      const int incl = warp_incl(n);
      const unsigned hit = __ballot_sync(0xffffffffu, from + incl > b);
      if (hit) {
        const int l = __ffs(hit) - 1;
        c = c0 + l;
        from += __shfl_sync(0xffffffffu, incl - n, l);
        break;
      }
      from += __shfl_sync(0xffffffffu, incl, 31);
      if (c0 + 32 >= chunks) break;  // (cannot be)
    }
    base = c * 32;
    if (chunks > 1) mine = seq_rows(a, base + lane);
    const int n = mine.tiles * units, incl = warp_incl(n);
    const unsigned hit = __ballot_sync(0xffffffffu, from + incl > b);
    const int l = hit ? __ffs(hit) - 1 : 0;
    take(l);
    const int rest = b - from - __shfl_sync(0xffffffffu, incl - n, l);
    unit = quotient(rest, max(cur.tiles, 1));
    t = rest - unit * cur.tiles;
    kvh = quotient(unit, a.n_chunks);
    part = unit - kvh * a.n_chunks;
  }
  // To the next tile (there is one).
  __device__ __forceinline__ void next(const PagedArgs& a, int units) {
    if (++t < cur.tiles) return;
    t = 0;
    if (++part == a.n_chunks) {
      part = 0;
      ++kvh;
    }
    if (++unit < units) return;
    unit = kvh = part = 0;
    unsigned later = __ballot_sync(0xffffffffu, mine.tiles > 0);
    const int l = s - base;
    later = l == 31 ? 0u : later & (0xffffffffu << (l + 1));
    while (!later && base + 32 < a.p.n_seqs) {
      base += 32;
      mine = seq_rows(a, base + (threadIdx.x & 31));
      later = __ballot_sync(0xffffffffu, mine.tiles > 0);
    }
    if (later) take(__ffs(later) - 1);
  }
  __device__ __forceinline__ int key0() const { return (cur.t0 + t) * kKeys; }
  __device__ __forceinline__ bool hides() const {  // a key of the tile that is not seen
    return key0() < cur.lo || key0() + kKeys > cur.hi;
  }
};

// Of 128 scale words in shared memory, those of the rows lo .. hi - 1: the biased exponent of the first that
// is neither 0 nor none (else 0), in all lanes.  Seldom run.
__device__ __noinline__ uint32_t first_exponent(uint32_t words, int lo, int hi) {
  const int row = 4 * (threadIdx.x & 31);
  const uint4 w = lds128(words + row * 4);
  const uint32_t word[4] = {w.x, w.y, w.z, w.w};
  uint32_t e = 0;
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    const uint32_t mine = word[k] >> 23 & 255u;
    if (row + k >= lo && row + k < hi && mine - 1u < 254u) e = mine;
  }
  const unsigned have = __ballot_sync(0xffffffffu, e != 0);
  return have ? __shfl_sync(0xffffffffu, e, __ffs(have) - 1) : 0u;
}

// Sums over the warp of N values per lane (N a power of two up to 16): N - 1 exchanges
// halve them, the others finish; lane l ends with value number l % N.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = N / 2; h > 0; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, h);
    }
  }
  float x = v[0];
#pragma unroll
  for (int o = N; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int FMT, int HD, int GT, bool CAP>
__global__ void __launch_bounds__(Cfg<FMT, HD, GT>::kThreads, kBlocksPerSm)
    pages_attn_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
  using namespace sm100;
  using C = Cfg<FMT, HD, GT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t sb = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sb - raw_base);
  const uint32_t bar0 = sb + C::kBar;
  constexpr int R = C::kRing, W = C::kWordSlots > 0 ? C::kWordSlots : 1;
  auto bar_full = [&](int i) { return bar0 + 8u * i; };
  auto bar_empty = [&](int i) { return bar0 + 8u * (R + i); };
  auto bar_word = [&](int i) { return bar0 + 8u * (2 * R + i); };
  auto bar_word_free = [&](int i) { return bar0 + 8u * (2 * R + W + i); };
  constexpr int kB2 = 2 * R + 2 * W;
  auto bar_q = [&](int i) { return bar0 + 8u * (kB2 + i); };
  auto bar_q_free = [&](int i) { return bar0 + 8u * (kB2 + 2 + i); };
  auto bar_s = [&](int i) { return bar0 + 8u * (kB2 + 4 + i); };
  auto bar_p = [&](int i) { return bar0 + 8u * (kB2 + 6 + i); };
  auto bar_o = [&](int i) { return bar0 + 8u * (kB2 + 8 + i); };
  auto bar_c = [&](int kv, int i) { return bar0 + 8u * (kB2 + 10 + 2 * kv + i); };
  auto bar_c_free = [&](int kv, int i) { return bar0 + 8u * (kB2 + 14 + 2 * kv + i); };
  const uint32_t bar_done = bar0 + 8u * (kB2 + 18);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  int* sums = reinterpret_cast<int*>(smem + C::kSums);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = C::kThreads / 32;
  const int units = a.p.n_kv_heads * a.n_chunks;  // of a sequence

  if (warp == 5) tmem_alloc(sb + C::kMisc, C::kTmemCols), tmem_relinquish();
  if (threadIdx.x == 0) {
    for (int i = 0; i < R; ++i) {
      mbar_init(bar_full(i), 1);
      mbar_init(bar_empty(i), 1);
    }
    for (int i = 0; i < W; ++i) {
      mbar_init(bar_word(i), 32);
      mbar_init(bar_word_free(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q(i), 1);
      mbar_init(bar_q_free(i), 1);
      mbar_init(bar_s(i), 1);
      mbar_init(bar_p(i), 4);
      mbar_init(bar_o(i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_c(i >> 1, i & 1), 1);
      mbar_init(bar_c_free(i >> 1, i & 1), 1);
    }
    mbar_init(bar_done, 1);
    mbar_init_fence();
    *abort_flag = 0;
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds32(sb + C::kMisc);
  const int chunks = (a.p.n_seqs + 31) >> 5;
  Walk w;
  int n = 0;            // this block's tiles
  int unit_tiles = 0;   // (a cluster's unit)
  const uint32_t rank = a.cluster > 1 ? cluster_rank() : 0u;
  if (a.cluster > 1) {
    const int u = static_cast<int>(blockIdx.x) / a.cluster;
    w.base = u / units;
    w.unit = u - w.base * units;
    w.kvh = w.unit / a.n_chunks;
    w.part = w.unit - w.kvh * a.n_chunks;
  }
  grid_dep_wait();
  grid_dep_launch();
  if (a.cluster > 1) {
    // (the sequence's first pages on their way while its length is)
    if (lane * 32 < a.p.max_pages)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(a.p.table + static_cast<int64_t>(w.base) * a.p.max_pages + lane * 32));
    w.mine = seq_rows(a, w.base);
    w.take(0);
    unit_tiles = w.cur.tiles;
    const int each = quotient(unit_tiles, a.cluster), more = unit_tiles - each * a.cluster, r = static_cast<int>(rank);
    w.t = each * r + min(r, more);
    n = each + (r < more ? 1 : 0);
  } else {
    w.mine = seq_rows(a, (chunks > 1 ? 32 * warp : 0) + lane);
    int total = __reduce_add_sync(0xffffffffu, w.mine.tiles);
    if (chunks > 1) {
      for (int c = warp; c < chunks; c += kWarps) {
        if (c != warp) total = __reduce_add_sync(0xffffffffu, seq_rows(a, c * 32 + lane).tiles);
        if (lane == 0) sums[c] = total;
      }
      __syncthreads();
      total = 0;
      for (int c = lane; c < chunks; c += 32) total += sums[c];
      total = __reduce_add_sync(0xffffffffu, total);
    }
    total *= units;
    // Equal shares; every block up to the last that has any has tiles: the join counts on it.
    const int share = min(total, static_cast<int>(gridDim.x)), x = blockIdx.x;
    if (x < share) {
      const int each = quotient(total, share), more = total - each * share;
      n = each + (x < more ? 1 : 0);
      w.start(a, sums, units, each * x + min(x, more));
    }
  }

  // Q of a unit, in the products' order of bytes
  auto make_q = [&](int s, int kvh, int part, int unit_no) {
    constexpr int kPer = HD / 32;  // channels of a lane
    const uint32_t buf = unit_no & 1;
    if (unit_no >= 2) warp_wait(bar_q_free(buf), ((unit_no >> 1) - 1) & 1, abort_flag, a.status);
    const int first = part * a.chunk;
    const int heads = min(a.chunk, a.group - first);
    const uint16_t* q = a.q + s * a.q_stride + static_cast<int64_t>(kvh * a.group + first) * HD;
    const uint32_t dst = sb + C::kQAt + buf * C::kQ;
    uint32_t raw[GT][kPer / 2];
#pragma unroll
    for (int g = 0; g < GT; ++g) {
#pragma unroll
      for (int x = 0; x < kPer / 2; ++x) raw[g][x] = 0;
      if (g < heads) {
        if constexpr (kPer == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(q + g * HD + 4 * lane);
          raw[g][0] = v.x, raw[g][1] = v.y;
        } else {
          raw[g][0] = *reinterpret_cast<const uint32_t*>(q + g * HD + 2 * lane);
        }
      }
    }
    // byte of an operand row's position `at` (bytes) in row r
    auto place = [&](int r, int at) {
      const int blk = at / C::kBlk, in = at % C::kBlk, piece = in >> 4;
      const int mix = C::kBlk == 128 ? r & 7 : (r >> 1) & 3;
      return dst + blk * C::kQBlk + r * C::kBlk + ((piece ^ mix) << 4) + (in & 15);
    };
#pragma unroll
    for (int g = 0; g < GT; ++g) {
      if constexpr (!C::kCodes) {
        if constexpr (kPer == 4)
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(place(g, 8 * lane)), "r"(raw[g][0]),
                       "r"(raw[g][1])
                       : "memory");
        else
          sts32(place(g, 4 * lane), raw[g][0]);
      } else {
        float x[kPer];
        uint32_t top = 0;
        bool bad = false;
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
          x[c] = c & 1 ? __uint_as_float(raw[g][c / 2] & 0xffff0000u) : __uint_as_float(raw[g][c / 2] << 16);
          const uint32_t mag = __float_as_uint(x[c]) & 0x7fffffffu;
          bad |= mag >= 0x7f800000u;
          top = max(top, mag);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        bad = __any_sync(0xffffffffu, bad);
        // the power of two that brings the largest to 2^7 .. 2^8
        const int e = max(static_cast<int>(top >> 23), 30);
        const float mul = __uint_as_float(static_cast<uint32_t>(261 - min(e, 254) ) << 23);
        const float inv = __uint_as_float(static_cast<uint32_t>(max(min(e, 254) - 7, 1)) << 23);
        float sum = 0.f;
        uint32_t code[2][kPer / 2];
#pragma unroll
        for (int c = 0; c < kPer; c += 2) {
          const float y0 = x[c] * mul, y1 = x[c + 1] * mul;
          code[0][c / 2] = to_e4m3x2(y0, y1);
          const float2 p = __half22float2(from_e4m3x2(code[0][c / 2]));
          code[1][c / 2] = to_e4m3x2((y0 - p.x) * 16.f, (y1 - p.y) * 16.f);
          const float2 r = __half22float2(from_e4m3x2(code[1][c / 2]));
          sum += (p.x + p.y) + (r.x + r.y) * 0.0625f;
        }
        sum = warp_sum(sum);
        if (lane == 0) {
          // (read until a unit's last scores are: two units later, Q itself one)
          const uint32_t at = sb + C::kQMulAt + (unit_no & 3) * (2 * GT * 4) + g * 4;
          sts32(at, bad ? 0x7fc00000u : __float_as_uint(inv * a.scale_log2));
          sts32(at + GT * 4, __float_as_uint(sum));
        }
#pragma unroll
        for (int pc = 0; pc < 2; ++pc) {
          const int r = pc * GT + g;
          if constexpr (!C::kInt4) {
            if constexpr (kPer == 4) sts32(place(r, 4 * lane), code[pc][0] | code[pc][1] << 16);
            else sts16(place(r, 2 * lane), code[pc][0]);
          } else {
            // a chunk's 32 channels lie even ones first, as the nibbles come
            const int ch = kPer * lane, at = (ch & ~31) + ((ch & 31) >> 1);
            if constexpr (kPer == 4) {
              sts16(place(r, at), __byte_perm(code[pc][0], code[pc][1], 0x0040));
              sts16(place(r, at + 16), __byte_perm(code[pc][0], code[pc][1], 0x0051));
            } else {
              sts8(place(r, at), code[pc][0] & 255u);
              sts8(place(r, at + 16), code[pc][0] >> 8);
            }
          }
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_q(buf));
  };
  // The pages of a warp's tiles: 32 of a sequence from number `first` on, one a lane; n_pages for
  // one that is none.
  struct Pages {
    int32_t page = 0;
    int first = 0, of_seq = -1;
  };
  const int shift = a.p.page_shift, P = 1 << shift, box_rows = min(P, kKeys), per_tile = kKeys / box_rows;
  auto look_up = [&](Pages& pg) {
    const int p0 = w.key0() >> shift;
    if (w.s == pg.of_seq && p0 >= pg.first && p0 + per_tile <= pg.first + 32) return;
    pg.first = p0;
    pg.of_seq = w.s;
    const int at = p0 + lane;
    pg.page = 0;
    if (at >= w.cur.lo >> shift && at <= (w.cur.hi - 1) >> shift) {
      pg.page = a.p.table[static_cast<int64_t>(w.s) * a.p.max_pages + at];
      if (pg.page < 0 || pg.page >= a.p.n_pages) {
        atomicOr(a.status, kStatusBadPage);
        pg.page = a.p.n_pages;
      }
    }
  };
  // The scale words of the walk's tile, number i: four keys a lane, zeros where a page is none or not seen.
  const int word_lane = 4 * lane / box_rows, word_row = 4 * lane & (box_rows - 1);
  auto copy_words = [&](const Pages& pg, int i) {
    const int key0 = w.key0(), row = key0 + word_lane * box_rows;
    const int32_t page = __shfl_sync(0xffffffffu, pg.page, (key0 >> shift) - pg.first + word_lane);
    const bool ok = row < w.cur.hi && row + box_rows > w.cur.lo && page < a.p.n_pages;
    const int64_t at = ok ? ((static_cast<int64_t>(page) * a.p.n_kv_heads + w.kvh) << shift) + word_row +
                                (key0 & (P - 1))
                          : 0;
    const uint32_t dst = sb + C::kWordsAt + (i % W) * 1024u + lane * 16;
    copy16(dst, a.p.k_scale + at, ok);
    copy16(dst + 512, a.p.v_scale + at, ok);
  };
  // Copies of the tiles of K (kv 0) and V from kv0 to kv1, and of the scale words.
  auto copies = [&](auto kv0, auto kv1, auto words) {
    // (more than eight heads read a kv head's rows more than once)
    const uint64_t hint = a.n_chunks > 1 ? policy_evict_normal() : policy_evict_first();
    constexpr int kSteps = kv1 - kv0 + 1;
    Pages pg;
    int used = 0;               // tiles loaded so far
    [[maybe_unused]] int words_used = 0;
    int st = kv0;               // the half's stage
    uint32_t phase = 1;         // parity of its last use (the first: of none, which is over)
    for (int i = 0; i < n; ++i) {
      look_up(pg);
      const int key0 = w.key0(), y = key0 & (P - 1), row = key0 + lane * box_rows, kvh = w.kvh;  // (whole pages: y is 0)
      const bool live = lane < per_tile && row < w.cur.hi && row + box_rows > w.cur.lo;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * box_rows * C::kRawRow;
      // (a box outside of the pool is zeros)
      const int page = __shfl_sync(0xffffffffu, pg.page, ((key0 >> shift) - pg.first + lane) & 31);
      bool go = true;
      if constexpr (words) {
        if (i >= W) go = warp_wait(bar_word_free(i % W), (i / W - 1) & 1, abort_flag, a.status);
        if (!go) break;
        copy_words(pg, i);
        copies_arrive(bar_word(i % W));
        words_used = i + 1;
      }
      [[maybe_unused]] const Rows cur = w.cur;
      if (i + 1 < n) w.next(a, units);
      if constexpr (C::kInt4) {  // K's boxes by lanes 0 to 15, V's by the others (at most 16 pages a tile)
        go = warp_wait(bar_empty(st), phase, abort_flag, a.status) &&
             warp_wait(bar_empty(st + 1), phase, abort_flag, a.status);
        if (!go) break;
        used = i + 1;
        const int kv = lane >> 4, mine = lane & 15, at = key0 + mine * box_rows;
        const uint32_t bar = bar_full(st + kv);
        if (mine == 0) mbar_arrive_expect_tx(bar, bytes);
        const int pn = __shfl_sync(0xffffffffu, page, mine);
        __syncwarp();
        if (mine < per_tile && at < cur.hi && at + box_rows > cur.lo) {
          const uint32_t dst = sb + C::kRingAt + (st + kv) * C::kHalf + mine * box_rows * C::kRawRow;
          // a head's rows of a page side by side: one piece (64-byte rows one by one take TMA longer than
          // HBM would need for them)
          if (a.whole_pages && pn < a.p.n_pages)
            load_bytes(dst, (kv ? a.p.v : a.p.k) + pn * a.p.page_stride + (kvh * a.p.head_stride + y * C::kRawRow),
                       box_rows * C::kRawRow, bar);
          else
            load_box(dst, kv ? &map_v : &map_k, bar, 0, y, kvh, pn, hint);
        }
        __syncwarp();
        st += 2;
        if (st >= R) {
          st -= R;
          phase ^= 1;
        }
      } else {
#pragma unroll
        for (int kv = kv0; kv <= kv1; ++kv) {
          go = go && warp_wait(bar_empty(st), phase, abort_flag, a.status);
          if (!go) break;
          used = i + 1;
          const uint32_t bar = bar_full(st);
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (live) {
            const CUtensorMap* map = kv ? &map_v : &map_k;
            const uint32_t dst = sb + C::kRingAt + st * C::kHalf + lane * box_rows * C::kBlk;
#pragma unroll
            for (int x = 0; x < C::kBlks; ++x)
              load_box(dst + x * 128 * C::kBlk, map, bar, x * C::kBlk / C::kEl, y, kvh, page, hint);
          }
          __syncwarp();
          st += kSteps == 2 ? 1 : 2;
          if (st >= R) {
            st -= R;
            phase ^= 1;
          }
        }
      }
      if (!go) break;
    }
    // what was copied has landed before the block leaves
    for (int i = max(used - R, 0); i < used; ++i) {
#pragma unroll
      for (int kv = kv0; kv <= kv1; ++kv) {
        const int h = 2 * i + kv;
        if (h + R >= 2 * used) last_wait(bar_full(h % R), (h / R) & 1);
      }
    }
    if constexpr (words)
      for (int i = max(words_used - W, 0); i < words_used; ++i) last_wait(bar_word(i % W), (i / W) & 1);
  };
  using Zero = std::integral_constant<int, 0>;
  using One = std::integral_constant<int, 1>;

  if (warp == 4) {
    if (n > 0) copies(Zero{}, std::integral_constant<int, !C::kTwoCopiers>{},
                      std::bool_constant<C::kCodes && !C::kTwoCopiers>{});
    // meanwhile: sequences without a token are zeros, refused ones reported
    for (int s = blockIdx.x; s < a.p.n_seqs; s += gridDim.x) {
      const int64_t end = rows_end(a.p, a.new_rows, s);
      if (end < 0 && lane == 0) atomicOr(a.status, kStatusBadLength);
      if (end == 0)
        for (int i = lane; i < a.n_heads * (HD / 8); i += 32)
          *reinterpret_cast<uint4*>(a.o + s * a.o_stride + i * 8) = make_uint4(0, 0, 0, 0);
    }
  } else if (n > 0 && C::kTwoCopiers && warp == 6) {
    copies(One{}, One{}, std::bool_constant<C::kCodes>{});
  } else if (n > 0 && !C::kInt4 && warp == 7) {
    int unit_no = 0;
    for (int i = 0; i < n;) {
      make_q(w.s, w.kvh, w.part, unit_no++);
      const int rest = min(w.cur.tiles - w.t, n - i);
      i += rest;
      w.t += rest - 1;
      if (i < n) w.next(a, units);
    }
  } else if (n > 0 && warp == 5) {
    // ----------------------------------------------------------- products
    constexpr uint32_t kIdS = idesc(128, C::kN, !C::kCodes, false, false);
    constexpr uint32_t kIdO = idesc(HD, C::kNO, !C::kCodes, true, true);
    constexpr uint32_t kLayout = C::kBlk == 128 ? 2 : 4;
    int unit_no = 0;
    bool first = true;  // of the block, of a unit
    bool go = true;     // no wait has given up
    constexpr uint32_t kHiK = desc_hi(8 * C::kBlk, kLayout), kHiP = desc_hi(2048, 0);
    auto scores = [&](int i) {
      const bool last = w.t + 1 == w.cur.tiles || i + 1 == n;
      const int h = 2 * i, st = h % R;
      if (first) go = go && warp_wait(bar_q(unit_no & 1), (unit_no >> 1) & 1, abort_flag, a.status);
      if constexpr (C::kCodes)  // (S tells of the scale words too, which most often come before K)
        go = go && warp_wait(bar_word(i % W), (i / W) & 1, abort_flag, a.status);
      if constexpr (C::kInt4) go = go && warp_wait(bar_c(0, i & 1), (i >> 1) & 1, abort_flag, a.status);
      else go = go && warp_wait(bar_full(st), (h / R) & 1, abort_flag, a.status);
      tc_fence_after();
      const uint32_t ka = same_in_warp(desc_lo(C::kInt4 ? sb + C::kConvAt + (i & 1) * C::kTile
                                                        : sb + C::kRingAt + st * C::kHalf, 16));
      const uint32_t qa = same_in_warp(desc_lo(sb + C::kQAt + (unit_no & 1) * C::kQ, 16));
      const uint32_t d = same_in_warp(tmem + C::kTmS + (i & 1) * 16);
      if (go && elect_one()) {
#pragma unroll
        for (int x = 0; x < C::kOpRow / 32; ++x) {
          const uint32_t blk = x * 32 / C::kBlk, in = x * 32 % C::kBlk;
          mma<C::kCodes>(d, ka + ((blk * 128 * C::kBlk + in) >> 4), kHiK, qa + ((blk * C::kQBlk + in) >> 4), kHiK,
                         kIdS, x > 0);
        }
        umma_commit(C::kInt4 ? bar_c_free(0, i & 1) : bar_empty(st));
        umma_commit(bar_s(i & 1));
        if (last) umma_commit(bar_q_free(unit_no & 1));
      }
      __syncwarp();
      first = last;
      if (last) ++unit_no;
      if (i + 1 < n) w.next(a, units);
    };
    scores(0);
    for (int i = 0; i < n; ++i) {
      if (i + 1 < n) scores(i + 1);
      const int h = 2 * i + 1, st = h % R;
      // (what comes last, most often, is waited for last: bytes of 4-bit rows, else the weights)
      if constexpr (!C::kInt4) go = go && warp_wait(bar_full(st), (h / R) & 1, abort_flag, a.status);
      go = go && warp_wait(bar_p(i & 1), (i >> 1) & 1, abort_flag, a.status);
      const int vat = i % C::kVBytes;
      if constexpr (C::kInt4) go = go && warp_wait(bar_c(1, vat), (i / C::kVBytes) & 1, abort_flag, a.status);
      tc_fence_after();
      const uint32_t va = same_in_warp(desc_lo(C::kInt4 ? sb + C::kConvAt + (2 + vat) * C::kTile
                                                        : sb + C::kRingAt + st * C::kHalf, 128 * C::kBlk));
      const uint32_t pa = same_in_warp(desc_lo(sb + C::kPAt + (i & 1) * C::kP, 128));
      const uint32_t d = same_in_warp(tmem + C::kTmO + (i & 1) * 32);
      if (go && elect_one()) {
#pragma unroll
        for (int x = 0; x < kKeys / C::kKeyStep; ++x)
          mma<C::kCodes>(d, va + ((x * C::kKeyStep * C::kBlk) >> 4), kHiK, pa + x * C::kKeyStep, kHiP, kIdO, x > 0);
        umma_commit(C::kInt4 ? bar_c_free(1, vat) : bar_empty(st));
        if constexpr (C::kCodes) umma_commit(bar_word_free(i % W));
        umma_commit(bar_o(i & 1));
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(bar_done);
    __syncwarp();
    last_wait(bar_done, 0);
  } else if (n > 0 && C::kInt4 && warp >= 6) {
    // -------------------------------------------- 4-bit codes to bytes
    const int kv = warp - 6;
    int unit_no = 0;
    constexpr int kPieces = HD / 32, kEach = 128 * kPieces / 32;  // 16-byte pieces of a row, of a lane
    constexpr int kStep = 32 / kPieces;
    const int r0 = lane / kPieces, c0 = lane % kPieces, mix = C::kBlk == 128 ? r0 & 7 : (r0 >> 1) & 3;
    for (int i = 0; i < n; ++i) {
      if (!kv && (i == 0 || w.t == 0)) make_q(w.s, w.kvh, w.part, unit_no++);
      const bool hides = kv && w.hides();
      const int lo = w.cur.lo - w.key0(), hi = w.cur.hi - w.key0();
      if (i + 1 < n) w.next(a, units);
      const int h = 2 * i + kv, st = h % R;
      warp_wait(bar_full(st), (h / R) & 1, abort_flag, a.status);
      const int places = kv ? C::kVBytes : 2, use = i / places, at = i % places;
      if (use > 0) warp_wait(bar_c_free(kv, at), (use - 1) & 1, abort_flag, a.status);
      const uint32_t src = sb + C::kRingAt + st * C::kHalf + lane * 16;
      const uint32_t dst = sb + C::kConvAt + (2 * kv + at) * C::kTile;
      // piece lane + 32 k: row r0 + kStep k, and the swizzle repeats every eight rows
      const uint32_t d0 = dst + r0 * C::kBlk + (((2 * c0) ^ mix) << 4);
      const uint32_t d1 = dst + r0 * C::kBlk + (((2 * c0 + 1) ^ mix) << 4);
      constexpr uint32_t m = 0x0f0f0f0fu;
      constexpr int kFlight = kEach < 8 ? kEach : 8;
#pragma unroll
      for (int k0 = 0; k0 < kEach; k0 += kFlight) {
        uint4 x[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) x[k] = lds128(src + (k0 + k) * 512);
        if (hides) {
#pragma unroll
          for (int k = 0; k < kFlight; ++k) {
            const int r = r0 + kStep * (k0 + k);
            if (r < lo || r >= hi) x[k] = make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
          const uint32_t off = (k0 + k) * kStep * C::kBlk;
          st_shared_u4(d0 + off, x[k].x & m, x[k].y & m, x[k].z & m, x[k].w & m);
          st_shared_u4(d1 + off, (x[k].x >> 4) & m, (x[k].y >> 4) & m, (x[k].z >> 4) & m, (x[k].w >> 4) & m);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_c(kv, at));
        mbar_arrive(bar_empty(st));
      }
    }
  } else if (n > 0 && warp < 4) {
    // ---------------------------------------------------- softmax and O
    const int tid = threadIdx.x;
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;  // TMEM lane 32 warp
    const SoftCap cap = soft_cap(a.cap_log2);
    // Q's factors and sums stay in registers where there are enough
    constexpr bool kKeepQ = C::kCodes && GT <= 4;
    constexpr int kQm = kKeepQ ? GT : 1, kZ = C::kInt4 ? GT : 1;
    float acc[GT], l[GT], m[GT], zl[kZ], q_mul[kQm], q_sum[kQm];
    float fix_a[GT], fix_b[GT];  // of O two tiles ago, and one
    float lv0 = 0.f;  // exponent of the unit's first V scale here that is not 0
    bool find_lv0 = false;
    bool from_start = w.t == 0;  // the unit's first tile is this block's
    int of_unit = 0;             // tiles of the unit so far
    int unit_no = 0, flags = 0, end_s = 0, end_unit = 0;
    auto o_at = [&](int j) { return tmem + lanes + C::kTmO + (j & 1) * 32; };
    // O of a tile joins acc, which was kept against an older reference
    auto join_o = [&](float (&v)[C::kOCols], const float (&fix)[GT]) {
#pragma unroll
      for (int g = 0; g < GT; ++g) {
        float x;
        if constexpr (C::kCodes) x = v[g] + (v[GT + g] * 0.0625f + v[2 * GT + g] * 0.00390625f);
        else x = v[g] + v[GT + g];
        acc[g] = acc[g] * fix[g] + x;
      }
    };
    for (int i = 0; i < n; ++i) {
      const int key = w.key0() + tid;
      const bool hides = w.hides(), live = key >= w.cur.lo && key < w.cur.hi;
      const bool last = w.t + 1 == w.cur.tiles || i + 1 == n;
      uint32_t kw = 0, vw = 0;
      float x[GT];
      {
        const uint32_t qm = sb + C::kQMulAt + (unit_no & 3) * (2 * GT * 4);
        float v[C::kSCols], vo[C::kOCols];
        // S(i) was issued after the second product of tile i - 2, and its commit waits for that too
        warp_wait(bar_s(i & 1), (i >> 1) & 1, abort_flag, a.status);
        tc_fence_after();
        const uint32_t s_at = tmem + lanes + C::kTmS + (i & 1) * 16;
        if constexpr (C::kCodes) {
          const uint32_t at = sb + C::kWordsAt + (i % W) * 1024u;
          kw = lds32(at + tid * 4);
          vw = lds32(at + 512 + tid * 4);
          if (hides && !live) vw = 0u;  // (what is not seen may be a NaN)
          if constexpr (kKeepQ) {
            if (of_unit == 0) {
#pragma unroll
              for (int g = 0; g < GT; ++g) {
                q_mul[g] = __uint_as_float(lds32(qm + g * 4));
                q_sum[g] = __uint_as_float(lds32(qm + GT * 4 + g * 4));
              }
            }
          }
        }
        if (of_unit == 0) {
#pragma unroll
          for (int g = 0; g < GT; ++g) {
            acc[g] = l[g] = fix_b[g] = 0.f;
            m[g] = -3.402823466e38f;  // (finite: differences stay numbers)
            if constexpr (C::kInt4) zl[g] = 0.f;
          }
        }
        if constexpr (C::kCodes) {
          // As long as no scale was found the sums are of rows of zeros alone, and move with lv0: l is kept
          // against m - lv0, O is 0.
          if (of_unit == 0) {
            const int first = max(w.cur.lo - w.key0(), 0);
            const uint32_t e = lds32(sb + C::kWordsAt + (i % W) * 1024u + 512 + first * 4) >> 23 & 255u;
            find_lv0 = e - 1u >= 254u;
            lv0 = find_lv0 ? 0.f : small_float(e) - 127.f;
          }
          if (__builtin_expect(find_lv0, 0)) {
            const uint32_t e = first_exponent(sb + C::kWordsAt + (i % W) * 1024u + 512, w.cur.lo - w.key0(),
                                              w.cur.hi - w.key0());
            if (e) {
              find_lv0 = false;
              lv0 = small_float(e) - 127.f;
#pragma unroll
              for (int g = 0; g < GT; ++g) m[g] += lv0;
            }
          }
        }
        if constexpr (GT <= 4) {  // (without an O to take, what is there is read and left)
          tmem_read<C::kSCols, C::kOCols>(s_at, v, o_at(i), vo);
          if (of_unit >= 2) join_o(vo, fix_a);
        } else {
          if (of_unit >= 2) {
            tmem_read<C::kOCols>(o_at(i), vo);
            join_o(vo, fix_a);
          }
          tmem_read<C::kSCols>(s_at, v);
        }
        if constexpr (C::kCodes) {
          const float ks = __uint_as_float(C::kInt4 ? kw & 0xffff0000u : kw);
          const float kz = small_float(kw & 15u);
#pragma unroll
          for (int g = 0; g < GT; ++g) {
            float y = v[g] + v[GT + g] * 0.0625f;
            const float mul = kKeepQ ? q_mul[g % kQm] : __uint_as_float(lds32(qm + g * 4));
            if constexpr (C::kInt4)
              y = y * 512.f - kz * (kKeepQ ? q_sum[g % kQm] : __uint_as_float(lds32(qm + GT * 4 + g * 4)));
            x[g] = y * (mul * ks);
          }
        } else {
#pragma unroll
          for (int g = 0; g < GT; ++g) x[g] = v[g] * a.scale_log2;
        }
      }
      if constexpr (CAP) {
#pragma unroll
        for (int g = 0; g < GT; ++g) x[g] = cap.wide() ? capped_wide(x[g], cap) : capped(x[g], cap);
      }
      // V's scale is vm 2^lv, 1 <= vm < 2: the exponent goes into the weight's, exactly; ps = 2^(lv0 - lv) 2^-7
      // leads back from 2^lv times a weight to the weight
      float lv = 0.f, vm = 1.f, ps = 1.f;
      if constexpr (C::kCodes) {
        const uint32_t ve = (vw >> 23) & 255u;
        lv = small_float(ve) - 127.f;
        ps = exp2_fast(lv0 - 7.f - lv);
        vm = __uint_as_float((vw & (C::kInt4 ? 0x807f0000u : 0x807fffffu)) | 0x3f800000u);
        if (ve - 1u >= 254u) {  // a row of zeros (as if of a far smaller scale), or not a number
          vm = ve == 0 ? 0.f : __uint_as_float(0x7fc00000u);
          lv = ve == 0 ? lv0 - 80.f : lv0;
          ps = ve == 0 ? 9.44473297e21f : 0.0078125f;  // 2^73, 2^-7
        }
      }
      const uint32_t xch = sb + C::kXchAt + (i & 1) * (GT * 16);
      float mine = 0.f;  // lane g: the warp's largest of head g
#pragma unroll
      for (int g = 0; g < GT; ++g) {
        if (hides && !live) x[g] = -INFINITY;
        if constexpr (C::kCodes) x[g] += lv;
        const float t = warp_top(x[g]);
        if (lane == g) mine = t;
      }
      if (lane < GT) sts32(xch + lane * 16 + warp * 4, __float_as_uint(mine));
      named_bar_sync(1, 128);
      float wt[GT];
#pragma unroll
      for (int g = 0; g < GT; ++g) {
        const float4 t = ld_shared_f4(xch + g * 16);
        const float top = max3(max3(m[g], t.x, t.y), t.z, t.w);
        fix_a[g] = fix_b[g];
        fix_b[g] = exp2_fast(m[g] - top);
        m[g] = top;
        wt[g] = exp2_fast(x[g] - (C::kCodes ? top - 7.f : top));
        l[g] = l[g] * fix_b[g] + (C::kCodes ? wt[g] * ps : wt[g]);
        if constexpr (C::kCodes) wt[g] *= vm;
      }
      // the pieces of the weights, this key's row of P
      const uint32_t pd = sb + C::kPAt + (i & 1) * C::kP + tid * 16;
      if constexpr (!C::kCodes) {
        uint32_t hi[GT / 2], lo[GT / 2];
#pragma unroll
        for (int g = 0; g < GT; g += 2) {
          hi[g / 2] = pack_bf16x2(wt[g], wt[g + 1]);
          lo[g / 2] = pack_bf16x2(wt[g] - __uint_as_float(hi[g / 2] << 16),
                                  wt[g + 1] - __uint_as_float(hi[g / 2] & 0xffff0000u));
        }
        if constexpr (GT == 8) {
          st_shared_u4(pd, hi[0], hi[1], hi[2], hi[3]);
          st_shared_u4(pd + 2048, lo[0], lo[1], lo[2], lo[3]);
        } else {
          st_shared_u4(pd, hi[0], hi[1], lo[0], lo[1]);
        }
        // a row that is not seen may hold anything
        if (hides) {
          const int h = 2 * i + 1, st = h % R;
          warp_wait(bar_full(st), (h / R) & 1, abort_flag, a.status);
        }
      } else {
        uint32_t piece[3][GT / 4] = {};
#pragma unroll
        for (int g = 0; g < GT; g += 2) {
          const int at = 16 * ((g >> 1) & 1);
          // fp16 first (2^-11 of a weight), whose 11 bits the pieces hold; all exact from there
          const __half2 h = __floats2half2_rn(wt[g], wt[g + 1]), up = __float2half2_rn(16.f);
          const uint32_t c1 = to_e4m3x2(h);
          const __half2 r1 = __hmul2(__hsub2(h, from_e4m3x2(c1)), up);
          const uint32_t c2 = to_e4m3x2(r1);
          const uint32_t c3 = to_e4m3x2(__hmul2(__hsub2(r1, from_e4m3x2(c2)), up));
          piece[0][g / 4] |= c1 << at;
          piece[1][g / 4] |= c2 << at;
          piece[2][g / 4] |= c3 << at;
          if constexpr (C::kInt4) {
            const float2 p = __half22float2(h);
            const float vz = small_float(vw & 15u);
            zl[g] = zl[g] * fix_b[g] + vz * p.x;
            zl[g + 1] = zl[g + 1] * fix_b[g + 1] + vz * p.y;
          }
        }
        if constexpr (GT == 8) {
          st_shared_u4(pd, piece[0][0], piece[0][1], piece[1][0], piece[1][1]);
          st_shared_u4(pd + 2048, piece[2][0], piece[2][1], 0u, 0u);
        } else {
          st_shared_u4(pd, piece[0][0], piece[1][0], piece[2][0], 0u);
        }
        if (!C::kInt4 && hides) {
          const int h = 2 * i + 1, st = h % R;
          warp_wait(bar_full(st), (h / R) & 1, abort_flag, a.status);
        }
      }
      if (!C::kInt4 && hides && !live) {
        const uint32_t row = sb + C::kRingAt + ((2 * i + 1) % R) * C::kHalf + tid * C::kBlk;
#pragma unroll
        for (int x = 0; x < C::kBlks; ++x)
#pragma unroll
          for (int c = 0; c < C::kBlk; c += 16)  // (neighbours in unlike banks)
            st_shared_u4(row + x * 128 * C::kBlk + ((c + (C::kBlk == 128 ? 16 * tid : 8 * tid)) & (C::kBlk - 16)), 0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p(i & 1));
      ++of_unit;
      if (last) {
        // ---------------------------------------------- the unit's rows
        float v[GT];
#pragma unroll
        for (int g = 0; g < GT; ++g) v[g] = l[g];
        const uint32_t sum_at = sb + C::kSumAt + (unit_no & 1) * (2 * GT * 16);
        float sum = warp_sums<GT>(v);
        if (lane < GT) sts32(sum_at + lane * 16 + warp * 4, __float_as_uint(sum));
        if constexpr (C::kInt4) {
          sum = warp_sums<GT>(zl);
          if (lane < GT) sts32(sum_at + (GT + lane) * 16 + warp * 4, __float_as_uint(sum));
        }
        named_bar_sync(1, 128);
        // while the products end: what the sums are good for
        float scale[GT], shift[kZ];
        const float unit = C::kCodes ? exp2_fast((lv0 - 7.f) * 0.5f) : 1.f;  // (its square may be out of range)
        const bool to_end = w.t + 1 == w.cur.tiles, whole = from_start && to_end;
#pragma unroll
        for (int g = 0; g < GT; ++g) {
          const float4 t = ld_shared_f4(sum_at + g * 16);
          l[g] = (t.x + t.y) + (t.z + t.w);
          // (a part whose scores are all -infinity counts for nothing in the join, but its 0 / 0 would)
          scale[g] = l[g] == 0.f && !whole ? 0.f : unit * __frcp_rn(l[g]);
          if constexpr (C::kInt4) {
            const float4 z = ld_shared_f4(sum_at + (GT + g) * 16);
            shift[g] = (z.x + z.y) + (z.z + z.w);
          }
        }
        auto take = [&](int j, const float (&fix)[GT]) {
          warp_wait(bar_o(j & 1), (j >> 1) & 1, abort_flag, a.status);
          tc_fence_after();
          float vo[C::kOCols];
          tmem_read<C::kOCols>(o_at(j), vo);
          join_o(vo, fix);
        };
        if (of_unit > 1) take(i - 1, fix_a);
        take(i, fix_b);
        tc_fence_before();
        of_unit = 0;
        const int kvh = w.kvh, head0 = w.part * a.chunk;
        const int heads = min(a.chunk, a.group - head0);
        // lane -> channel: 64 rows of O lie in the first 16 lanes of each warp
        const bool has = HD == 128 || lane < 16;
        const int pos = HD == 128 ? tid : 16 * warp + lane;
        const int ch = C::kInt4 ? (pos & ~31) + 2 * (pos & 15) + ((pos >> 4) & 1) : pos;
        const int slot = 2 * static_cast<int>(blockIdx.x) + (from_start ? 1 : 0);
        uint16_t* out = a.o + w.s * a.o_stride + static_cast<int64_t>(kvh * a.group + head0) * HD + ch;
#pragma unroll
        for (int g = 0; g < GT; ++g) {
          float x = acc[g];
          if constexpr (C::kInt4) x = x * 512.f - shift[g];
          x = x * scale[g] * unit;
          if (g < heads && has) {
            if (a.cluster > 1) {
              // (over the stages: everything that was copied has been used)
              sts32(sb + (g * HD + ch) * 4, __float_as_uint(x));
              if (tid == 0)
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sb + kMaxHeads * HD * 4 + g * 8),
                             "f"(m[g] - lv0), "f"(l[g])
                             : "memory");
            } else if (whole) {
              out[g * HD] = f32_to_bf16(x);
            } else {
              a.part[(static_cast<int64_t>(slot) * kMaxHeads + g) * HD + ch] = x;
              if (tid == 0) a.ml[slot * kMaxHeads + g] = make_float2(m[g] - lv0, l[g]);
            }
          }
        }
        if (!from_start) {
          flags |= kHasEnd | (to_end ? kEndsUnit : 0);
          end_s = w.s;
          end_unit = w.unit;
        } else if (!to_end) {
          flags |= kHasStart;
        }
        ++unit_no;  // (the sums' place is used again two units and a barrier later)
        from_start = true;
      }
      if (i + 1 < n) w.next(a, units);
    }
    if (a.cluster <= 1 && tid == 0) a.desc[blockIdx.x] = make_int4(flags, end_s, end_unit, 0);
  }
  if (n == 0) {
    if (a.cluster <= 1) {
      if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    } else if (threadIdx.x < GT) {  // nothing to add
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sb + kMaxHeads * HD * 4 + threadIdx.x * 8),
                   "f"(-INFINITY), "f"(0.f)
                   : "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) tmem_dealloc(tmem, C::kTmemCols);
  if (a.cluster > 1) {
    // The unit's parts, joined in the order of the blocks, each of which takes a piece of the row.
    cluster_sync();
    const int kvh = w.kvh, head0 = w.part * a.chunk;
    const int all = min(a.chunk, a.group - head0) * HD, per = (all + a.cluster - 1) / a.cluster;
    const int parts = min(a.cluster, unit_tiles);  // (those behind have no tiles)
    for (int k = threadIdx.x; k < per && parts > 0; k += C::kThreads) {
      const int at = static_cast<int>(rank) * per + k, g = at / HD;
      if (at >= all) break;
      float2 ml[kMaxCluster];
      float v[kMaxCluster], top = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        const uint32_t part = mapa_shared(sb, min(i, parts - 1));
        ml[i] = ld_cluster_f2(part + kMaxHeads * HD * 4 + g * 8);
        v[i] = ld_cluster(part + at * 4);
      }
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) top = fmaxf(top, ml[i].x);
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        const float wt = i < parts ? ml[i].y * exp2_fast(ml[i].x - top) : 0.f;
        l += wt;
        o += i < parts ? wt * v[i] : 0.f;
      }
      a.o[w.s * a.o_stride + static_cast<int64_t>(kvh * a.group + head0) * HD + at] = f32_to_bf16(o / l);
    }
    // until all have read this block's part
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
}

// Joins the units that blocks share: block x looks after the one whose last part is block x's
// of the attention.  Its parts are those of a row of blocks, the first of which starts the unit.
// A warp takes 32 channels of a head, each quarter of its lanes every fourth part, kFlight at a time;
// the order is fixed, so that the same call gives the same bits.  No shared memory, which the attention's blocks
// leave none of.  Bound by latency: descriptors, parts, sums; 2.7 us beside the attention's end, 4.1
// for units of 38 parts.
template <int HD>
__global__ void __launch_bounds__(1024) pages_join_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kSlices = HD / 32, kFlight = 4;
  const int last = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = warp / kSlices, ch = (warp % kSlices) * 32 + (lane & 7) * 4, sub = lane >> 3;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int4 d = a.desc[last];
  int first = last;  // the nearest block before that starts a unit
  for (int b0 = last - 1; b0 >= 0; b0 -= 32) {
    const unsigned hit = __ballot_sync(0xffffffffu, b0 - lane >= 0 && (a.desc[max(b0 - lane, 0)].x & kHasStart));
    if (hit) {
      first = b0 - (__ffs(hit) - 1);
      break;
    }
    if ((d.x & (kHasEnd | kEndsUnit)) != (kHasEnd | kEndsUnit)) return;
  }
  if ((d.x & (kHasEnd | kEndsUnit)) != (kHasEnd | kEndsUnit)) return;
  const int kvh = d.z / a.n_chunks, head0 = (d.z - kvh * a.n_chunks) * a.chunk;
  if (g >= min(a.chunk, a.group - head0)) return;
  const int n = last - first + 1;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  auto add = [&](float4 v, float wt) {
    l += wt;
    o.x += wt * v.x, o.y += wt * v.y, o.z += wt * v.z, o.w += wt * v.w;
  };
  auto move = [&](float top) {  // to a reference above all so far
    const float fix = top == -INFINITY ? 1.f : exp2_fast(m - top);
    m = top;
    l *= fix;
    o.x *= fix, o.y *= fix, o.z *= fix, o.w *= fix;
  };
  for (int i0 = 0; i0 < n; i0 += 4 * kFlight) {
    float2 ml[kFlight];
    float4 v[kFlight];
    float top = m;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int i = min(i0 + 4 * k + sub, n - 1);
      const int at = (2 * (first + i) + (i == 0 ? 1 : 0)) * kMaxHeads + g;
      ml[k] = a.ml[at];
      v[k] = *reinterpret_cast<const float4*>(a.part + static_cast<int64_t>(at) * HD + ch);
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) top = fmaxf(top, ml[k].x);
    move(top);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (i0 + 4 * k + sub < n) add(v[k], ml[k].y * exp2_fast(ml[k].x - ref));
  }
#pragma unroll
  for (int x = 8; x < 32; x <<= 1) {
    const float top = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    move(top);
    l += __shfl_xor_sync(0xffffffffu, l, x);
    o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, x);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, x);
  }
  if (sub == 0) {
    uint16_t* out = a.o + d.y * a.o_stride + static_cast<int64_t>(kvh * a.group + head0 + g) * HD + ch;
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(o.x / l, o.y / l), pack_bf16x2(o.z / l, o.w / l));
  }
}

// ------------------------------------------------------------ host side

// Units of at most eight heads, as even as they come.
struct Groups {
  int chunk, n_chunks;
};
Groups head_groups(int group) {
  const int n = (group + kMaxHeads - 1) / kMaxHeads;
  const int chunk = (group + n - 1) / n;
  return Groups{chunk, (group + chunk - 1) / chunk};
}

// Blocks of a cluster that share a unit, 1 if the units are cut into equal shares over all
// blocks instead.  A cluster needs no second kernel and no search; but it cuts every
// sequence into as many pieces, so the longest one decides, and blocks stay idle that no whole
// cluster fills.  The host does not know the lengths: `tiles` are those of the longest sequence that the table, or
// the window, has room for, and a short sequence in a wide table is cut into shares (one of 1024 / 2048 rows, 24/8 x
// 128, in a table of as many rows and of 32768: bf16 5.4 and 7.4 / 6.7 and 7.6 us, e4m3 5.7 and 7.6 / 6.7 and 8.1, 4
// bits 6.0 and 8.4 / 7.3 and 9.0).  So clusters serve up to one tile a block of bf16 rows and two of codes, whose
// tiles wait more for each other and less for HBM, and twice as many where they take a quarter of the
// places or less, so that hardly two blocks share an SM.  24/8 x 128, us by clusters / by shares, bf16:
// one sequence of 1024 rows 5.4 / 7.4, of 2048 7.0 / 7.7, of 4096 9.9 / 8.8; two of 2048 9.7 / 8.2; eight of 512
// 7.6 / 8.5; e4m3: one of 4096 8.7 / 9.1, of 8192 13.6 / 11.1; two of 4096 13.2 / 9.7; eight of 1024 9.1 / 9.3.
int unit_cluster(int64_t units, int64_t tiles, int blocks, bool codes) {
  int c = 1;
  while (c < kMaxCluster && c < tiles && units * c * 2 <= blocks) c *= 2;
  const int each = (codes ? 2 : 1) * (units * c * 4 <= blocks ? 2 : 1);
  if (tiles > static_cast<int64_t>(each) * c) c = 1;
  return c;
}

size_t desc_bytes(int blocks) { return static_cast<size_t>(blocks) * sizeof(int4); }
size_t ml_bytes(int blocks) { return static_cast<size_t>(blocks) * 2 * kMaxHeads * sizeof(float2); }

template <int FMT, int HD, int GT, bool CAP>
cudaError_t launch(PagedArgs a, const CUtensorMap& mk, const CUtensorMap& mv, int blocks,
                   cudaStream_t st) {
  using C = Cfg<FMT, HD, GT>;
  const auto kernel = pages_attn_kernel<FMT, HD, GT, CAP>;
  cudaError_t ce = kernel_smem_attr(reinterpret_cast<const void*>(kernel), static_cast<int>(C::kSmem));
  if (ce != cudaSuccess) return ce;
  if (a.cluster > 1) {  // as large a one as the GPU has room for all of
    const void* fn = reinterpret_cast<const void*>(kernel);
    const int units = a.p.n_seqs * a.p.n_kv_heads * a.n_chunks;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    while (a.cluster > 1 && kernel_max_clusters(fn, cfg, a.cluster) < units) a.cluster /= 2;
    if (a.cluster > 1)
      return launch_after_cluster(kernel, dim3(units * a.cluster), C::kThreads, C::kSmem, a.cluster, st, a, mk, mv);
  }
  ce = launch_after(kernel, dim3(blocks), C::kThreads, C::kSmem, st, a, mk, mv);
  if (ce != cudaSuccess) return ce;
  return launch_after(pages_join_kernel<HD>, dim3(blocks), a.chunk * HD, 0, st, a);
}
template <int FMT, int HD>
cudaError_t launch_groups(const PagedArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int blocks,
                          cudaStream_t st) {
  const bool cap = a.cap_log2 > 0.f;
  if (a.chunk <= 4)
    return cap ? launch<FMT, HD, 4, true>(a, mk, mv, blocks, st) : launch<FMT, HD, 4, false>(a, mk, mv, blocks, st);
  return cap ? launch<FMT, HD, 8, true>(a, mk, mv, blocks, st) : launch<FMT, HD, 8, false>(a, mk, mv, blocks, st);
}

}  // namespace

size_t pages_attention_ws_bytes(int hd, int num_sms) {
  const int blocks = kBlocksPerSm * num_sms;
  return desc_bytes(blocks) + ml_bytes(blocks) + static_cast<size_t>(blocks) * 2 * kMaxHeads * hd * 4;
}

pds_status pages_attention(const PagesAttnCall& c, cudaStream_t st, std::string* err) {
  const PageView& p = c.pages;
  const int hd = c.head_dim, blocks = kBlocksPerSm * c.num_sms;
  PagedArgs a{};
  a.p = p;
  a.new_rows = c.new_rows;
  a.q = c.q;
  a.o = c.o;
  a.q_stride = c.q_stride;
  a.o_stride = c.o_stride;
  a.n_heads = c.n_heads;
  a.group = c.n_heads / p.n_kv_heads;
  const Groups gr = head_groups(a.group);
  a.chunk = gr.chunk;
  a.n_chunks = gr.n_chunks;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(hd));
  a.cap_log2 = c.softcap * 1.4426950408889634f;
  a.window = c.window;
  a.whole_pages = p.row_stride == (c.format == PDS_KV_INT4 ? hd / 2 : c.format == PDS_KV_E4M3 ? hd : 2 * hd);
  a.status = c.status;
  a.desc = reinterpret_cast<int4*>(c.ws);
  a.ml = reinterpret_cast<float2*>(c.ws + desc_bytes(blocks));
  a.part = reinterpret_cast<float*>(c.ws + desc_bytes(blocks) + ml_bytes(blocks));
  // tiles are counted in 32 bits
  const int64_t most = static_cast<int64_t>(p.max_pages) << p.page_shift;
  if (static_cast<double>(p.n_seqs) * p.n_kv_heads * a.n_chunks * static_cast<double>(most / kKeys + 2) > 2.0e9) {
    *err = "declined: pds_pages_attend: sequences x kv heads x rows are too many";
    return PDS_DECLINED;
  }
  a.cluster = unit_cluster(static_cast<int64_t>(p.n_seqs) * p.n_kv_heads * a.n_chunks,
                           (c.window > 0 ? std::min<int64_t>(most, c.window) + kKeys - 2 : most - 1) / kKeys + 1,
                           blocks, c.format != PDS_KV_BF16);
  CUtensorMap maps[2];
  const bool bf16 = c.format == PDS_KV_BF16;
  const int channels = c.format == PDS_KV_INT4 ? hd / 2 : hd;  // elements of a row
  const uint32_t box_rows = static_cast<uint32_t>(std::min(1 << p.page_shift, kKeys));
  const uint32_t row_bytes = static_cast<uint32_t>(bf16 ? 2 * channels : channels);
  const CUtensorMapSwizzle swizzle = c.format == PDS_KV_INT4 ? CU_TENSOR_MAP_SWIZZLE_NONE
                                     : row_bytes >= 128      ? CU_TENSOR_MAP_SWIZZLE_128B
                                                             : CU_TENSOR_MAP_SWIZZLE_64B;
  for (int i = 0; i < 2; ++i) {
    const pds_status rc = tc_map_pages(&maps[i], i ? p.v : p.k, bf16, static_cast<uint64_t>(channels),
                                       1ull << p.page_shift, static_cast<uint64_t>(p.n_kv_heads),
                                       static_cast<uint64_t>(p.n_pages), static_cast<uint64_t>(p.row_stride),
                                       static_cast<uint64_t>(p.head_stride), static_cast<uint64_t>(p.page_stride),
                                       std::min(row_bytes, 128u) / (bf16 ? 2u : 1u), box_rows, swizzle, err);
    if (rc != PDS_OK) return rc;
  }
  auto by_width = [&](auto fmt) {
    return hd == 128 ? launch_groups<fmt, 128>(a, maps[0], maps[1], blocks, st)
                     : launch_groups<fmt, 64>(a, maps[0], maps[1], blocks, st);
  };
  const cudaError_t ce = bf16 ? by_width(std::integral_constant<int, PDS_KV_BF16>{})
                         : c.format == PDS_KV_E4M3 ? by_width(std::integral_constant<int, PDS_KV_E4M3>{})
                                                   : by_width(std::integral_constant<int, PDS_KV_INT4>{});
  if (ce != cudaSuccess) {
    *err = std::string("paged attention launch: ") + cudaGetErrorString(ce);
    return PDS_ELAUNCH;
  }
  return PDS_OK;
}

}  // namespace pds
