// What the attention kernels over a cache share: the call's arguments, the
// schedule that cuts the sequences into chunks, asynchronous copies, and the
// conversion of cached codes.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "kv.h"

namespace pds {
namespace cacheattn {

constexpr int kMaskWords = kMaxDraftTokens / 32;

struct Args {
  CacheView c;
  const uint16_t* q;
  uint16_t* o;
  int64_t q_stride, o_stride;
  const int32_t* parents;
  int n_tokens, n_heads, group;  // group: query heads per kv head
  float per_group;               // 1 / group
  int max_len;
  float scale_log2;              // log2(e) / sqrt(hd)
  float cap;                     // softcap in units of q.k (0: none)
  int window;
  int step_shift;                // log2 of the keys of a step
  int row_tiles;                 // blocks of query rows per (sequence, kv head)
  int tile_rows;                 // rows of one
  int slots;                     // blocks to spread the chunks over, more than n_kv_heads x
                                 // row_tiles; 0: one chunk each
  int fit;                       // 1: choose chunks so that all units run at once; 0: there are
                                 // more sequences than that
  float per_chunk;               // n_seqs == 1: 1 / (chunks that fit the slots)
  int min_steps;                 // shortest chunk, in steps
  int cluster;                   // > 1: every sequence in this many chunks, one cluster's blocks
  float* o_part;                 // [unit][tile_rows][hd], each kernel in its own order
  float2* ml_part;               // [unit][tile_rows]: (maximum, sum)
  uint32_t* status;
};

// --------------------------------------------------------------- schedule
//
// Units: (chunk of a sequence) x (kv head, row tile), the latter fastest, so
// that blocks running together read neighbouring heads of the same rows.

// Steps of sequence s: [first, first + n) in units of 2^step_shift keys; n = 0 for a
// length that does not fit.
__device__ __forceinline__ int seq_steps(const Args& a, int s, int& first, int& len) {
  len = a.c.lens[s];
  first = 0;
  if (len < 0 || len > a.max_len) return 0;
  // the first row any token can see: a root's, at position len
  if (a.window > 0 && len - a.window + 1 > 0) first = (len - a.window + 1) >> a.step_shift;
  return ((len + a.n_tokens - 1) >> a.step_shift) + 1 - first;
}

// Token of query row R = t group + i: R is below 2^21 (256 tokens, 8192 heads), so
// the rounded product is off by less than half of 1 / group.
__device__ __forceinline__ int token_of(const Args& a, int R) {
  return static_cast<int>((static_cast<float>(R) + 0.5f) * a.per_group);
}

__device__ __forceinline__ unsigned warp_sum_uint(unsigned v) {
  return __reduce_add_sync(0xffffffffu, v);
}

// One warp's view of the schedule: lane i holds sequence i's steps (the first
// 32 sequences; further ones are read again, from L1, where they are needed).
struct Lane {
  int n, first, len;
};
__device__ __forceinline__ Lane lane_steps(const Args& a, int s) {
  Lane l{0, 0, 0};
  if (s < a.c.n_seqs) l.n = seq_steps(a, s, l.first, l.len);
  return l;
}

// Steps per chunk (the same for every sequence) where all units run at once, by
// one warp.
__device__ __forceinline__ int chunk_steps(const Args& a, int lane, const Lane& mine) {
  const int per = a.c.n_kv_heads * a.row_tiles;
  float total = static_cast<float>(mine.n);
#pragma unroll 1
  for (int s = lane + 32; s < a.c.n_seqs; s += 32) total += static_cast<float>(lane_steps(a, s).n);
  total = warp_sum(total);
  int c = max(a.min_steps, static_cast<int>(__fdividef(total * per, static_cast<float>(a.slots))));
  // Sequences' last chunks are short: lengthen until the units fit the slots.
  // Each lane counts the chunks (to within the rounding of a quotient) for a length
  // of its own, in steps of a thirty-second.
  const unsigned most = static_cast<unsigned>(a.slots / per);
  if (a.c.n_seqs <= 32) {
    const int mine_c = c + max(1, c >> 5) * lane;
    const float per_c = __fdividef(1.0f, static_cast<float>(mine_c));
    unsigned chunks = 0;
#pragma unroll 4
    for (int s = 0; s < a.c.n_seqs; ++s)
      chunks += static_cast<unsigned>(
          ceilf(static_cast<float>(__shfl_sync(0xffffffffu, mine.n, s)) * per_c));
    const unsigned fits = __ballot_sync(0xffffffffu, chunks <= most);
    c = __shfl_sync(0xffffffffu, mine_c, fits ? __ffs(fits) - 1 : 31);
  }
  // Then exactly.  One chunk per sequence always fits; the length grows by a
  // sixteenth a round, and past the longest sequence there is nothing left to grow
  // for.  (From the start so, some five rounds of divisions took a microsecond.)
#pragma unroll 1
  for (;;) {
    unsigned chunks = static_cast<unsigned>(mine.n + c - 1) / static_cast<unsigned>(c);
#pragma unroll 1
    for (int s = lane + 32; s < a.c.n_seqs; s += 32) chunks += (lane_steps(a, s).n + c - 1) / c;
    if (warp_sum_uint(chunks) <= most) return c;
    c += max(1, c >> 4);
  }
}

struct Unit {
  int seq, chunk, n_chunks, first, n_steps, len;  // steps [first, first + n_steps)
  int base, more;  // among all chunks: the sequence's first is `base`, its k-th more + k
};

// One sequence: its chunks by a few instructions, in every thread.
__device__ __forceinline__ bool only_unit(const Args& a, int w, Unit& u) {
  int first, len;
  const int n = seq_steps(a, 0, first, len);
  const int most = a.slots / (a.c.n_kv_heads * a.row_tiles);
  int c = static_cast<int>(static_cast<float>(n) * a.per_chunk) + 1;
  if (static_cast<long long>(c) * most < n) ++c;  // (the quotient was rounded)
  c = max(c, a.min_steps);
  u.seq = 0;
  u.len = len;
  u.base = u.more = 0;
  u.n_chunks = n == 0 ? 0 : static_cast<int>(static_cast<unsigned>(n - 1) / static_cast<unsigned>(c)) + 1;
  u.chunk = max(w, 0);
  u.first = first + u.chunk * c;
  u.n_steps = min(c, n - u.chunk * c);
  return u.chunk < u.n_chunks;
}

// Uncut sequences (slots == 0): the w-th is unit w, whether its length fits or not.
// (By a search like the one below 1024 sequences of 200 e4m3 rows, 8/2 heads, took
// 86 us instead of 39.)
__device__ __forceinline__ bool whole_unit(const Args& a, int w, Unit& u) {
  u.seq = w;
  u.n_steps = seq_steps(a, w, u.first, u.len);
  u.n_chunks = u.n_steps > 0;
  return u.n_chunks != 0;
}

// The sequence and chunk of the w-th chunk overall (w < 0: of sequence `seq`,
// whole range).  False past the last one.  By one warp; every lane returns it.
__device__ __forceinline__ bool find_unit(const Args& a, int c, int w, int seq, int lane,
                                          const Lane& mine, Unit& u) {
  int base = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < a.c.n_seqs; s0 += 32) {
    const Lane l = s0 == 0 ? mine : lane_steps(a, s0 + lane);
    const int chunks = l.n == 0 ? 0 : (l.n - 1) / c + 1;
    int incl = chunks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const int excl = base + incl - chunks;
    const bool here = w >= 0 ? (w >= excl && w < base + incl) : s0 + lane == seq;
    const unsigned hit = __ballot_sync(0xffffffffu, here);
    if (hit) {
      const int src = __ffs(hit) - 1;
      u.seq = s0 + src;
      u.n_chunks = __shfl_sync(0xffffffffu, chunks, src);
      u.base = u.more = __shfl_sync(0xffffffffu, excl, src);
      u.len = __shfl_sync(0xffffffffu, l.len, src);
      const int f = __shfl_sync(0xffffffffu, l.first, src), m = __shfl_sync(0xffffffffu, l.n, src);
      u.chunk = w >= 0 ? w - u.base : 0;
      u.first = f + u.chunk * c;
      u.n_steps = min(c, m - u.chunk * c);
      return true;
    }
    base = __shfl_sync(0xffffffffu, base + incl, 31);
  }
  return false;
}

// More sequences than run at once: only those longer than an average block's
// share are cut, at the share.  The sequences' first chunks come first among the
// units, found without a search (only the lengths are summed); the others, of
// which there are never more than fit the slots, follow.  One token of 256
// sequences of 1000 e4m3 rows, 32/8 heads, takes 96 us (5.6 TB/s); with a search
// over all sequences in every block, the join's too, it took 136.
struct Share {
  int c;     // steps of a chunk
  bool any;  // whether any sequence is longer
};
constexpr int kShareScratch = 64 * 12;  // bytes of shared memory, 8-byte aligned
// By all threads of a block, with one barrier.
__device__ __forceinline__ Share block_share(const Args& a, void* scratch) {
  unsigned long long* sums = static_cast<unsigned long long*>(scratch);
  unsigned* longest = reinterpret_cast<unsigned*>(sums + 64);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  unsigned long long sum = 0;
  unsigned most = 0;
#pragma unroll 1
  for (int s = threadIdx.x; s < a.c.n_seqs; s += blockDim.x) {
    const unsigned n = static_cast<unsigned>(lane_steps(a, s).n);
    sum += n;
    most = max(most, n);
  }
  auto reduce = [&]() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = __reduce_max_sync(0xffffffffu, most);
  };
  reduce();
  if (lane == 0) {
    sums[warp] = sum;
    longest[warp] = most;
  }
  __syncthreads();
  sum = lane < warps ? sums[lane] : 0ull;
  most = lane < warps ? longest[lane] : 0u;
  reduce();
  // at most (slots + sequences x per) units: with c >= total per / slots (to within
  // 2^-22) the sum of floor((n - 1) / c) is at most slots / per
  const float share = __fdiv_rn(__fmul_rn(static_cast<float>(sum),
                                          static_cast<float>(a.c.n_kv_heads * a.row_tiles)),
                                static_cast<float>(a.slots));
  const int c = max(a.min_steps, static_cast<int>(fminf(share, 1073741824.f)) + 1);
  return Share{c, most > static_cast<unsigned>(c)};
}
// Chunk 0 of sequence w.
__device__ __forceinline__ bool first_unit(const Args& a, const Share& h, int w, Unit& u) {
  u.seq = w;
  const int n = seq_steps(a, w, u.first, u.len);
  u.n_chunks = n == 0 ? 0 : (n - 1) / h.c + 1;
  u.n_steps = min(n, h.c);
  return n != 0;
}
// The e-th of the chunks behind the first ones, by one warp.
__device__ __forceinline__ bool later_unit(const Args& a, const Share& h, int e, int lane, Unit& u) {
  if (!h.any) return false;
  int base = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < a.c.n_seqs; s0 += 32) {
    const Lane l = lane_steps(a, s0 + lane);
    const int chunks = l.n == 0 ? 0 : (l.n - 1) / h.c;
    int incl = chunks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const int excl = base + incl - chunks;
    const unsigned hit = __ballot_sync(0xffffffffu, e >= excl && e < excl + chunks);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int k = e - __shfl_sync(0xffffffffu, excl, src) + 1;
      const int f = __shfl_sync(0xffffffffu, l.first, src), n = __shfl_sync(0xffffffffu, l.n, src);
      u.seq = s0 + src;
      u.n_chunks = __shfl_sync(0xffffffffu, chunks, src) + 1;
      u.len = __shfl_sync(0xffffffffu, l.len, src);
      u.first = f + k * h.c;
      u.n_steps = min(h.c, n - k * h.c);
      return true;
    }
    base = __shfl_sync(0xffffffffu, base + incl, 31);
  }
  return false;
}
// Where the chunks of sequence `seq` are, by one warp.
__device__ __forceinline__ void chunks_of(const Args& a, const Share& h, int seq, int lane, Unit& u) {
  first_unit(a, h, seq, u);
  u.base = seq;
  u.more = 0;
  if (u.n_chunks <= 1) return;
  unsigned before = 0;
#pragma unroll 1
  for (int s = lane; s < seq; s += 32) {
    const int n = lane_steps(a, s).n;
    before += n == 0 ? 0 : (n - 1) / h.c;
  }
  u.more = a.c.n_seqs + static_cast<int>(warp_sum_uint(before)) - 1;
}

// ------------------------------------------------------------ instructions

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes (or zeros, when !live) into shared memory, not through L1.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c tanh(y / c) = c - 2 c / (2^(2 log2(e) y / c) + 1), scores and cap in powers of two.
// The difference is off by some 2^-22 c, which a small cap makes nothing (2^-15 in
// the exponent at 64) and a large one more than the scores: beyond that, where |y| is
// below c / 4, it is y (1 - u^2/3 + 2 u^4/15 - 17 u^6/315), u = y / c, the start of
// tanh's series, off by 2^-21 of y, and elsewhere c times a difference of 2^-1 and more.
struct SoftCap {
  float c, rate;
  __device__ __forceinline__ bool wide() const { return c > 64.f * 1.4426950408889634f; }
};
__device__ __forceinline__ SoftCap soft_cap(float c) {
  return SoftCap{c, fminf(2.0f * 1.4426950408889634f / c, 3.0e38f)};
}
__device__ __forceinline__ float capped(float y, const SoftCap& s) {
  return s.c - __fdividef(2.0f * s.c, exp2_fast(y * s.rate) + 1.0f);
}
__device__ __forceinline__ float capped_wide(float y, const SoftCap& s) {
  const float x = y * s.rate, u2 = x * x * (0.25f * 0.6931471805599453f * 0.6931471805599453f);
  const float near = y * (1.0f + u2 * (-1.0f / 3 + u2 * (2.0f / 15 - u2 * (17.0f / 315))));
  return u2 < 0.0625f ? near : s.c * (1.0f - __fdividef(2.0f, exp2_fast(x) + 1.0f));
}

// 8- and 4-bit rows go into the products as fp16, whose 11 bits hold every code
// exactly and round P eight times finer than bf16 would; the conversions are
// few and cheap (one instruction per pair of e4m3 codes, where spreading the
// bits to bf16 takes five, and the pipe that runs those was the busiest).
// fp16's range is narrow, so both other operands are brought into it by powers
// of two:
//  * Q: each row by one of its own, so that its largest value is 2^14 .. 2^15 and
//    what that rounds is below 2^-31 of it; a row's scale never depends on
//    another's, which may be a padding token's or as large as bf16 goes.  (The
//    tile kernel gives rows within 2^8 of the block's largest the block's one,
//    with the same bound, and multiplies the scores of the others.)
//  * P times V's scale: by one (the unit, from the largest V scale met so far) that
//    brings that scale to 2^6 .. 2^7, and by the row's reference, which follows the
//    row's largest product of a weight and a scale, not its largest weight: where the
//    scale of the key with the largest score is below the unit by more than 2^4 the
//    reference is lower by as much (level_shift).  So a row's largest product is 2^2
//    or more when it is taken, later ones are below 2^15, and what rounding to fp16's
//    smallest steps loses is below 2^-27 of the row's largest product per key, and below
//    2^-31 of the largest scale: keys that a row does not see, or hardly, take no
//    precision from it whatever their scales (up to 2^80 above; weights stay below 2^88,
//    their sums in float32).
__device__ __forceinline__ void e4m3_pairs(uint32_t r, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(r));
}
// Codes that stand for NaN (never stored by a write, but unwritten rows may hold
// anything) as the largest number instead: a zero weight then keeps them out.
__device__ __forceinline__ uint32_t e4m3_finite(uint32_t w) {
  const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return w ^ (nan >> 7);
}
// Two 4-bit codes in the low (lo) or high (hi) nibbles of the low bytes of
// 16-bit halves, less their zero points: 1024 + code and 1024 + 16 code are
// fp16 numbers, and so is every difference.  Zero points as int4_zero makes them.
__device__ __forceinline__ uint32_t int4_lo(uint32_t r, uint32_t zero) {
  const uint32_t bits = (r & 0x000f000fu) | 0x64006400u;
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(bits), "r"(zero));
  return d;
}
__device__ __forceinline__ uint32_t int4_hi(uint32_t r, uint32_t zero) {
  const uint32_t bits = (r & 0x00f000f0u) | 0x64006400u;
  // (1024 + 16 code) / 16 - (64 + z); 0xd400 + 16 z is -(64 + z)
  const uint32_t neg = ((zero & 0x000f000fu) << 4) | 0xd400d400u;
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(bits), "r"(0x2c002c00u), "r"(neg));
  return d;
}
// 1024 + zero point in both halves: of the keys with scale words a (low) and b.
__device__ __forceinline__ uint32_t int4_zero(uint32_t a, uint32_t b) {
  return 0x64006400u | (a & 15u) | (b & 15u) << 16;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Bits of |x| if it is finite, else 0 (they order as the values do).
__device__ __forceinline__ uint32_t finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// From the bits of the largest value of a row (or block) of Q: its exponent, and
// the power of two that brings it to 2^14 .. 2^15, with its inverse.
__device__ __forceinline__ uint32_t q_exponent(uint32_t max_bits) { return max(max_bits >> 23, 20u); }
__device__ __forceinline__ float q_multiplier(uint32_t e) { return __uint_as_float((268u - e) << 23); }
__device__ __forceinline__ float q_inverse(uint32_t e) { return __uint_as_float((e - 14u) << 23); }
// The block's exponent stays where its product with a scale of K cannot overflow.
__device__ __forceinline__ uint32_t q_block_exponent(uint32_t max_bits) {
  return min(max(q_exponent(max_bits), 127u - 40u), 127u + 40u);
}
__device__ __forceinline__ uint32_t q_row_exponent(uint32_t max_bits, uint32_t block) {
  const uint32_t e = max_bits ? q_exponent(max_bits) : block;
  return e <= block && block - e <= 8u ? block : e;
}
// V's unit, from the biased exponent of the largest scale: products of scales with the
// multiplier are below 2^7.  Larger scales than 2^60 do not raise it further, so that
// those of ordinary keys stay normal float32 numbers beside them.
constexpr uint32_t kMinScaleExp = 8, kMaxScaleExp = 127 + 60;
__device__ __forceinline__ float v_multiplier(uint32_t e) { return __uint_as_float((260u - e) << 23); }
__device__ __forceinline__ float v_inverse(uint32_t e) { return __uint_as_float((e - 6u) << 23); }
// What a key's score is moved by where its V scale (biased exponent e) is far from the unit.
__device__ __forceinline__ float level_shift(uint32_t e, uint32_t unit) {
  const int d = static_cast<int>(e) - static_cast<int>(unit);
  return static_cast<float>(d < -4 ? max(d + 4, -80) : max(d, 0));
}
// The unit grows by 2^d: a row's reference goes down by as much instead of its O, which
// keeps its bits, as far as its sum (at most `sum`) allows; O takes the rest.
__device__ __forceinline__ int unit_shift(int d, float sum) {
  return max(min(min(d, 90), 127 + 90 - static_cast<int>(__float_as_uint(sum) >> 23)), 0);
}

__device__ __forceinline__ bool not_finite2(uint32_t w) {  // either bf16 of a pair
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

}  // namespace cacheattn

// The tensor-core kernel and its join (attn_cache_tc.cu): a step is 64 keys,
// a.tile_rows 128 or 256 query rows per block, one block per SM.
cudaError_t launch_tile_attention(const cacheattn::Args& a, int format, int hd, int64_t grid,
                                  int num_sms, cudaStream_t st);

}  // namespace pds
