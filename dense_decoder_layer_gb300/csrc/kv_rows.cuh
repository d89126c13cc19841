// What the kernels that turn, store and fetch K/V rows share: a thread's 16
// channels of a head, rotations by position, and the formats of cached rows.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

#include "common.cuh"
#include "kv.h"

namespace pds {

struct Vec16 {  // 16 channels: channels a .. a+7 and b .. b+7 of the head
  float x[16];
};

__device__ __forceinline__ void widen8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 narrow8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// First channels (a, b) of the two vectors of unit u of a head.
__device__ __forceinline__ void unit_channels(int u, int rot_dim, int layout, int& a, int& b) {
  if (16 * u < rot_dim && layout == PDS_ROPE_NEOX) {
    a = 8 * u;
    b = rot_dim / 2 + 8 * u;
  } else {
    a = 16 * u;
    b = 16 * u + 8;
  }
}

// (cos, sin) * mscale of pair i at position pos.  The angle is a fixed-point
// fraction of a turn: position times a 64-bit fraction, modulo 2^64, is the
// exact remainder modulo whole turns, so no position loses accuracy and no
// 64-bit floating point is needed (its rate on this chip is a hundredth of
// float32's).  The nearest quarter turn comes off as an integer; what is left, at
// most an eighth, becomes an angle xh + xl (Dekker's products), and sine and
// cosine are their Taylor series with the rounding errors of the leading terms
// added to the small ones: off by little more than their own last rounding.
__device__ __forceinline__ float2 pair_turn(const RopeTurns& r, int i, int64_t pos) {
  const uint64_t turn = static_cast<uint64_t>(pos) * r.turns[i];
  const uint32_t quarter = static_cast<uint32_t>((turn + (1ull << 61)) >> 62) & 3u;
  const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
  const int32_t hi = static_cast<int32_t>(rest >> 32);  // below 2^29
  const float f = __int2float_rn(hi);
  const float low = static_cast<float>(hi - static_cast<int32_t>(f)) +
                    __uint2float_rn(static_cast<uint32_t>(rest)) * 2.3283064365386963e-10f;
  // 2 pi 2^-32 as the sum of two float32
  constexpr double kTurn = 6.283185307179586476925 / 4294967296.0;
  constexpr float kTurnHi = static_cast<float>(kTurn);
  constexpr float kTurnLo = static_cast<float>(kTurn - static_cast<double>(kTurnHi));
  const float xh = f * kTurnHi;
  const float xl = __fmaf_rn(f, kTurnHi, -xh) + (f * kTurnLo + low * kTurnHi);
  const float h = xh * xh, h_err = __fmaf_rn(xh, xh, -h);
  const float one = 1.0f - 0.5f * h, one_err = (1.0f - one) - 0.5f * h;
  const float odd = h * (-1.0f / 6 + h * (1.0f / 120 + h * (-1.0f / 5040 + h * (1.0f / 362880 -
                                                                                h * (1.0f / 39916800)))));
  const float even = h * h * (1.0f / 24 + h * (-1.0f / 720 + h * (1.0f / 40320 - h * (1.0f / 3628800))));
  const float s = xh + (xh * odd + xl * one);
  const float c = one + (one_err + (even - (0.5f * h_err + xl * xh)));
  const float cc = quarter & 1u ? s : c, ss = quarter & 1u ? c : s;
  const bool neg_c = quarter == 1u || quarter == 2u, neg_s = quarter >= 2u;
  return make_float2((neg_c ? -cc : cc) * r.mscale, (neg_s ? -ss : ss) * r.mscale * r.sign);
}
// Where pair i is in a table: the same pair of neighbouring units side by side, so
// that the lanes of a head read neighbouring banks (with the pairs in order 8192
// rows of 32 x 128 took 29.6 us instead of 24.6, four rows to a block).
__device__ __forceinline__ int turn_at(const RopeTurns& r, int i) {
  return (i & 7) * (r.rot_dim >> 4) + (i >> 3);
}
__device__ __forceinline__ void fill_table(float2* table, const RopeTurns& r, int64_t pos) {
  for (int i = threadIdx.x; i < r.rot_dim / 2; i += blockDim.x)
    table[turn_at(r, i)] = pair_turn(r, i, pos);
}

// Turn the pairs of unit u (table in shared memory); a unit past rot_dim stays.
__device__ __forceinline__ void rotate_unit(Vec16& v, int u, const RopeTurns& r,
                                            const float2* table) {
  if (16 * u >= r.rot_dim) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 cs = table[i * (r.rot_dim >> 4) + u];
    const bool neox = r.layout == PDS_ROPE_NEOX;
    const float p = neox ? v.x[i] : v.x[2 * i], q = neox ? v.x[8 + i] : v.x[2 * i + 1];
    const float y0 = p * cs.x - q * cs.y, y1 = p * cs.y + q * cs.x;
    // selects, not indexed stores: the layout is uniform, the registers fixed
    v.x[i] = neox ? y0 : v.x[i];
    v.x[8 + i] = neox ? y1 : v.x[8 + i];
    if (!neox) {
      v.x[2 * i] = y0;
      v.x[2 * i + 1] = y1;
    }
  }
}

// The larger, or a NaN if either is one.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
// Extremum over the LANES neighbouring lanes that hold one head.
template <int LANES>
__device__ __forceinline__ float head_max(float m) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = max_or_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Codes of four float32 on the e4m3 grid, nearest even, in channel order.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

constexpr float kMinScale = 1.17549435e-38f;  // smaller scales are stored as 0

// x / s to float32's nearest for many x and one s, with r = 1 / s rounded to nearest.  x r is off by less than
// two units of the last place; its remainder, times r, corrects it to within one; and from there the same
// step ends on the nearest (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  Five operations where the general division takes some ten and a branch: 8750 rows of 8 x
// 128, rotated, take 20.3 us in e4m3 and 22.9 in 4 bits, 21.8 and 24.4 with it.  Exact for s >= 2^-62 and |x| >= 2^-103;
// a smaller |x| / s stays below 2^-40.  The sign of a zero is lost.
__device__ __forceinline__ float quotient_of(float x, float s, float r) {
  const float q0 = x * r;
  const float q1 = __fmaf_rn(__fmaf_rn(-q0, s, x), r, q0);
  return __fmaf_rn(__fmaf_rn(-q1, s, x), r, q1);
}
// A power of two that brings s into that range, x / s being the same.
__device__ __forceinline__ float quotient_unit(float s) { return s < 8.67361738e-19f ? 1.84467441e19f : 1.f; }

// A thread's part of an 8- or 4-bit row: the codes of its two vectors, 8 channels each,
// and the row's scale word, the same in the kPerHead lanes of a head.
struct Codes {
  uint2 a = {0u, 0u}, b = {0u, 0u};
  uint32_t word;
};
template <int FMT, int kPerHead>
__device__ __forceinline__ Codes encode16(const Vec16& x) {
  Codes c;
  float scale;
  if constexpr (FMT == PDS_KV_E4M3) {
    float top = fabsf(x.x[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) top = max_or_nan(top, fabsf(x.x[i]));
    top = head_max<kPerHead>(top);
    const bool finite = top < INFINITY;
    scale = __fdiv_rn(top, 448.0f);
    if (!(scale >= kMinScale)) scale = 0.f;
    if (finite && scale > 0.f) {
      float y[16];
      const float unit = quotient_unit(scale), s = scale * unit, r = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = copysignf(quotient_of(x.x[i] * unit, s, r), x.x[i]);
      c.a = make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
      c.b = make_uint2(e4m3x4(y[8], y[9], y[10], y[11]), e4m3x4(y[12], y[13], y[14], y[15]));
    }
    c.word = finite ? __float_as_uint(scale) : 0x7fc00000u;
  } else {
    float hi = 0.f, low = 0.f;  // low: the other way round
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      hi = max_or_nan(hi, x.x[i]);
      low = max_or_nan(low, -x.x[i]);
    }
    hi = head_max<kPerHead>(hi);
    low = head_max<kPerHead>(low);
    const bool finite = hi < INFINITY && low < INFINITY;
    scale = bf16_to_f32(f32_to_bf16(__fdiv_rn(hi, 15.0f) + __fdiv_rn(low, 15.0f)));
    if (!(scale >= kMinScale)) scale = 0.f;
    float z = 0.f;
    if (finite && scale > 0.f) {
      z = fminf(fmaxf(rintf(__fdiv_rn(low, scale)), 0.f), 15.f);
      // (clipped first, for the bounds are integers; rounded by what a sum near 2^23 cannot hold)
      const float unit = quotient_unit(scale), s = scale * unit, r = __frcp_rn(s);
      const uint32_t base = 0x4b400000u - static_cast<uint32_t>(z);
      uint32_t n[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float y = fminf(fmaxf(quotient_of(x.x[i] * unit, s, r), -z), 15.f - z);
        n[i] = __float_as_uint(y + 12582912.f) - base;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c.a.x += n[i] << (4 * i);
        c.b.x += n[8 + i] << (4 * i);
      }
    }
    c.word = finite ? (__float_as_uint(scale) | static_cast<uint32_t>(z)) : 0x7fc00000u;
  }
  return c;
}

// The 16 channels that two pieces of 8 codes stand for (e4m3: q.xy and q.zw, 4 bits: q.x
// and q.y), with their row's scale word.
template <int FMT>
__device__ __forceinline__ void decode16(const uint4& q, uint32_t word, float (&x)[16]) {
  if constexpr (FMT == PDS_KV_E4M3) {
    const uint32_t qs[4] = {q.x, q.y, q.z, q.w};
    const float scale = __uint_as_float(word);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
          static_cast<__nv_fp8x2_storage_t>(qs[e >> 1] >> (16 * (e & 1))), __NV_E4M3);
      const float2 f = __half22float2(__half2(hr));
      x[2 * e] = f.x * scale;
      x[2 * e + 1] = f.y * scale;
    }
  } else {
    const float scale = __uint_as_float(word & 0xffff0000u);
    const int z = word & 15;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int n4 = ((e < 8 ? q.x : q.y) >> (4 * (e & 7))) & 15;
      x[e] = static_cast<float>(n4 - z) * scale;
    }
  }
}

}  // namespace pds
