// Rows of the decoding path: rotary positions (pds_rope), the K/V rows of new
// tokens into a cache that may hold 8- or 4-bit rows (pds_cache_write) and
// back (pds_cache_read).
//
// All three are bound by HBM when there are many rows and by latency when
// there are few: every value is read once and written once, and nothing else
// of their size exists.  A thread owns 16 channels of a head, as two 16-byte
// vectors that hold both channels of 8 rotated pairs: with the Neox layout
// channels [8u, 8u+8) and [rot/2 + 8u, ...+8), with the Norm layout (and
// without rotation) 16 adjacent ones.  So a rotation needs no exchange between
// threads and may run in place, and the extrema that a quantised row needs are
// taken over the 4 or 8 neighbouring lanes of its head.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kv.h"
#include "kv_rows.cuh"
#include "sm100.cuh"

namespace pds {
namespace {

// The kernels below start while the one before them may still write what they read, and wait for it: no
// pointer to const is __restrict__, which would let its loads pass the wait.
constexpr int kRowThreads = 256;

// One block per ROWS rows (and slice of their units): a thread's units of all of
// them are loaded before the table is made and while it is.  Two rows per block
// when there are many (us for 8192 / 2048 rows of 32 x 128 with one, two and four:
// 24.4/5.7, 22.0/5.1, 24.6/5.8; one waits more for its table, four leave fewer
// blocks per SM), one when there are few and latency counts.
template <int ROWS>
__global__ void __launch_bounds__(kRowThreads) rope_kernel(const uint16_t* x, uint16_t* y, int rows,
                                                           int heads, int hd, int64_t x_stride,
                                                           int64_t y_stride,
                                                           const int32_t* positions, int start_pos,
                                                           const __grid_constant__ RopeTurns r) {
  __shared__ float2 table[ROWS * kMaxTurnPairs];
  const int row0 = blockIdx.x * ROWS;
  const int per_head = hd >> 4, units = heads * per_head;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int step = blockDim.x * gridDim.y;
  int u = blockIdx.y * blockDim.x + threadIdx.x;
  uint4 wa[ROWS], wb[ROWS];
  int off_a = 0, off_b = 0, uu = 0;
  auto load = [&]() {
    const int h = u / per_head;
    int a, b;
    uu = u - h * per_head;
    unit_channels(uu, r.rot_dim, r.layout, a, b);
    off_a = h * hd + a;
    off_b = h * hd + b;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (ROWS > 1 && row0 + i >= rows) continue;
      const uint16_t* xr = x + (row0 + i) * x_stride;
      wa[i] = *reinterpret_cast<const uint4*>(xr + off_a);
      wb[i] = *reinterpret_cast<const uint4*>(xr + off_b);
    }
  };
  if (u < units) load();
  const int pairs = r.rot_dim / 2;
  for (int i = threadIdx.x; i < ROWS * pairs; i += blockDim.x) {
    const int k = ROWS > 1 ? i / pairs : 0, row = row0 + k;
    if (ROWS > 1 && row >= rows) break;
    const int64_t pos = positions ? static_cast<int64_t>(positions[row])
                                  : static_cast<int64_t>(start_pos) + row;
    table[k * kMaxTurnPairs + turn_at(r, i - k * pairs)] = pair_turn(r, i - k * pairs, pos);
  }
  __syncthreads();
  while (u < units) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (ROWS > 1 && row0 + i >= rows) break;
      Vec16 v;
      widen8(wa[i], v.x);
      widen8(wb[i], v.x + 8);
      rotate_unit(v, uu, r, table + i * kMaxTurnPairs);
      uint16_t* yr = y + (row0 + i) * y_stride;
      *reinterpret_cast<uint4*>(yr + off_a) = narrow8(v.x);
      *reinterpret_cast<uint4*>(yr + off_b) = narrow8(v.x + 8);
    }
    u += step;
    if (u < units) load();
  }
}

// One block per new token: its Hkv K rows, then its Hkv V rows.  The loads of
// the thread's first unit do not depend on the sequence's length, so they go
// out before lens and the parents are read.  2048 tokens of 8 x 128, rotated and
// stored as e4m3, 12.8 MB, take 5.9 us, 8 single tokens as 4-bit 2.3: latency
// (lengths, the turns, a head's extrema, divisions, stores), not bytes.
template <int FMT, int HD>
__global__ void __launch_bounds__(kRowThreads)
    cache_write_kernel(const __grid_constant__ CacheView c, const __grid_constant__ RopeTurns r,
                       const uint16_t* k, const uint16_t* v, int n_tokens, int64_t k_stride,
                       int64_t v_stride, const int32_t* parents, const int32_t* positions,
                       uint32_t* status) {
  constexpr int kPerHead = HD / 16;
  __shared__ float2 table[HD / 2];
  __shared__ int32_t par[kMaxDraftTokens];
  const int row = blockIdx.x;
  const int s = row / n_tokens, t = row - s * n_tokens;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int half_units = c.n_kv_heads * kPerHead, units = 2 * half_units;
  int u = threadIdx.x;
  uint4 wa = {}, wb = {};
  int h = 0, uu = 0, ch_a = 0, ch_b = 0;
  bool is_v = false;
  auto load = [&]() {
    is_v = u >= half_units;
    const int w = is_v ? u - half_units : u;
    h = w / kPerHead;
    uu = w - h * kPerHead;
    unit_channels(uu, is_v ? 0 : r.rot_dim, r.layout, ch_a, ch_b);
    const uint16_t* src = (is_v ? v + row * v_stride : k + row * k_stride) + h * HD;
    wa = *reinterpret_cast<const uint4*>(src + ch_a);
    wb = *reinterpret_cast<const uint4*>(src + ch_b);
  };
  if (u < units) load();
  const int len = c.lens[s];
  if (len < 0 || len > c.capacity - n_tokens) {  // the whole sequence is refused
    if (threadIdx.x == 0) atomicOr(status, kStatusBadLength);
    return;
  }
  int depth = t;
  if (parents) {
    const int32_t* p = parents + static_cast<int64_t>(s) * n_tokens;
    for (int i = threadIdx.x; i <= t; i += blockDim.x) par[i] = p[i];
    __syncthreads();
    depth = tree_depth(par, t);
    if (depth < 0) {  // padding, or a path that does not end in a root
      if (depth == kBadParent && threadIdx.x == 0) atomicOr(status, kStatusBadParent);
      return;
    }
  }
  if (r.rot_dim > 0) {
    fill_table(table, r, positions ? static_cast<int64_t>(positions[row])
                                   : static_cast<int64_t>(len) + depth);
    __syncthreads();
  }
  const int64_t j = len + t;
  // warp-uniform bound: every lane of a warp takes part in the extrema
  for (int base = threadIdx.x & ~31; base < units; base += blockDim.x) {
    const bool live = u < units;
    Vec16 x;
    widen8(wa, x.x);
    widen8(wb, x.x + 8);
    if (live && !is_v) rotate_unit(x, uu, r, table);
    char* dst = (is_v ? c.v : c.k) + s * c.seq_stride + j * c.row_stride + h * c.head_stride;
    if constexpr (FMT == PDS_KV_BF16) {
      if (live) {
        *reinterpret_cast<uint4*>(dst + 2 * ch_a) = narrow8(x.x);
        *reinterpret_cast<uint4*>(dst + 2 * ch_b) = narrow8(x.x + 8);
      }
    } else {
      const Codes w = encode16<FMT, kPerHead>(x);
      if (live) {
        if constexpr (FMT == PDS_KV_E4M3) {
          *reinterpret_cast<uint2*>(dst + ch_a) = w.a;
          *reinterpret_cast<uint2*>(dst + ch_b) = w.b;
        } else {
          *reinterpret_cast<uint32_t*>(dst + ch_a / 2) = w.a.x;
          *reinterpret_cast<uint32_t*>(dst + ch_b / 2) = w.b.x;
        }
        if (uu == 0)
          (is_v ? c.v_scale : c.k_scale)[(static_cast<int64_t>(s) * c.n_kv_heads + h) * c.capacity +
                                         j] = w.word;
      }
    }
    u += blockDim.x;
    if (u < units) load();
  }
}

// A block takes kReadRows rows (all heads) of one sequence's K or V: the scale
// words of a head are adjacent rows, so a block uses most of each sector of
// them that it fetches.  A thread's 16 channels are two pieces of 8, half a head
// apart, so that a warp's stores lie side by side: 8 x 8192 rows of e4m3, 407 MB,
// take 60.9 us (6.7 TB/s; with 16 adjacent channels 69.5), 8192 rows 9.5.
constexpr int kReadRows = 16;

template <int FMT, int HD>
__global__ void __launch_bounds__(kRowThreads)
    cache_read_kernel(const __grid_constant__ CacheView c, int first_row, int rows,
                      uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out,
                      uint32_t* status) {
  constexpr int kPerHead = HD / 16;
  const int s = blockIdx.y;
  const bool is_v = k_out == nullptr || blockIdx.z == 1;
  const char* src = (is_v ? c.v : c.k) + s * c.seq_stride;
  const uint32_t* scales = (is_v ? c.v_scale : c.k_scale);
  uint16_t* out = is_v ? v_out : k_out;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int len = c.lens[s];
  const bool at_lens = first_row < 0;
  if (len < 0 || len > c.capacity || (at_lens && len > c.capacity - rows)) {
    if (threadIdx.x == 0) atomicOr(status, kStatusBadLength);
    return;
  }
  const int r0 = blockIdx.x * kReadRows;
  const int64_t j0 = at_lens ? len : first_row;          // cache row of output row 0
  const int64_t live = at_lens ? rows : min(static_cast<int64_t>(rows), len - j0);
  const int n = static_cast<int>(min(static_cast<int64_t>(kReadRows), live - r0));
  // four units per thread in flight
  const int per_row = c.n_kv_heads * kPerHead, total = n * per_row;
  constexpr int kFlight = 4;
  for (int u0 = threadIdx.x; u0 < total; u0 += kFlight * kRowThreads) {
    uint4 qa[kFlight], qb[kFlight];
    uint32_t word[kFlight];
    int64_t to[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int u = u0 + i * kRowThreads;
      to[i] = -1;
      if (u >= total) continue;
      const int r = u / per_row, w = u - r * per_row;
      const int h = w / kPerHead, ch = (w - h * kPerHead) * 8;
      const int64_t j = j0 + r0 + r;
      const char* p = src + j * c.row_stride + h * c.head_stride;
      to[i] = ((static_cast<int64_t>(s) * rows + r0 + r) * c.n_kv_heads + h) * HD + ch;
      if constexpr (FMT == PDS_KV_BF16) {
        qa[i] = *reinterpret_cast<const uint4*>(p + 2 * ch);
        qb[i] = *reinterpret_cast<const uint4*>(p + HD + 2 * ch);
      } else if constexpr (FMT == PDS_KV_E4M3) {
        const uint2 lo = *reinterpret_cast<const uint2*>(p + ch);
        const uint2 hi = *reinterpret_cast<const uint2*>(p + HD / 2 + ch);
        qa[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        qa[i].x = *reinterpret_cast<const uint32_t*>(p + ch / 2);
        qa[i].y = *reinterpret_cast<const uint32_t*>(p + HD / 4 + ch / 2);
      }
      if constexpr (FMT != PDS_KV_BF16)
        word[i] = scales[(static_cast<int64_t>(s) * c.n_kv_heads + h) * c.capacity + j];
    }
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (to[i] < 0) continue;
      uint4 lo = qa[i], hi = qb[i];
      if constexpr (FMT != PDS_KV_BF16) {
        float x[16];
        decode16<FMT>(qa[i], word[i], x);
        lo = narrow8(x);
        hi = narrow8(x + 8);
      }
      *reinterpret_cast<uint4*>(out + to[i]) = lo;
      *reinterpret_cast<uint4*>(out + to[i] + HD / 2) = hi;
    }
  }
}

// Calls f with the format and head width as compile-time constants.
template <typename F>
cudaError_t by_format(int format, int hd, F&& f) {
  auto with_hd = [&](auto fmt) {
    return hd == 128 ? f(fmt, std::integral_constant<int, 128>{})
                     : f(fmt, std::integral_constant<int, 64>{});
  };
  switch (format) {
    case PDS_KV_BF16: return with_hd(std::integral_constant<int, PDS_KV_BF16>{});
    case PDS_KV_E4M3: return with_hd(std::integral_constant<int, PDS_KV_E4M3>{});
    default: return with_hd(std::integral_constant<int, PDS_KV_INT4>{});
  }
}

constexpr int kManyRows = 2048;

int round_threads(int units) {  // a block that covers the units, whole warps
  return units >= kRowThreads ? kRowThreads : (units + 31) / 32 * 32;
}

}  // namespace

cudaError_t launch_rope(const RopeTurns& r, const uint16_t* x, uint16_t* y, int rows, int heads,
                        int hd, int64_t x_stride, int64_t y_stride, const int32_t* positions,
                        int start_pos, cudaStream_t st) {
  const int units = heads * (hd / 16);
  const int threads = round_threads(units);
  const int slices = std::min((units + threads - 1) / threads, 65535);
  // many rows: enough blocks of two to fill the GPU
  if (rows >= kManyRows)
    return launch_after(rope_kernel<2>, dim3(rows / 2 + rows % 2), threads, 0, st, x, y, rows, heads, hd,
                        x_stride, y_stride, positions, start_pos, r);
  // few: the units of a row are spread over several blocks
  return launch_after(rope_kernel<1>, dim3(rows, slices), threads, 0, st, x, y, rows, heads, hd,
                      x_stride, y_stride, positions, start_pos, r);
}
cudaError_t launch_cache_write(const CacheView& c, int format, int hd, const RopeTurns& r,
                               const uint16_t* k, const uint16_t* v, int n_tokens,
                               int64_t k_stride, int64_t v_stride, const int32_t* parents,
                               const int32_t* positions, uint32_t* status, cudaStream_t st) {
  const int units = 2 * c.n_kv_heads * (hd / 16);
  return by_format(format, hd, [&](auto fmt, auto w) {
    return launch_after(cache_write_kernel<fmt, w>, dim3(c.n_seqs * n_tokens), round_threads(units),
                        0, st, c, r, k, v, n_tokens, k_stride, v_stride, parents, positions, status);
  });
}

cudaError_t launch_cache_read(const CacheView& c, int format, int hd, int first_row, int rows,
                              uint16_t* k_out, uint16_t* v_out, uint32_t* status,
                              cudaStream_t st) {
  const dim3 grid((rows + kReadRows - 1) / kReadRows, c.n_seqs, k_out && v_out ? 2 : 1);
  return by_format(format, hd, [&](auto fmt, auto w) {
    return launch_after(cache_read_kernel<fmt, w>, grid, kRowThreads, 0, st, c, first_row, rows,
                        k_out, v_out, status);
  });
}

}  // namespace pds
