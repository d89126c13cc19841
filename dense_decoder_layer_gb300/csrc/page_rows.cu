// The paged K/V cache but for its attention: pages taken and given back, the
// slots of rows, rows written and read by slot.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kv_rows.cuh"
#include "pages.h"
#include "sm100.cuh"
#include "tc.h"

namespace pds {
namespace {

// ------------------------------------------------- tables and slot maps
//
// Prefix sums over the sequences, then a page or a row per thread, which finds its
// sequence by bisection in shared memory.  Nothing here is large: what bounds the calls is
// the latency of a launch, the lengths' loads, the sums, a table entry's load and its
// store, one after the other; so blocks are as small as the work and loads go out early.
// Measured in replayed graphs, a reserve and a release together: 8 sequences, one row each, 4.3 us;
// 256 with up to 512 rows each 12.8; 64 with 1000 to 4096 10.4.

constexpr int kMaxScanThreads = 1024;
// Up to this many rows the block that takes pages writes their slots too: a launch less, but one SM's loads
// and stores.  us of a reserve and a release with one block / with a second kernel, pages of 16: 256 sequences
// of 4 rows 5.8 / 9.4, 8 of 512 6.2 / 7.0, 8 of 1024 8.4 / 7.0, 64 of 128 10.9 / 7.7, 64 of 256 17.1 / 8.2, 256 of 64
// 18.8 / 9.6.  (They meet between 4096 and 8192 rows.)
constexpr int kRowsOfOneBlock = 8192;
constexpr int kSlotThreads = 256, kSlotsPerThread = 4;

struct Sums {
  int64_t a, b;
  int32_t bad;
};
// Exclusive sums over the block's threads of (a, b), the totals, and whether any was bad; one barrier.
// Only the first `threads` have any.
__device__ __forceinline__ Sums block_sums(const Sums& x, int threads, Sums* scratch, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (threads + 31) >> 5;
  Sums incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, incl.a, o);
    const int64_t b = __shfl_up_sync(0xffffffffu, incl.b, o);
    if (lane >= o) {
      incl.a += a;
      incl.b += b;
    }
  }
  incl.bad = __any_sync(0xffffffffu, x.bad);
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  Sums before{0, 0, 0};
  *total = Sums{0, 0, 0};
  for (int w = 0; w < warps; ++w) {  // (broadcast reads)
    const Sums s = scratch[w];
    if (w < warp) {
      before.a += s.a;
      before.b += s.b;
    }
    total->a += s.a;
    total->b += s.b;
    total->bad |= s.bad;
  }
  return Sums{before.a + incl.a - x.a, before.b + incl.b - x.b, 0};
}

// The last s < n with before[s] <= i (before[0] = 0, ascending).
__device__ __forceinline__ int holder(const int32_t* before, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Row t of the map: its slot and position; -1 and 0 behind the last.
__device__ __forceinline__ void map_row(const PageView& p, const int32_t* starts,
                                        const int32_t* first, int t, int32_t* slots,
                                        int32_t* positions, uint32_t* status) {
  int32_t slot = -1, pos = 0;
  if (t < starts[p.n_seqs]) {
    const int s = holder(starts, p.n_seqs, t);
    pos = first[s] + (t - starts[s]);
    const int page = p.table[static_cast<int64_t>(s) * p.max_pages + (pos >> p.page_shift)];
    if (page >= 0 && page < p.n_pages)
      slot = (page << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
    else
      atomicOr(status, kStatusBadPage);
  }
  slots[t] = slot;
  if (positions) positions[t] = pos;
}

// TAKE: one block takes pages for rows first[s] .. first[s] + count[s] - 1 of every
// sequence from the free ones and enters them into the table (first is lens), writes the starts
// and with `map` the rows' slots.  Else every block makes the sums for itself and maps
// rows of its own.  A thread has PER sequences.
template <bool TAKE, int PER>
__global__ void __launch_bounds__(kMaxScanThreads, 1)
    pages_scan_kernel(const __grid_constant__ PageView p, const int32_t* first, const int32_t* count,
                      int n_rows, int32_t* slots, int32_t* positions, int32_t* starts, int map,
                      uint32_t* status) {
  extern __shared__ int32_t before_rows[];           // [n + 1]; TAKE: and the two below
  __shared__ Sums scratch[kMaxScanThreads / 32];
  const int n = p.n_seqs, P = 1 << p.page_shift;
  int32_t* before_pages = before_rows + n + 1;       // [n + 1]
  int32_t* at_page = before_pages + n + 1;           // [n]: where a sequence's first taken page goes, less its number
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  int32_t take[PER], rows[PER], held[PER];
  Sums mine{0, 0, 0};
  const int32_t n_free = TAKE ? *p.n_free : 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = static_cast<int>(threadIdx.x) * PER + i;
    take[i] = rows[i] = held[i] = 0;
    if (s >= n) continue;
    const int64_t len = first[s], add = count[s];
    const int h = p.held ? p.held[s] : p.max_pages;
    if (len < 0 || add < 0 || len + add > (static_cast<int64_t>(p.max_pages) << p.page_shift) || h < 0 ||
        h > p.max_pages) {
      mine.bad = 1;
      continue;
    }
    const int need = static_cast<int>((len + add + P - 1) >> p.page_shift);
    rows[i] = static_cast<int32_t>(add);
    held[i] = h;
    take[i] = max(need - h, 0);
    if (!TAKE && take[i] > 0 && add > 0) mine.bad = 1;  // rows that the sequence has no pages for
    mine.a += add;
    mine.b += take[i];
  }
  Sums total;
  Sums at = block_sums(mine, (n + PER - 1) / PER, scratch, &total);
  const bool bad_rows = total.bad || total.a > n_rows;
  const bool bad = bad_rows || (TAKE && (n_free < 0 || n_free > p.n_pages || total.b > n_free));
  if (bad && threadIdx.x == 0 && blockIdx.x == 0)  // nothing is taken and the map is empty
    atomicOr(status, bad_rows ? kStatusBadLength : kStatusNoPages);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = static_cast<int>(threadIdx.x) * PER + i;
    if (s < n) {
      const int32_t start = bad ? 0 : static_cast<int32_t>(at.a);
      before_rows[s] = start;
      if (starts && blockIdx.x == 0) starts[s] = start;
      if (TAKE && !bad) {
        before_pages[s] = static_cast<int32_t>(at.b);
        at_page[s] = held[i] - static_cast<int32_t>(at.b);
        if (take[i] > 0) p.held[s] = held[i] + take[i];
      }
    }
    at.a += rows[i];
    at.b += take[i];
  }
  if (threadIdx.x == 0) {
    const int32_t all = bad ? 0 : static_cast<int32_t>(total.a);
    before_rows[n] = all;
    if (starts && blockIdx.x == 0) starts[n] = all;
    if (TAKE && !bad && total.b > 0) *p.n_free = n_free - static_cast<int32_t>(total.b);
  }
  __syncthreads();
  if (TAKE && !bad && total.b > 0) {
    for (int i = threadIdx.x; i < total.b; i += blockDim.x) {
      const int s = holder(before_pages, n, i);
      p.table[static_cast<int64_t>(s) * p.max_pages + at_page[s] + i] = p.free_pages[n_free - 1 - i];
    }
    if (map) __syncthreads();
  }
  if (map)
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < n_rows;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x)
      map_row(p, before_rows, first, static_cast<int>(t), slots, positions, status);
}

// The slots of many rows: every block has the starts in shared memory.
__global__ void __launch_bounds__(kSlotThreads)
    pages_slots_kernel(const __grid_constant__ PageView p, const int32_t* first, int n_rows,
                       int32_t* slots, int32_t* positions, const int32_t* starts, uint32_t* status) {
  __shared__ int32_t before[kMaxPagedSeqs + 1];
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  for (int i = threadIdx.x; i <= p.n_seqs; i += kSlotThreads) before[i] = starts[i];
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * (kSlotThreads * kSlotsPerThread) + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kSlotsPerThread; ++i) {
    const int64_t t = t0 + i * kSlotThreads;
    if (t < n_rows) map_row(p, before, first, static_cast<int>(t), slots, positions, status);
  }
}

// One block: every sequence keeps the pages of its first keep[s] rows.
template <int PER>
__global__ void __launch_bounds__(kMaxScanThreads, 1)
    pages_release_kernel(const __grid_constant__ PageView p, const int32_t* keep, uint32_t* status) {
  extern __shared__ int32_t before[];  // [n], and:
  __shared__ Sums scratch[kMaxScanThreads / 32];
  const int n = p.n_seqs, P = 1 << p.page_shift;
  int32_t* at_page = before + n;       // [n]: where a sequence's first page to go is, less its number
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int32_t n_free = *p.n_free;
  int32_t gone[PER], left[PER];
  Sums mine{0, 0, 0};
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = static_cast<int>(threadIdx.x) * PER + i;
    gone[i] = left[i] = 0;
    if (s >= n) continue;
    const int64_t rows = keep[s];
    const int h = p.held[s];
    if (rows < 0 || h < 0 || h > p.max_pages) mine.bad = 1;
    left[i] = static_cast<int>(min(static_cast<int64_t>(h), (rows + P - 1) >> p.page_shift));
    gone[i] = h - left[i];
    mine.a += gone[i];
  }
  Sums total;
  Sums at = block_sums(mine, (n + PER - 1) / PER, scratch, &total);
  if (total.bad || n_free < 0 || total.a > p.n_pages - n_free) {  // (more pages than there are)
    if (threadIdx.x == 0) atomicOr(status, kStatusBadLength);
    return;
  }
  if (total.a == 0) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = static_cast<int>(threadIdx.x) * PER + i;
    if (s < n) {
      before[s] = static_cast<int32_t>(at.a);
      at_page[s] = left[i] - static_cast<int32_t>(at.a);
      if (gone[i] > 0) p.held[s] = left[i];
    }
    at.a += gone[i];
  }
  const int32_t all = static_cast<int32_t>(total.a);
  if (threadIdx.x == 0) *p.n_free = n_free + all;
  __syncthreads();
  for (int i = threadIdx.x; i < all; i += blockDim.x) {
    const int s = holder(before, n, i);
    p.free_pages[n_free + all - 1 - i] = p.table[static_cast<int64_t>(s) * p.max_pages + at_page[s] + i];
  }
}

// ------------------------------------------------------- rows by slot
//
// Slots, positions and rows may come from the kernel before, which is waited for: no pointer to
// const is __restrict__, which would let its loads pass the wait.

constexpr int kRowThreads = 256;

// Where a row's head starts; null (and the status) for a slot that is none, null
// alone for -1.
__device__ __forceinline__ bool slot_ok(const PageView& p, int32_t slot, uint32_t* status) {
  if (slot >= 0 && (slot >> p.page_shift) < p.n_pages) return true;
  if (slot != -1) atomicOr(status, kStatusBadPage);
  return false;
}
__device__ __forceinline__ char* row_at(const PageView& p, char* base, int32_t slot, int h) {
  return base + (slot >> p.page_shift) * p.page_stride +
         (slot & ((1 << p.page_shift) - 1)) * p.row_stride + h * p.head_stride;
}
__device__ __forceinline__ int64_t word_at(const PageView& p, int32_t slot, int h) {
  return ((static_cast<int64_t>(slot >> p.page_shift) * p.n_kv_heads + h) << p.page_shift) +
         (slot & ((1 << p.page_shift) - 1));
}

// A block takes ROWS new rows, their K and V heads.  Few rows are bound by latency (64 rows of
// 8 x 128, rotated, to e4m3: 2.2 us), so a block has one; many by issuing the turns, the rounding
// and the addresses, in 0.66 of all cycles (e4m3 0.70, 4 bits 0.75): 8750 rows of 8 x 128, rotated, 14.3 us in
// bf16, 74% of a copy's rate; e4m3 20.3 (39%), 4 bits 22.9 (29%), whose extrema, quotients and codes are as many
// again.
// (A row per warp saved addresses but made every turn once per warp: 64 rows took 3.7 us.)
template <int FMT, int HD, int ROWS>
__global__ void __launch_bounds__(kRowThreads)
    pages_write_kernel(const __grid_constant__ PageView p, const __grid_constant__ RopeTurns r,
                       const uint16_t* k, const uint16_t* v, const int32_t* slots, int n_rows,
                       int64_t k_stride, int64_t v_stride, const int32_t* positions, uint32_t* status) {
  constexpr int kPerHead = HD / 16;
  __shared__ float2 table[ROWS][HD / 2];
  const int row0 = blockIdx.x * ROWS;
  const int rows = min(ROWS, n_rows - row0);
  const int half_units = p.n_kv_heads * kPerHead, per_row = 2 * half_units, units = rows * per_row;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  int u = threadIdx.x;
  uint4 wa = {}, wb = {};
  int h = 0, uu = 0, ch_a = 0, ch_b = 0, i_row = 0;
  int32_t slot = -1;
  bool is_v = false;
  auto load = [&]() {
    i_row = 0;
#pragma unroll
    for (int j = 1; j < ROWS; ++j) i_row += u >= j * per_row;
    int w = u - i_row * per_row;
    is_v = w >= half_units;
    if (is_v) w -= half_units;
    h = w / kPerHead;
    uu = w - h * kPerHead;
    unit_channels(uu, is_v ? 0 : r.rot_dim, r.layout, ch_a, ch_b);
    const int64_t row = row0 + i_row;
    const uint16_t* src = (is_v ? v + row * v_stride : k + row * k_stride) + h * HD;
    wa = *reinterpret_cast<const uint4*>(src + ch_a);
    wb = *reinterpret_cast<const uint4*>(src + ch_b);
    slot = slots[row];
  };
  if (u < units) load();
  if (r.rot_dim > 0) {
    const int pairs = r.rot_dim / 2;
    for (int i = threadIdx.x; i < rows * pairs; i += blockDim.x) {
      const int j = ROWS == 1 ? 0 : i / pairs;
      table[j][turn_at(r, i - j * pairs)] = pair_turn(r, i - j * pairs, positions[row0 + j]);
    }
    __syncthreads();
  }
  // warp-uniform bound: every lane of a warp takes part in the extrema
  for (int base = threadIdx.x & ~31; base < units; base += blockDim.x) {
    const bool live = u < units && slot_ok(p, slot, status);
    Vec16 x;
    widen8(wa, x.x);
    widen8(wb, x.x + 8);
    if (u < units && !is_v) rotate_unit(x, uu, r, table[i_row]);
    char* dst = live ? row_at(p, is_v ? p.v : p.k, slot, h) : nullptr;
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
        if (uu == 0) (is_v ? p.v_scale : p.k_scale)[word_at(p, slot, h)] = w.word;
      }
    }
    u += blockDim.x;
    if (u < units) load();
  }
}

// A warp takes a row (or as many as fit its lanes): one slot and one address, then a step per head.
// (With a division and four 64-bit products for each 16 channels the read issued on 75% of all cycles.)
__host__ __device__ constexpr int lanes_of_row(int per_row) { return per_row < 32 ? per_row : 32; }
struct RowLanes {
  int lanes;    // of a row
  int rows;     // of a pass
  int sub, u0;  // this lane's row of a pass (rows: none), its first unit
};
__device__ __forceinline__ RowLanes row_lanes(int per_row) {
  const int lane = threadIdx.x & 31;
  RowLanes r;
  r.lanes = lanes_of_row(per_row);
  r.rows = 32 / r.lanes;
  r.sub = lane / r.lanes;
  r.u0 = lane - r.sub * r.lanes;
  return r;
}

constexpr int kReadThreads = 128;

// A warp takes two rows (or twice as many as fit its lanes) of K or V.  A thread's 16 channels are two
// pieces of 8, half a head apart, so that a warp's stores lie side by side.  Bound by HBM, as far as the
// output does not stay in L2, and the ramp.  262 thousand rows of 8 x 128: bf16 303 us, e4m3 231, 4 bits 200 (7.1,
// 7.1, 6.8 TB/s); 24.6 thousand e4m3 with their slot map 28.5 (5.3), 9.7 thousand 4-bit rows of 8 x 64 with it 8.9
// (2.9).
template <int FMT, int HD>
__global__ void __launch_bounds__(kReadThreads)
    pages_read_kernel(const __grid_constant__ PageView p, const int32_t* slots, int n_rows,
                      uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out, uint32_t* status) {
  constexpr int kPerHead = HD / 16, kRows = 2, kFlight = 2;
  const bool is_v = k_out == nullptr || blockIdx.y == 1;
  char* pool = is_v ? p.v : p.k;
  const uint32_t* scales = is_v ? p.v_scale : p.k_scale;
  uint16_t* out = is_v ? v_out : k_out;
  const int per_row = p.n_kv_heads * kPerHead;
  const RowLanes w = row_lanes(per_row);
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * (kReadThreads / 32) + (threadIdx.x >> 5)) * (kRows * w.rows);
  if (row0 >= n_rows) return;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  int32_t slot[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t row = row0 + j * w.rows + w.sub;
    slot[j] = w.sub < w.rows && row < n_rows ? slots[row] : -1;
  }
  const char* from[kRows];
  const uint32_t* words[kRows];
  uint16_t* to[kRows];
  bool ok[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    ok[j] = slot_ok(p, slot[j], status);
    const int32_t s = ok[j] ? slot[j] : 0;
    from[j] = row_at(p, pool, s, 0);
    words[j] = scales + (FMT != PDS_KV_BF16 ? word_at(p, s, 0) : 0);
    to[j] = out + (row0 + j * w.rows + w.sub) * (static_cast<int64_t>(p.n_kv_heads) * HD);
  }
  for (int u1 = w.u0; u1 < per_row; u1 += 32 * kFlight) {
    uint4 qa[kRows][kFlight], qb[kRows][kFlight];
    uint32_t word[kRows][kFlight];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int u = u1 + 32 * k, h = u / kPerHead, ch = (u - h * kPerHead) * 8;
        if (!ok[j] || u >= per_row) continue;
        const char* at = from[j] + h * p.head_stride;
        if constexpr (FMT == PDS_KV_BF16) {
          qa[j][k] = *reinterpret_cast<const uint4*>(at + 2 * ch);
          qb[j][k] = *reinterpret_cast<const uint4*>(at + HD + 2 * ch);
        } else if constexpr (FMT == PDS_KV_E4M3) {
          const uint2 lo = *reinterpret_cast<const uint2*>(at + ch);
          const uint2 hi = *reinterpret_cast<const uint2*>(at + HD / 2 + ch);
          qa[j][k] = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          qa[j][k].x = *reinterpret_cast<const uint32_t*>(at + ch / 2);
          qa[j][k].y = *reinterpret_cast<const uint32_t*>(at + HD / 4 + ch / 2);
        }
        if constexpr (FMT != PDS_KV_BF16) word[j][k] = words[j][static_cast<int64_t>(h) << p.page_shift];
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int u = u1 + 32 * k, h = u / kPerHead, ch = (u - h * kPerHead) * 8;
        if (!ok[j] || u >= per_row) continue;
        uint4 lo = qa[j][k], hi = qb[j][k];
        if constexpr (FMT != PDS_KV_BF16) {
          float x[16];
          decode16<FMT>(qa[j][k], word[j][k], x);
          lo = narrow8(x);
          hi = narrow8(x + 8);
        }
        uint16_t* at = to[j] + h * HD + ch;
        *reinterpret_cast<uint4*>(at) = lo;
        *reinterpret_cast<uint4*>(at + HD / 2) = hi;
      }
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

// From this many rows on a block takes four.  us with one / four, rows of 8 x 128, rotated: 64 bf16 1.9 / 2.5, e4m3
// 2.2 / 3.4, 4 bits 2.2 / 3.5; 1024 3.1 / 3.1, 3.8 / 4.3, 4.2 / 4.6; 4096 6.4 / 6.5, 9.3 / 10.1, 10.9 / 11.3, whose
// inputs lie in L2.
constexpr int kManyRows = 1024;

// Threads of a block that makes the sums of n sequences, one or four each.
int scan_threads(int n, int per, int least) {
  return std::min(kMaxScanThreads, std::max(least, ((n + per - 1) / per + 31) / 32 * 32));
}

}  // namespace

cudaError_t launch_pages_reserve(const PageView& p, const int32_t* new_rows, int n_rows,
                                 int32_t* slots, int32_t* positions, int32_t* starts,
                                 uint32_t* status, cudaStream_t st) {
  const bool one = n_rows <= kRowsOfOneBlock;
  const int n = p.n_seqs, per = n <= kMaxScanThreads ? 1 : 4;
  const size_t smem = (3 * static_cast<size_t>(n) + 2) * 4;
  const auto kernel = per == 1 ? pages_scan_kernel<true, 1> : pages_scan_kernel<true, 4>;
  // (more than 48 KB with the sums' own for the last hundred sequences)
  cudaError_t ce = kernel_smem_attr(reinterpret_cast<const void*>(kernel), (3 * kMaxPagedSeqs + 2) * 4);
  if (ce != cudaSuccess) return ce;
  const int least = one ? std::min(n_rows, kMaxScanThreads) / 32 * 32 + 32 : kMaxScanThreads;
  ce = launch_after(kernel, dim3(1), scan_threads(n, per, least),
                    smem, st, p, static_cast<const int32_t*>(p.lens), new_rows, n_rows, slots, positions, starts,
                    one ? 1 : 0, status);
  if (ce != cudaSuccess || one) return ce;
  const int rows = kSlotThreads * kSlotsPerThread;
  return launch_after(pages_slots_kernel, dim3((n_rows - 1) / rows + 1), kSlotThreads, 0, st, p, p.lens,
                      n_rows, slots, positions, starts, status);
}

cudaError_t launch_pages_slots(const PageView& p, const int32_t* first, const int32_t* count,
                               int n_rows, int32_t* slots, int32_t* positions, int32_t* starts,
                               uint32_t* status, cudaStream_t st) {
  const int n = p.n_seqs, per = n <= kSlotThreads ? 1 : 4;
  const int threads = scan_threads(n, per, kSlotThreads);
  const int blocks = n_rows > 0 ? (n_rows - 1) / (threads * kSlotsPerThread) + 1 : 1;
  const auto kernel = per == 1 ? pages_scan_kernel<false, 1> : pages_scan_kernel<false, 4>;
  return launch_after(kernel, dim3(blocks), threads, (static_cast<size_t>(n) + 1) * 4, st, p, first, count, n_rows,
                      slots, positions, starts, 1, status);
}

cudaError_t launch_pages_release(const PageView& p, const int32_t* keep, uint32_t* status,
                                 cudaStream_t st) {
  const int n = p.n_seqs, per = n <= kMaxScanThreads ? 1 : 4;
  const auto kernel = per == 1 ? pages_release_kernel<1> : pages_release_kernel<4>;
  // A small block starts sooner, a large one moves many pages faster.  us with 128 threads / 1024, with
  // two small copies that set the case up: 8 sequences, one page each, 3.9 / 4.0, 16 3.8 / 4.0, 128 5.8 / 4.0; 64 of 16 6.9 / 4.3.
  return launch_after(kernel, dim3(1), scan_threads(n, per, n <= 32 ? 128 : kMaxScanThreads),
                      2 * static_cast<size_t>(n) * 4, st, p, keep, status);
}

cudaError_t launch_pages_write(const PageView& p, int format, int hd, const RopeTurns& r,
                               const uint16_t* k, const uint16_t* v, const int32_t* slots,
                               int n_rows, int64_t k_stride, int64_t v_stride,
                               const int32_t* positions, uint32_t* status, cudaStream_t st) {
  const int per_row = 2 * p.n_kv_heads * (hd / 16);
  return by_format(format, hd, [&](auto fmt, auto w) {
    auto launch = [&](auto kernel, int rows) {
      const int threads = std::min(kRowThreads, (rows * per_row + 31) / 32 * 32);
      return launch_after(kernel, dim3((n_rows - 1) / rows + 1), threads, 0, st, p, r, k, v, slots,
                          n_rows, k_stride, v_stride, positions, status);
    };
    return n_rows >= kManyRows ? launch(pages_write_kernel<fmt, w, 4>, 4)
                               : launch(pages_write_kernel<fmt, w, 1>, 1);
  });
}

cudaError_t launch_pages_read(const PageView& p, int format, int hd, const int32_t* slots,
                              int n_rows, uint16_t* k_out, uint16_t* v_out, uint32_t* status,
                              cudaStream_t st) {
  const int rows = 2 * (32 / lanes_of_row(p.n_kv_heads * (hd / 16))) * (kReadThreads / 32);
  const dim3 grid((n_rows - 1) / rows + 1, k_out && v_out ? 2 : 1);
  return by_format(format, hd, [&](auto fmt, auto w) {
    return launch_after(pages_read_kernel<fmt, w>, grid, kReadThreads, 0, st, p, slots, n_rows, k_out,
                        v_out, status);
  });
}

}  // namespace pds
