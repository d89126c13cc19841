// Rotary positions, the quantised K/V cache and the attention of drafted
// tokens over it: launch interface between the host library and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

#include "../../include/pds.h"

namespace pds {

// A pds_cache as the kernels see it: strides in bytes.
struct CacheView {
  char* k;
  char* v;
  uint32_t* k_scale;
  uint32_t* v_scale;
  const int32_t* lens;
  int64_t seq_stride, row_stride, head_stride;
  int n_seqs, capacity, n_kv_heads;
};

// Rotated pairs of a head: pair i turns by p * turns[i] / 2^64 of a full turn
// at position p.
constexpr int kMaxTurnPairs = 128;
struct RopeTurns {
  uint64_t turns[kMaxTurnPairs];
  int rot_dim;  // rotated channels (2 * pairs); 0: no rotation
  int layout;
  float mscale;
  float sign;   // -1: the inverse rotation
};

// The most tokens of a sequence that may form a tree, and that
// pds_attention_tree takes.
constexpr int kMaxDraftTokens = 256;

struct TreeAttnCall {
  CacheView cache;
  int format, head_dim;
  const uint16_t* q;
  uint16_t* o;
  int64_t q_stride, o_stride;  // elements
  const int32_t* parents;
  int n_tokens, n_heads;
  int max_len;
  float softcap;
  int window;
  char* ws;  // null: key ranges are not split
  uint32_t* status;
  int num_sms;
};

// Launch with programmatic stream serialization: the kernel may begin while
// the one before it ends, so it waits (griddepcontrol.wait) before it touches
// memory.  Every kernel of the decoding path does and lets its successor begin
// early in turn: a decode step is a row of kernels of a few microseconds, of
// which a launch that waits for the end of its predecessor is a large part.
// The grid in clusters of `cluster` blocks along x.
template <typename... Params, typename... Given>
cudaError_t launch_after_cluster(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                                 int cluster, cudaStream_t st, Given&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}
template <typename... Params, typename... Given>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                         cudaStream_t st, Given&&... args) {
  return launch_after_cluster(kernel, grid, threads, smem, 1, st, args...);
}

cudaError_t launch_rope(const RopeTurns& r, const uint16_t* x, uint16_t* y, int rows, int heads,
                        int hd, int64_t x_stride, int64_t y_stride, const int32_t* positions,
                        int start_pos, cudaStream_t st);
cudaError_t launch_cache_write(const CacheView& c, int format, int hd, const RopeTurns& r,
                               const uint16_t* k, const uint16_t* v, int n_tokens,
                               int64_t k_stride, int64_t v_stride, const int32_t* parents,
                               const int32_t* positions, uint32_t* status, cudaStream_t st);
cudaError_t launch_cache_read(const CacheView& c, int format, int hd, int first_row, int rows,
                              uint16_t* k_out, uint16_t* v_out, uint32_t* status, cudaStream_t st);
size_t tree_attention_ws_bytes(int format, int hd, int n_seqs, int n_tokens, int n_heads,
                               int n_kv_heads, int num_sms);
pds_status tree_attention(const TreeAttnCall& a, cudaStream_t st, std::string* err);

}  // namespace pds
