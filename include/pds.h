/*
 * pds.h -- C ABI of the GB300 dense prefill stack.
 *
 * One call runs a batch of B new tokens through a run of L consecutive
 * dense Llama-style decoder layers on one GPU and returns the new hidden
 * batch plus every layer's new K/V rows.  Each layer computes
 *
 *     h  = x + wo(attn(rope(q,k), v))      q,k,v = rms_norm(x) . wq/wk/wv
 *     x' = h + down(silu(gate(m)) * up(m)), m     = rms_norm(h)
 *
 * (frink-models 0.49.0 src/fused_layer.rs, module doc "What it refuses":
 * the fused layer is exactly x + ffn(rms_norm(x + branch)) with a SwiGLU
 * FFN of one dense expert; frink-models 0.29.0
 * src/decoder/cuda_prefill.rs, module doc: the hidden batch goes up once
 * and comes back after the last layer, everything between the seven
 * matmuls is a kernel, and each layer's K/V rows come back.)
 *
 * Conventions for every entry point:
 *  - Weights are row-major [out, in] bf16 (passed as uint16_t bit
 *    patterns) and y = x . W^T.  Norm gains are float32 [d].
 *  - Device pointers must be 16-byte aligned.  The library never frees or
 *    keeps a caller pointer past the work it enqueues; all work is ordered
 *    on the caller's stream (a cudaStream_t passed as void*; NULL is the
 *    legacy default stream).
 *  - Errors: every entry point returns a pds_status.  PDS_DECLINED means
 *    the call is not one this library serves, decided on the host before
 *    any device work: nothing was enqueued and no buffer was touched
 *    (cuda_prefill.rs, try_cuda_prefill_dense_stack: None before
 *    touching the device or any cache).  PDS_EINVAL is a bad argument.
 *    PDS_ELAUNCH / PDS_ETIMEOUT are failures after admission: output
 *    buffers and cache rows [start_pos, start_pos+B) may have been
 *    written, rows [0, start_pos) never are; the caller must not advance
 *    its cache length.  The message of the last failure on the calling
 *    thread is pds_last_error(); each distinct failure message is also
 *    printed once per process on stderr (cuda_prefill.rs, warn_once).
 *  - One plan may be used by one stream at a time.
 */
#ifndef PDS_H_
#define PDS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pds_status {
  PDS_OK = 0,
  PDS_DECLINED = 1, /* not served; nothing enqueued, nothing touched       */
  PDS_EINVAL = 2,   /* bad pointer, size, alignment or workspace too small */
  PDS_ELAUNCH = 3,  /* a CUDA call failed after admission                  */
  PDS_ETIMEOUT = 4, /* a bounded device-side wait gave up                  */
  PDS_ENOMEM = 5    /* a host or plan-internal device allocation failed    */
} pds_status;

/* RoPE layouts (cuda_prefill.rs, RopeLayoutCuda). */
enum {
  PDS_ROPE_NEOX = 0, /* pair i = channels (i, i + rot_dim/2)  */
  PDS_ROPE_NORM = 1  /* pair i = channels (2i, 2i + 1)        */
};

/*
 * Model dimensions and the run-wide options (cuda_prefill.rs,
 * PrefillParams: n_heads, n_kv_heads, head_dim, rms_eps, attn_softcap,
 * window; LayerRopeCuda: theta, freq_factors, rot_dim, layout, mscale).
 * One rms_eps serves both norms (and the q/k norms); the attention scale
 * is 1/sqrt(head_dim).  Every layer of a run shares the RoPE description,
 * the softcap and the window (a model whose layers differ in them is run as
 * several runs).
 *
 * RoPE: the first rot_dim channels of every q and k head form rot_dim/2
 * pairs (see the layouts); pair i turns by the angle p * omega_i at
 * position p, omega_i = rope_theta^(-2i/rot_dim) / freq_factors[i], and
 * both channels of the pair are multiplied by rope_mscale; channels from
 * rot_dim on pass unchanged.  Softcap: a scaled score z becomes
 * attn_softcap * tanh(z / attn_softcap).  Window: the row at position p
 * sees the keys j with p - window < j <= p.
 *
 * A zero-initialised tail (from rope_layout on) means: Neox over the whole
 * head, no frequency factors, scale 1, no softcap, no window.
 */
typedef struct pds_dims {
  int32_t n_layers;   /* L >= 1                                    */
  int32_t d_model;    /* d: multiple of 128                        */
  int32_t n_heads;    /* H: multiple of n_kv_heads                 */
  int32_t n_kv_heads; /* Hkv                                       */
  int32_t head_dim;   /* hd: 64 or 128; H*hd and Hkv*hd mult. of 128 */
  int32_t ffn_dim;    /* F: multiple of 128                        */
  float rope_theta;   /* > 0                                       */
  float rms_eps;      /* >= 0                                      */
  int32_t rope_layout;        /* PDS_ROPE_NEOX or PDS_ROPE_NORM    */
  int32_t rot_dim;            /* 0 (= head_dim), or a positive multiple of
                                 32 (Neox) / 16 (Norm), <= head_dim */
  const float* freq_factors;  /* host [rot_dim/2] > 0, or NULL (all 1);
                                 copied by pds_plan_create          */
  float rope_mscale;          /* 0 (= 1), or > 0                    */
  float attn_softcap;         /* 0 (none), or > 0                   */
  int32_t window;             /* 0 (none), or > 0 positions         */
} pds_dims;

/*
 * One layer's weights, all device pointers (cuda_prefill.rs,
 * PrefillDenseLayerCuda: attn_norm_w, ffn_norm_w, q, k, v, o, gate, up,
 * down, and the attention extras of AttnExtrasCuda).  The caller owns
 * them; they are read, never written.
 *
 * The extras are optional (NULL: absent), each on its own: a bias is added
 * to its projection's output (after the attention norm's row scale); the
 * q/k norm gains make every head of q / k an RMSNorm of itself,
 * head / sqrt(mean(head^2) + rms_eps) * gain, after the bias and before
 * RoPE.
 */
typedef struct pds_layer {
  const float* attn_norm_w; /* [d]               */
  const float* ffn_norm_w;  /* [d]               */
  const uint16_t* wq;       /* [H*hd,   d]  bf16 */
  const uint16_t* wk;       /* [Hkv*hd, d]  bf16 */
  const uint16_t* wv;       /* [Hkv*hd, d]  bf16 */
  const uint16_t* wo;       /* [d, H*hd]    bf16 */
  const uint16_t* w_gate;   /* [F, d]       bf16 */
  const uint16_t* w_up;     /* [F, d]       bf16 */
  const uint16_t* w_down;   /* [d, F]       bf16 */
  const float* q_bias;      /* [H*hd]   or NULL  */
  const float* k_bias;      /* [Hkv*hd] or NULL  */
  const float* v_bias;      /* [Hkv*hd] or NULL  */
  const float* q_norm;      /* [hd]     or NULL  */
  const float* k_norm;      /* [hd]     or NULL  */
} pds_layer;

typedef struct pds_plan pds_plan;

/*
 * Validate the dimensions and make a plan.
 *
 * Validation is host-only and comes first: PDS_DECLINED (with *out = NULL)
 * for shapes the kernels do not serve (see the field comments of pds_dims)
 * or when the environment variable PDS_DISABLE is set to a non-empty value
 * other than "0" (cuda_prefill.rs: the cuda_dense_enabled() switch), and
 * PDS_EINVAL for a NULL argument or a non-positive size, are decided before
 * any device work.
 *
 * An admitted plan then makes all the device state the library itself
 * allocates, on the device current at this call, which the plan is bound
 * to: a 4-byte status word (cudaMalloc), its 4-byte pinned host copy
 * (cudaMallocHost) and a non-blocking capture stream; PDS_ENOMEM if that
 * fails.  No later call allocates device memory, except that instantiating
 * a CUDA graph of a call (see pds_prefill_dense_stack_device) makes the
 * driver hold memory for its executable graph: at most four per plan, each
 * of 2 + 5 * n_layers kernel nodes, freed by pds_plan_destroy.  Without a
 * CUDA device the plan is host-only: validation and pds_workspace_bytes
 * work, and every call returns PDS_ELAUNCH.
 *
 * Weights are used in place: the kernels read the caller's row-major
 * [out, in] bf16 matrices through TMA tensor maps built at call time
 * (128-byte swizzled boxes straight from the caller's layout), so there is
 * no packing step and no packed copy of the weights.
 */
pds_status pds_plan_create(const pds_dims* dims, pds_plan** out);

/* Release a plan, its device state and its graphs. NULL is a no-op. */
void pds_plan_destroy(pds_plan* plan);

/*
 * Bytes of device workspace for calls with batch <= max_batch and
 * start_pos <= max_start_pos.  The workspace holds the activations between
 * kernels (never the weights or the caches); its content on entry does not
 * matter.  A call needs at least pds_workspace_bytes(plan, batch, 0); what
 * it is given beyond that holds the partial rows of long key ranges, which
 * attention then spreads over all SMs in equal chunks (merged in a fixed
 * order) as far as they fit.  So the schedule, and the rounding of the
 * result, depends on the workspace size: the same inputs with the same
 * workspace size give the same bits.  0 for a NULL plan, max_batch < 1 or
 * max_start_pos < 0.
 */
size_t pds_workspace_bytes(const pds_plan* plan, int32_t max_batch, int32_t max_start_pos);

/*
 * The prefill call, host in / host out (cuda_prefill.rs,
 * try_cuda_prefill_dense_stack and the launch it makes).
 *
 *  layers        host array of n_layers pds_layer (device weight pointers).
 *  k_cache,
 *  v_cache       host arrays of n_layers device pointers, each a bf16 cache
 *                [cache_capacity, n_kv_heads, head_dim].  Rows
 *                [0, start_pos) hold the prefix (K already rotated) and are
 *                only read.  On PDS_OK rows [start_pos, start_pos+batch) hold
 *                this call's new K (post-RoPE) and V rows: these are the
 *                layer's k_rows / v_rows, row b of the batch at row
 *                start_pos+b.
 *  start_pos     s >= 0, the rows already in every cache; new row b is at
 *                position s+b.
 *  batch         B >= 1 new tokens; s+B <= cache_capacity.
 *  hidden_in     host float32 [B, d] (pinned memory makes the copy async
 *                with respect to other host work, pageable also works).
 *  hidden_out    host float32 [B, d]; may alias hidden_in.
 *  workspace     device buffer of >= pds_workspace_bytes(plan, B) bytes.
 *  stream        cudaStream_t as void*.
 *
 * Blocking: returns after the output is in hidden_out (it synchronizes
 * the stream), so device-side timeouts are reported here as PDS_ETIMEOUT.
 */
pds_status pds_prefill_dense_stack(pds_plan* plan, const pds_layer* layers,
                                   uint16_t* const* k_cache, uint16_t* const* v_cache,
                                   int32_t cache_capacity, int32_t start_pos, int32_t batch,
                                   const float* hidden_in, float* hidden_out,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same call with device input and output (float32 [B, d] each, may
 * alias), enqueued on the stream without synchronizing.  A device-side
 * timeout is reported by the next pds_plan_sync (or host-I/O call).
 *
 * Launch mode: the first call with a given set of pointers, start_pos and
 * batch captures all of the call's kernels into a CUDA graph, later calls
 * with the same set replay it (four sets are kept per plan, the least
 * recently used is dropped).  A caller whose pointers change on every call
 * can set the environment variable PDS_GRAPH=0 before pds_plan_create to
 * enqueue the kernels one by one instead; the computation is the same.
 */
pds_status pds_prefill_dense_stack_device(pds_plan* plan, const pds_layer* layers,
                                          uint16_t* const* k_cache, uint16_t* const* v_cache,
                                          int32_t cache_capacity, int32_t start_pos,
                                          int32_t batch, const float* hidden_in_dev,
                                          float* hidden_out_dev, void* workspace,
                                          size_t workspace_bytes, void* stream);

/*
 * Synchronize the stream and report whether any bounded device wait of
 * this plan's earlier calls gave up (PDS_ETIMEOUT; the flag is then
 * cleared) or a CUDA error is pending (PDS_ELAUNCH).
 */
pds_status pds_plan_sync(pds_plan* plan, void* stream);

/* Message of the last failure on the calling thread ("" if none). Valid until the next call on that thread. */
const char* pds_last_error(void);

/*
 * Per-kernel timing (measurement support; no counterpart on the pages).
 * While enabled, every kernel of the plan's calls is bracketed by CUDA
 * events recorded on the call's stream, so each kernel's device duration
 * is measured where it runs.  Off by default (events between kernels cost
 * a little).  pds_plan_kernel_times synchronizes the stream, adds the
 * durations of the calls since the last read to the totals and copies the
 * totals out; reset != 0 clears them afterwards.
 */
enum {
  PDS_KERNEL_PREP = 0,   /* RoPE table + first-layer norm prep, once per call */
  PDS_KERNEL_QKV = 1,    /* QKV GEMM + norm scale + RoPE + K/V row write      */
  PDS_KERNEL_ATTN = 2,   /* GQA causal attention                              */
  PDS_KERNEL_WO = 3,     /* wo GEMM + residual + FFN-norm statistics          */
  PDS_KERNEL_GATEUP = 4, /* gate/up GEMM + SwiGLU                             */
  PDS_KERNEL_DOWN = 5,   /* down GEMM + residual + next-norm statistics       */
  PDS_KERNEL_KINDS = 6
};
typedef struct pds_kernel_times {
  int64_t launches[PDS_KERNEL_KINDS];
  double total_ms[PDS_KERNEL_KINDS];
} pds_kernel_times;

/*
 * Failure-detection self test (no counterpart on the pages), a component
 * entry point like the ones below: enqueues on the stream a one-CTA kernel
 * that waits on an mbarrier nothing ever arrives on, through the same
 * bounded wait every tensor-core kernel of the library uses, with a limit of
 * limit_us microseconds (0 < limit_us <= 10 s, else PDS_EINVAL).  The wait
 * gives up, sets the timeout bit of the component status word and the
 * kernel exits; the next pds_component_sync returns PDS_ETIMEOUT.  Returns
 * PDS_OK once enqueued.
 */
pds_status pds_selftest_stuck_wait(uint32_t limit_us, void* stream);

pds_status pds_plan_set_timing(pds_plan* plan, int32_t enable);
pds_status pds_plan_kernel_times(pds_plan* plan, void* stream, pds_kernel_times* out,
                                 int32_t reset);

/*
 * Component entry points: the stack's kernels one at a time, on device
 * buffers, enqueued on the stream (no synchronization).  They serve the
 * kernel-level tests and take the same shape limits as the stack.  Their
 * kernels' bounded waits report a timeout in a status word of the library
 * (one per device), which pds_component_sync reads.
 */

/*
 * Synchronize the stream, then read and clear the component status words
 * of the current device (those of pds_gemm_bf16, pds_gemm_bf16_noalloc,
 * pds_attention and pds_selftest_stuck_wait).  Returns PDS_ETIMEOUT if a
 * bounded device wait of any of their kernels gave up since the previous
 * pds_component_sync on this device (the output of that call is then not
 * valid), PDS_EINVAL if one of the cached-decoding calls (below) met a
 * sequence length or a parent index that it cannot serve, PDS_ELAUNCH if the
 * stream reports a CUDA error, else PDS_OK.  Allocates nothing.
 */
pds_status pds_component_sync(void* stream);

/*
 * C[M, N] (float32, row-major, ldc = N) = A[M, K] . W[N, K]^T for bf16 A and
 * W (row-major, K contiguous).  M >= 1, N multiple of 128, K multiple of
 * 64.  The same persistent tensor-core GEMM the stack uses, with a plain
 * store epilogue.  `workspace` (device, >= pds_gemm_workspace_bytes(M, N)
 * bytes, 16-byte aligned) holds the partial tiles of the k-split and is
 * written; its content on entry does not matter.
 */
pds_status pds_gemm_bf16(const uint16_t* A, const uint16_t* W, float* C, int32_t M, int32_t N,
                         int32_t K, void* workspace, size_t workspace_bytes, void* stream);

/* Scratch bytes of pds_gemm_bf16 for an M x N output (0 for non-positive sizes). */
size_t pds_gemm_workspace_bytes(int32_t M, int32_t N);

/*
 * pds_gemm_bf16 for callers that cannot allocate device memory: the same
 * product, C[M, N] = A[M, K] . W[N, K]^T, with the same operand rules, but
 * no workspace argument.  The pages have no counterpart; this entry exists
 * for callers that must not call cudaMalloc -- for example a serving
 * process whose device memory is all reserved up front by its own pool,
 * or a plugin that runs inside a host application which owns every
 * allocation -- and so cannot provide the scratch pds_gemm_bf16 takes.
 *
 * The scratch (tile counters and partial tiles of the k-split) lives in a
 * 24 MiB array of the library's own device memory, which every GPU that
 * loads the library holds until the process exits.  Limit: at most 16384
 * output tiles of 128 x 128, i.e. ceil(M/128) * (N/128) <= 16384; larger
 * sizes return PDS_EINVAL with a message and enqueue nothing.  The call
 * allocates nothing (no cudaMalloc, cudaFree or allocating library call).
 *
 * Every call shares the one array and it keeps the last call's contents
 * (the call clears the counters it needs on its stream): calls that overlap
 * on the same GPU, on any streams, race -- order them on one stream or
 * serialize them.  The first call on a device looks up the array's device
 * address for that device (set-up); make that first call before any
 * stream capture.  A device-side timeout of the call is reported by
 * pds_component_sync, which reads and clears the array's status word.
 */
pds_status pds_gemm_bf16_noalloc(const uint16_t* A, const uint16_t* W, float* C, int32_t M,
                                 int32_t N, int32_t K, void* stream);

/*
 * GQA causal attention of B new query rows over a cache (cuda_prefill.rs,
 * PrefillParams: prefix_k/prefix_v, start_pos, attn_scale = 1/sqrt(hd),
 * attn_softcap, window).
 *  q        bf16 [B, H, hd], already rotated (not pre-scaled).
 *  k, v     bf16 [>= start_pos+B, Hkv, hd]; rows [0, start_pos+B) are read.
 *  o        bf16 [B, H*hd]; row b (position p = start_pos + b) attends rows
 *           j <= p, and with window > 0 only p - window < j <= p; query head
 *           h reads kv head h / (H/Hkv).
 *  softcap  0 (none) or > 0: scaled scores z become softcap*tanh(z/softcap).
 *  workspace, workspace_bytes  device scratch for long key ranges (see
 *           pds_attention_workspace_bytes), or NULL and 0.
 * Fails with PDS_DECLINED for hd not in {64, 128} or H % Hkv != 0, and with
 * PDS_EINVAL for a negative softcap or window.
 */
pds_status pds_attention(const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* o,
                         int32_t batch, int32_t start_pos, int32_t n_heads, int32_t n_kv_heads,
                         int32_t head_dim, float softcap, int32_t window, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Workspace bytes with which pds_attention can spread long key ranges over
 * all SMs (its workspace argument; NULL / 0 also works, with long ranges
 * then split over CTA pairs only).  0 for bad sizes.
 */
size_t pds_attention_workspace_bytes(int32_t batch, int32_t start_pos, int32_t n_heads,
                                     int32_t head_dim);

/*
 * Cached decoding: rotary positions, a K/V cache that may hold 8- or 4-bit
 * rows, and attention of a few new tokens per sequence over it (no
 * counterpart on the pages, whose cache is float32 on the host and whose
 * decode is one token at a time).  Component entry points like the ones
 * above: device buffers of the current device, enqueued on the stream
 * without synchronizing, nothing allocated, capturable into a CUDA graph.
 *
 * What only the device can see -- a sequence length that does not fit, a
 * parent that is not an earlier token -- is checked by the kernels before
 * any address is formed from it; the rows concerned are neither read nor
 * written (attention: their output is not written, or zero for a bad
 * parent) and the next pds_component_sync returns PDS_EINVAL.
 */

/*
 * Rotation of head channels by position.  rot_dim, layout, freq_factors and
 * mscale mean what they mean in pds_dims; head_dim is an argument of the
 * calls.  scaling stretches the context:
 *   PDS_ROPE_UNSCALED  omega_i as in pds_dims
 *   PDS_ROPE_LINEAR    omega_i / factor (positions divided by factor)
 *   PDS_ROPE_YARN      omega_i ((1 - r_i) + r_i / factor),
 *                      r_i = clamp((i - lo) / (hi - lo), 0, 1),
 *                      lo = max(0, floor(edge(beta_fast))),
 *                      hi = min(rot_dim - 1, ceil(edge(beta_slow))),
 *                      edge(b) = rot_dim ln(orig_context / (2 pi b)) / (2 ln theta):
 *                      pairs that turn more than beta_fast times within the
 *                      original context keep their frequency, those that turn
 *                      less than beta_slow times are interpolated (hi - lo is
 *                      taken as at least 0.001).  Its usual attention factor
 *                      0.1 ln(factor) + 1 is the caller's to put in mscale.
 */
enum { PDS_ROPE_UNSCALED = 0, PDS_ROPE_LINEAR = 1, PDS_ROPE_YARN = 2 };
typedef struct pds_rope_spec {
  float theta;               /* > 0 (YaRN: > 1)                            */
  int32_t layout;            /* PDS_ROPE_NEOX or PDS_ROPE_NORM             */
  int32_t rot_dim;           /* 0 (= head_dim), or a positive multiple of
                                16, <= head_dim                            */
  int32_t scaling;           /* PDS_ROPE_UNSCALED / _LINEAR / _YARN        */
  const float* freq_factors; /* host [rot_dim/2] > 0, or NULL; not kept    */
  float mscale;              /* 0 (= 1), or > 0                            */
  float factor;              /* LINEAR, YARN: > 0                          */
  int32_t orig_context;      /* YARN: > 0                                  */
  float beta_fast;           /* YARN: > beta_slow                          */
  float beta_slow;           /* YARN: > 0                                  */
} pds_rope_spec;

/*
 * y = the rows of x turned at their positions: bf16 [rows, n_heads, head_dim]
 * with head_dim a multiple of 16 up to 256; row r of x starts at element
 * r * x_stride, of y at r * y_stride (0: packed, n_heads * head_dim; multiples
 * of 8, no smaller than packed).  y may be x (same stride), else they must not
 * overlap.  Row r is at position positions[r] (device int32, may be negative)
 * or, with positions NULL, start_pos + r.  inverse != 0 turns the other way:
 * for mscale 1 it undoes the rotation, and for any mscale it is the
 * transpose, i.e. the gradient with respect to x of a loss whose gradient
 * with respect to y is given as x.  A position's angle is exact to 2^-31 of a
 * turn but for the frequency, which is float64 arithmetic: off by at most 2^-48 of
 * itself, so the angle by that part of the turns made until there (2^-30 of a turn
 * at position 2^20, 2^-19 at 2^31).  The products are float32, rounded once to bf16.
 */
pds_status pds_rope(const pds_rope_spec* spec, const uint16_t* x, uint16_t* y, int32_t rows,
                    int32_t n_heads, int32_t head_dim, int64_t x_stride, int64_t y_stride,
                    const int32_t* positions, int32_t start_pos, int32_t inverse, void* stream);

/*
 * A K/V cache of n_seqs sequences (one layer's).  The row of sequence s, row
 * j and kv head g starts at element s seq_stride + j row_stride +
 * g head_stride of k / v (all three 0: packed [n_seqs, capacity, n_kv_heads,
 * head_dim]; an "element" is one channel, so half a byte for PDS_KV_INT4; every
 * stride a multiple of 16 bytes and no smaller than a head's row).  Strides that
 * let rows overlap are refused: each has to step over all that the smaller ones
 * span.  The head's channels are contiguous.  A cache of pds_prefill_dense_stack
 * is the PDS_KV_BF16 cache with n_seqs = 1.
 *
 * Formats:
 *   PDS_KV_BF16  the values, bf16.
 *   PDS_KV_E4M3  a byte per channel, 1-4-3 floating point (bias 7, largest
 *                448); scale word: the float32 scale.  A row x of a head
 *                is stored as scale = max|x| / 448, code = x / scale rounded to
 *                nearest even; it stands for code * scale.
 *   PDS_KV_INT4  two channels per byte (even channel in the low nibble);
 *                scale word: bits 31..16 the scale in bf16, bits 3..0 the zero
 *                point z, the rest 0.  lo = min(0, min x), hi = max(0, max x),
 *                scale = hi/15 - lo/15, z = rint(-lo / scale) and code =
 *                rint(x / scale) + z, both limited to 0..15; it stands for
 *                (code - z) * scale.
 * A row whose scale would be below the smallest normal float32 is stored as
 * zeros (scale 0); a row with an infinity or a NaN has a NaN scale and
 * stands for NaN throughout (codes of NaN are never stored, and mean nothing).  The scale words of sequence s, kv head g and
 * row j sit at [(s n_kv_heads + g) capacity + j].
 *
 * lens[s] is the number of cached rows of sequence s before the call.  The
 * calls never change it: the caller advances it (on the device) by the
 * tokens it keeps.
 */
enum { PDS_KV_BF16 = 0, PDS_KV_E4M3 = 1, PDS_KV_INT4 = 2 };
typedef struct pds_cache {
  int32_t format;
  int32_t n_seqs;     /* 1 .. 4096                                      */
  int32_t capacity;   /* rows per sequence, >= 1                        */
  int32_t n_kv_heads;
  int32_t head_dim;   /* 64 or 128                                      */
  int32_t reserved;   /* 0                                              */
  int64_t seq_stride, row_stride, head_stride; /* elements; all 0: packed */
  void* k;
  void* v;
  uint32_t* k_scale;  /* device [n_seqs, n_kv_heads, capacity]; unused  */
  uint32_t* v_scale;  /*   (may be NULL) for PDS_KV_BF16                */
  const int32_t* lens; /* device [n_seqs]                               */
} pds_cache;

/*
 * Drafted tokens.  n_tokens tokens per sequence sit at rows lens[s] ..
 * lens[s] + n_tokens - 1.  parents, device int32 [n_seqs, n_tokens], makes
 * them a forest: parents[t] is the index of t's parent among the sequence's
 * tokens (smaller than t), -1 for a root, below -1 for a padding token
 * (whose row is not written, and whose output is zero).  parents NULL is the
 * chain t -> t - 1: a decode step, or a run of tokens of the sequence.  A
 * token's depth is the number of its ancestors and its position
 * lens[s] + depth.  At most 256 tokens with parents.
 */

/*
 * Store n_tokens new K and V rows of every sequence: bf16 input, token t of
 * sequence s at element (s n_tokens + t) * k_stride (v_stride) of k (v),
 * [n_kv_heads, head_dim] each (stride 0: packed; multiples of 8).  With spec
 * not NULL the K rows are rotated first, at the tokens' positions or at
 * positions[s n_tokens + t] (device) where given; the rotated values are
 * quantised from float32 (PDS_KV_BF16: rounded to bf16).  Rows other than the
 * new ones are left as they are.
 */
pds_status pds_cache_write(const pds_cache* cache, const pds_rope_spec* spec, const uint16_t* k,
                           const uint16_t* v, int32_t n_tokens, int64_t k_stride,
                           int64_t v_stride, const int32_t* parents, const int32_t* positions,
                           void* stream);

/*
 * Rows back as bf16 (the value a row stands for, rounded once):
 * k_out, v_out [n_seqs, rows, n_kv_heads, head_dim], either may be NULL.
 * first_row >= 0: rows first_row .. first_row + rows - 1, those below
 * lens[s]; the rest of the output is left as it is.  first_row ==
 * PDS_AT_LENS: the rows lens[s] .. lens[s] + rows - 1 that a write of `rows`
 * tokens stored.
 */
enum { PDS_AT_LENS = -1 };
pds_status pds_cache_read(const pds_cache* cache, int32_t first_row, int32_t rows,
                          uint16_t* k_out, uint16_t* v_out, void* stream);

/*
 * GQA attention of the n_tokens new tokens of every sequence (already
 * written) over its cache: token t sees the lens[s] cached rows, its
 * ancestors and itself; with window > 0 only those whose position (a cached
 * row's is its index) is above its own less window.  Scores, softcap and the
 * head groups as in pds_attention; the softmax's statistics are float32.  The
 * weights that go into the products with V are rounded, to bf16 (2^-8 of each at
 * most) over a bf16 cache and to fp16 (2^-11) over codes; the sum that divides them is
 * not.  Over codes a weight times its V scale is held in fp16: what is lost below
 * its smallest steps is under 2^-27 of the token's largest such product per key,
 * as long as the V scales lie within 2^80 of each other.
 *  q, o     bf16, token t of sequence s at element (s n_tokens + t) * q_stride
 *           (o_stride), [n_heads, head_dim] each (0: packed; multiples of 8).
 *           o may not overlap q (the same buffer is refused).
 *  n_tokens 1 .. 256; n_heads a multiple of n_kv_heads, at most 8192.
 *  max_len  an upper bound of lens known on the host, or 0 (the capacity less
 *           n_tokens); sizes the launch, not the result's meaning.  A longer
 *           sequence is refused as one that does not fit.
 *  workspace  >= pds_attention_tree_workspace_bytes(...) bytes, so that key
 *           ranges are split over all SMs, or NULL and 0 (long ranges stay on
 *           one SM each).  Its content on entry does not matter; calls that may run at
 *           the same time need one each.  How ranges are split, and so the
 *           rounding of the result, depends on whether there is one, on
 *           max_len and on lens; the same call on the same inputs gives the
 *           same bits.
 * A row that sees no key (padding) is zero.  An infinity or a NaN in a row
 * that a token does not see does not reach its output, nor does a finite value of
 * any size, nor another token's query (a padding token's may hold anything).
 */
pds_status pds_attention_tree(const pds_cache* cache, const uint16_t* q, uint16_t* o,
                              int32_t n_tokens, int32_t n_heads, int64_t q_stride,
                              int64_t o_stride, const int32_t* parents, float softcap,
                              int32_t window, int32_t max_len, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Workspace bytes of pds_attention_tree on the current device (0 for bad sizes or without one). */
size_t pds_attention_tree_workspace_bytes(const pds_cache* cache, int32_t n_tokens,
                                          int32_t n_heads);

/*
 * A paged K/V cache: one pool of pages for many sequences (one layer's), a page
 * holding page_size consecutive rows of one sequence for all kv heads.  A sequence
 * takes pages as it grows, so the memory held follows the rows there are and not
 * the longest sequence there may be.  Component entry points like those of cached
 * decoding, whose row formats, scale words and rotations they share.
 *
 * Row r (of page_size) and kv head g of page p start at element p page_stride +
 * r row_stride + g head_stride of k / v (all three 0: packed [n_pages,
 * n_kv_heads, page_size, head_dim]; elements, multiples and overlap as for
 * pds_cache), their scale words are at [(p n_kv_heads + g) page_size + r], 16-byte
 * aligned arrays.  Row j of sequence s is row j % page_size of page table[s
 * max_pages + j / page_size], and page_size p + r is the slot of row r of page p.
 * Tables may share pages among sequences, and may be the caller's own: only
 * reserve and release use held, free_pages and n_free (elsewhere they may be
 * NULL).  held[s] counts the pages that sequence s has; free_pages[0 .. n_free)
 * are the pages that nobody has, taken from the end.
 *
 * lens[s] is the number of rows of sequence s before its new ones.  The calls never
 * change it.  What only the device can see is checked there, nothing is read or
 * written through a number that fails, and the next pds_component_sync returns
 * PDS_EINVAL: a length or a count that is negative or that the table has no room
 * for, a table entry or a slot that is no page, fewer free pages than needed.
 */
typedef struct pds_pages {
  int32_t format;     /* PDS_KV_BF16 / _E4M3 / _INT4                    */
  int32_t n_seqs;     /* 1 .. 4096                                      */
  int32_t n_pages;    /* n_pages page_size < 2^31                       */
  int32_t page_size;  /* 8, 16, 32 ... 1024                             */
  int32_t max_pages;  /* width of the table; times page_size <= 2^30    */
  int32_t n_kv_heads; /* 1 .. 1024                                      */
  int32_t head_dim;   /* 64 or 128                                      */
  int32_t reserved;   /* 0                                              */
  int64_t page_stride, row_stride, head_stride; /* elements; all 0: packed */
  void* k;
  void* v;
  uint32_t* k_scale;   /* device; unused (may be NULL) for PDS_KV_BF16   */
  uint32_t* v_scale;
  int32_t* table;      /* device [n_seqs, max_pages]                     */
  int32_t* held;       /* device [n_seqs]                                */
  const int32_t* lens; /* device [n_seqs]                                */
  int32_t* free_pages; /* device [n_pages]                               */
  int32_t* n_free;     /* device [1]                                     */
} pds_pages;

/*
 * Pages for new_rows[s] >= 0 rows (device [n_seqs]) of every sequence behind its
 * lens[s], and the map of those rows.  A sequence that holds fewer than
 * ceil((lens + new_rows) / page_size) pages takes the missing ones: the sequences in
 * order, each page the last free one.  The new rows of all sequences are numbered
 * in order: sequence s's are starts[s] .. starts[s + 1] - 1 (starts: device
 * [n_seqs + 1]); slots[t] is row t's slot and positions[t] (may be NULL) its
 * position, lens[s] + t - starts[s]; both have n_rows >= 0 entries, those behind
 * the last row are -1 and 0.  Where a number is refused, the rows are more than
 * n_rows or the free pages fewer than needed, nothing is taken, and the map is
 * empty (starts 0, slots -1).
 */
pds_status pds_pages_reserve(const pds_pages* pages, const int32_t* new_rows, int32_t n_rows,
                             int32_t* slots, int32_t* positions, int32_t* starts, void* stream);

/*
 * The same map of rows first[s] .. first[s] + count[s] - 1 that the sequences
 * have (pages held for all of them, where held is given); nothing is taken.
 * positions and starts may be NULL.
 */
pds_status pds_pages_slots(const pds_pages* pages, const int32_t* first, const int32_t* count,
                           int32_t n_rows, int32_t* slots, int32_t* positions, int32_t* starts,
                           void* stream);

/*
 * Every sequence keeps the pages of its first keep[s] >= 0 rows (or those it has, if
 * fewer) and the others become free: of all pages let go, the sequences and their
 * pages in order, the first is the last free one, so that a release undoes a
 * reserve.  Table entries stay as they are.  Pages that several sequences share
 * are the caller's to count: they must not be let go by each.
 */
pds_status pds_pages_release(const pds_pages* pages, const int32_t* keep, void* stream);

/*
 * Store n_rows K and V rows (bf16, row t at element t * k_stride (v_stride), [n_kv_heads,
 * head_dim]; 0: packed, multiples of 8) at slots[t] (device); a slot of -1 leaves its
 * row out.  With spec not NULL the K rows are rotated first, at positions[t]
 * (device).  The rows are stored as pds_cache_write stores them, bit for bit.
 * No two rows of a call may have the same slot.
 */
pds_status pds_pages_write(const pds_pages* pages, const pds_rope_spec* spec, const uint16_t* k,
                           const uint16_t* v, const int32_t* slots, int32_t n_rows, int64_t k_stride,
                           int64_t v_stride, const int32_t* positions, void* stream);

/*
 * The rows at slots[0 .. n_rows) (device) back as bf16 (the value a row stands for, rounded
 * once): k_out, v_out [n_rows, n_kv_heads, head_dim], either may be NULL.  A slot of -1
 * leaves its row of the output as it is.
 */
pds_status pds_pages_read(const pds_pages* pages, const int32_t* slots, int32_t n_rows,
                          uint16_t* k_out, uint16_t* v_out, void* stream);

/*
 * GQA attention of one token per sequence, its last: sequence s's sees the rows
 * j < n = lens[s] + new_rows[s] (new_rows NULL: 1 each), with window > 0 only
 * j >= n - window.  Scores, softcap and head groups as in pds_attention.  A sequence
 * with new_rows[s] == 0 has no token: its output is zero; one whose numbers are
 * refused: its output is not written.  A page of the table that is none stands for rows of
 * zeros (and is reported).
 *  q, o     bf16, sequence s at element s * q_stride (o_stride), [n_heads, head_dim]
 *           (0: packed; multiples of 8); o may not overlap q.
 *  n_heads  a multiple of n_kv_heads, at most 8192.
 *  workspace  >= pds_pages_attend_workspace_bytes(...) bytes, 16-byte aligned; its content
 *           on entry does not matter; calls that may run at the same time need one each.
 * The softmax's statistics and the sums are float32; a row's output is rounded to bf16 once.
 * Over bf16 rows a weight enters its product as two bf16 numbers, off by 2^-16 of itself.
 * Over codes the query enters as two 8-bit numbers per channel: exact down to 2^-13 of the head's
 * largest, off by at most 2^-21 of that largest below; and a weight times its row's V scale is
 * rounded to fp16 (2^-11 of itself), and off by at most 2^-25 of the largest such product where it is
 * far smaller, as long as the V scales that the token sees lie within 2^80 of each other; a row whose V
 * scale is 0 counts there as one of 2^-80 of the first other's.
 * Rows that a token does not see may hold anything: infinities and NaN there, in scale words
 * too, do not reach its output.  A token all of whose scores are -infinity is NaN.
 * How sequences are cut over the GPU goes by the lengths that there may be, max_pages page_size or the
 * window, besides those there are: a short sequence costs up to 2.4 us more in a wide table, and its last
 * bits may differ.  The same call on the same inputs gives the same bits.
 */
pds_status pds_pages_attend(const pds_pages* pages, const int32_t* new_rows, const uint16_t* q,
                            uint16_t* o, int32_t n_heads, int64_t q_stride, int64_t o_stride,
                            float softcap, int32_t window, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Workspace bytes of pds_pages_attend on the current device (0 for bad sizes or without one). */
size_t pds_pages_attend_workspace_bytes(const pds_pages* pages, int32_t n_heads);

#ifdef __cplusplus
}
#endif

#endif /* PDS_H_ */
