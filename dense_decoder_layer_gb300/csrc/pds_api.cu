// Host side of the C ABI: validation and declines, workspace layout, the
// per-call enqueue of the layer loop, error reporting.
//
// The call shape follows frink-models 0.29.0 src/decoder/cuda_prefill.rs
// (try_cuda_prefill_dense_stack / cuda_prefill_layer): refusals are
// decided on the host before any device work; one enqueue covers the whole
// run of layers; the hidden batch crosses host<->device once each way; a
// failure after admission is reported once per distinct message.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <set>
#include <string>
#include <vector>

#include "../../include/pds.h"
#include "facts.h"
#include "kernels.h"
#include "kv.h"
#include "plan.h"
#include "tc.h"

namespace {

thread_local std::string t_last_error;

void warn_once(const std::string& msg) {
  static std::mutex mu;
  static std::set<std::string> seen;
  std::lock_guard<std::mutex> g(mu);
  if (seen.insert(msg).second) std::fprintf(stderr, "%s\n", msg.c_str());
}

pds_status fail(pds_status st, const std::string& msg) {
  t_last_error = msg;
  if (st == PDS_ELAUNCH || st == PDS_ETIMEOUT || st == PDS_ENOMEM)
    warn_once("pds: prefill stack failed after admission: " + msg);
  return st;
}

bool env_flag(const char* name) {
  const char* v = std::getenv(name);
  return v && *v && std::strcmp(v, "0") != 0;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

namespace pds {

Layout make_layout(const Plan& p, int B) {
  Layout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  const size_t Bz = (size_t)B;
  const int d = p.dims.d_model;
  L.x = take(Bz * d * 4);
  L.h = take(Bz * d * 4);
  L.a = take(Bz * d * 2);
  L.ss_attn = take(Bz * (d / 64) * 4);
  L.ss_ffn = take(Bz * (d / 64) * 4);
  L.q = take(Bz * p.q_width * 2);
  L.o = take(Bz * p.q_width * 2);
  L.act = take(Bz * p.dims.ffn_dim * 2);
  L.rope = take(Bz * (p.dims.head_dim / 2) * 8);
  L.gemm_ws = take(gemm_workspace_bytes(p, B));
  L.attn = off;
  L.total = off;
  return L;
}

size_t workspace_bytes(const Plan& p, int B, int s_max) {
  const Layout L = make_layout(p, B);
  return L.attn + align_up(tc_attention_scratch_bytes(B, s_max, p.dims.n_heads,
                                                      p.dims.head_dim), 256);
}

}  // namespace pds

using pds::Plan;

struct pds_plan : Plan {};

extern "C" {

const char* pds_last_error(void) { return t_last_error.c_str(); }

pds_status pds_plan_create(const pds_dims* dims, pds_plan** out) {
  if (!out) return fail(PDS_EINVAL, "pds_plan_create: out is NULL");
  *out = nullptr;
  if (!dims) return fail(PDS_EINVAL, "pds_plan_create: dims is NULL");
  const pds_dims& d = *dims;
  if (d.n_layers < 1 || d.d_model < 1 || d.n_heads < 1 || d.n_kv_heads < 1 || d.head_dim < 1 ||
      d.ffn_dim < 1)
    return fail(PDS_EINVAL, "pds_plan_create: every dimension must be positive");
  if (!(d.rope_theta > 0.f) || !(d.rms_eps >= 0.f) || !std::isfinite(d.rope_theta) ||
      !std::isfinite(d.rms_eps))
    return fail(PDS_EINVAL, "pds_plan_create: rope_theta must be > 0 and rms_eps >= 0");
  if (env_flag("PDS_DISABLE")) return fail(PDS_DECLINED, "declined: PDS_DISABLE is set");
  if (d.n_heads % d.n_kv_heads != 0)
    return fail(PDS_DECLINED, "declined: n_heads is not a multiple of n_kv_heads");
  if (d.head_dim != 64 && d.head_dim != 128)
    return fail(PDS_DECLINED, "declined: head_dim must be 64 or 128");
  if (d.d_model % 128 != 0 || d.ffn_dim % 128 != 0)
    return fail(PDS_DECLINED, "declined: d_model and ffn_dim must be multiples of 128");
  if ((d.n_heads * d.head_dim) % 128 != 0 || (d.n_kv_heads * d.head_dim) % 128 != 0)
    return fail(PDS_DECLINED, "declined: n_heads*head_dim and n_kv_heads*head_dim must be multiples of 128");
  // run-wide RoPE and attention options
  if (d.rope_layout != PDS_ROPE_NEOX && d.rope_layout != PDS_ROPE_NORM)
    return fail(PDS_EINVAL, "pds_plan_create: rope_layout must be PDS_ROPE_NEOX or PDS_ROPE_NORM");
  if (d.rot_dim < 0 || d.rot_dim > d.head_dim || d.rot_dim % 2)
    return fail(PDS_EINVAL, "pds_plan_create: rot_dim must be 0 or even and <= head_dim");
  const int rot = d.rot_dim ? d.rot_dim : d.head_dim;
  if (rot % (d.rope_layout == PDS_ROPE_NEOX ? 32 : 16) != 0)
    return fail(PDS_DECLINED, "declined: rot_dim must be a multiple of 32 (Neox) or 16 (Norm)");
  if (!std::isfinite(d.rope_mscale) || d.rope_mscale < 0.f)
    return fail(PDS_EINVAL, "pds_plan_create: rope_mscale must be 0 or > 0");
  if (!std::isfinite(d.attn_softcap) || d.attn_softcap < 0.f)
    return fail(PDS_EINVAL, "pds_plan_create: attn_softcap must be 0 or > 0");
  if (d.window < 0) return fail(PDS_EINVAL, "pds_plan_create: window must be >= 0");
  if (d.freq_factors)
    for (int i = 0; i < rot / 2; ++i)
      if (!(d.freq_factors[i] > 0.f) || !std::isfinite(d.freq_factors[i]))
        return fail(PDS_EINVAL, "pds_plan_create: freq_factors must be finite and > 0");
  pds_plan* p = new (std::nothrow) pds_plan();
  if (!p) return fail(PDS_ENOMEM, "pds_plan_create: out of host memory");
  p->dims = d;
  p->dims.freq_factors = nullptr;  // the caller's array is not kept
  p->q_width = d.n_heads * d.head_dim;
  p->kv_width = d.n_kv_heads * d.head_dim;
  p->rope_layout = d.rope_layout;
  p->rot_dim = rot;
  // omega_i = theta^(-2i/rot_dim) / freq_factors[i], in float64
  // (cuda_prefill.rs, LayerRopeCuda: theta, freq_factors, rot_dim)
  p->omega.resize(rot / 2);
  for (int i = 0; i < rot / 2; ++i)
    p->omega[i] = std::pow(static_cast<double>(d.rope_theta), -2.0 * i / rot) /
                  (d.freq_factors ? static_cast<double>(d.freq_factors[i]) : 1.0);
  p->rope_mscale = d.rope_mscale > 0.f ? d.rope_mscale : 1.0f;
  p->attn_softcap = d.attn_softcap;
  p->window = d.window;
  const char* g = std::getenv("PDS_GRAPH");
  p->graphs = !(g && std::strcmp(g, "0") == 0);
  // The plan's device state, on the current device, once the shape is
  // admitted; without a CUDA device the plan stays host-only.
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) == cudaSuccess && ndev > 0) {
    std::string err;
    const pds_status st = pds::plan_attach_device(*p, &err);
    if (st != PDS_OK) {
      delete p;
      return fail(st, err);
    }
  } else {
    cudaGetLastError();
  }
  *out = p;
  return PDS_OK;
}

void pds_plan_destroy(pds_plan* plan) {
  if (!plan) return;
  pds::plan_release_device(*plan);
  delete plan;
}

size_t pds_workspace_bytes(const pds_plan* plan, int32_t max_batch, int32_t max_start_pos) {
  if (!plan || max_batch < 1 || max_start_pos < 0) return 0;
  return pds::workspace_bytes(*plan, max_batch, max_start_pos);
}

static pds_status check_call(pds_plan* plan, const pds_layer* layers, uint16_t* const* kc,
                             uint16_t* const* vc, int32_t cap, int32_t s, int32_t B,
                             const void* in, const void* out, void* ws, size_t ws_bytes,
                             bool device_io) {
  if (!plan) return fail(PDS_EINVAL, "plan is NULL");
  if (!layers || !kc || !vc) return fail(PDS_EINVAL, "layers / k_cache / v_cache is NULL");
  if (!in || !out) return fail(PDS_EINVAL, "hidden_in / hidden_out is NULL");
  if (B < 1) return fail(PDS_EINVAL, "batch must be >= 1");
  if (s < 0) return fail(PDS_EINVAL, "start_pos must be >= 0");
  if ((int64_t)s + B > cap)
    return fail(PDS_DECLINED, "declined: start_pos + batch exceeds the cache capacity");
  if (!ws) return fail(PDS_EINVAL, "workspace is NULL");
  if (!aligned16(ws)) return fail(PDS_EINVAL, "workspace is not 16-byte aligned");
  if (ws_bytes < pds::make_layout(*plan, B).total)
    return fail(PDS_EINVAL, "workspace is smaller than pds_workspace_bytes(plan, batch, 0)");
  if (device_io && (!aligned16(in) || !aligned16(out)))
    return fail(PDS_EINVAL, "device hidden_in / hidden_out not 16-byte aligned");
  for (int l = 0; l < plan->dims.n_layers; ++l) {
    const pds_layer& w = layers[l];
    const void* ptrs[] = {w.attn_norm_w, w.ffn_norm_w, w.wq, w.wk, w.wv,
                          w.wo,          w.w_gate,     w.w_up, w.w_down, kc[l], vc[l]};
    for (const void* q : ptrs) {
      if (!q) return fail(PDS_EINVAL, "layer " + std::to_string(l) + ": NULL weight or cache");
      if (!aligned16(q))
        return fail(PDS_EINVAL, "layer " + std::to_string(l) + ": pointer not 16-byte aligned");
    }
    for (const void* q : {(const void*)w.q_bias, (const void*)w.k_bias, (const void*)w.v_bias,
                          (const void*)w.q_norm, (const void*)w.k_norm})
      if (q && !aligned16(q))
        return fail(PDS_EINVAL,
                    "layer " + std::to_string(l) + ": extra (bias / norm) not 16-byte aligned");
  }
  // Fault injection for the callers' failure handling: the call is admitted,
  // then fails as a launch would, before any device work.
  if (env_flag("PDS_FAULT_AFTER_ADMIT"))
    return fail(PDS_ELAUNCH, "injected failure after admission (PDS_FAULT_AFTER_ADMIT)");
  return PDS_OK;
}

pds_status pds_prefill_dense_stack_device(pds_plan* plan, const pds_layer* layers,
                                          uint16_t* const* k_cache, uint16_t* const* v_cache,
                                          int32_t cache_capacity, int32_t start_pos,
                                          int32_t batch, const float* hidden_in_dev,
                                          float* hidden_out_dev, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  pds_status st = check_call(plan, layers, k_cache, v_cache, cache_capacity, start_pos, batch,
                             hidden_in_dev, hidden_out_dev, workspace, workspace_bytes, true);
  if (st != PDS_OK) return st;
  std::string err;
  st = pds::run_stack(*plan, layers, k_cache, v_cache, start_pos, batch, hidden_in_dev,
                      hidden_out_dev, static_cast<char*>(workspace), workspace_bytes,
                      static_cast<cudaStream_t>(stream), &err);
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

pds_status pds_prefill_dense_stack(pds_plan* plan, const pds_layer* layers,
                                   uint16_t* const* k_cache, uint16_t* const* v_cache,
                                   int32_t cache_capacity, int32_t start_pos, int32_t batch,
                                   const float* hidden_in, float* hidden_out, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  pds_status st = check_call(plan, layers, k_cache, v_cache, cache_capacity, start_pos, batch,
                             hidden_in, hidden_out, workspace, workspace_bytes, false);
  if (st != PDS_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const pds::Layout lay = pds::make_layout(*plan, batch);
  float* xdev = reinterpret_cast<float*>(static_cast<char*>(workspace) + lay.x);
  const size_t bytes = (size_t)batch * plan->dims.d_model * sizeof(float);
  cudaError_t ce = cudaMemcpyAsync(xdev, hidden_in, bytes, cudaMemcpyHostToDevice, s);
  if (ce != cudaSuccess)
    return fail(PDS_ELAUNCH, std::string("upload of hidden_in: ") + cudaGetErrorString(ce));
  std::string err;
  st = pds::run_stack(*plan, layers, k_cache, v_cache, start_pos, batch, xdev, xdev,
                      static_cast<char*>(workspace), workspace_bytes, s, &err);
  if (st != PDS_OK) return fail(st, err);
  ce = cudaMemcpyAsync(hidden_out, xdev, bytes, cudaMemcpyDeviceToHost, s);
  if (ce != cudaSuccess)
    return fail(PDS_ELAUNCH, std::string("download of hidden_out: ") + cudaGetErrorString(ce));
  return pds_plan_sync(plan, stream);
}

pds_status pds_plan_sync(pds_plan* plan, void* stream) {
  if (!plan) return fail(PDS_EINVAL, "plan is NULL");
  std::string err;
  pds_status st = pds::plan_sync(*plan, static_cast<cudaStream_t>(stream), &err);
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

pds_status pds_selftest_stuck_wait(uint32_t limit_us, void* stream) {
  if (limit_us == 0 || limit_us > 10000000u)
    return fail(PDS_EINVAL, "pds_selftest_stuck_wait: limit_us must be in (0, 10 s]");
  std::string err;
  pds_status st = pds::run_stuck_wait(limit_us, static_cast<cudaStream_t>(stream), &err);
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

pds_status pds_component_sync(void* stream) {
  std::string err;
  pds_status st = pds::component_sync(static_cast<cudaStream_t>(stream), &err);
  if (st == PDS_ETIMEOUT) {
    t_last_error = err;  // reported to the caller, who asked for it
    return st;
  }
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

pds_status pds_plan_set_timing(pds_plan* plan, int32_t enable) {
  if (!plan) return fail(PDS_EINVAL, "plan is NULL");
  plan->timing = enable != 0;
  return PDS_OK;
}

pds_status pds_plan_kernel_times(pds_plan* plan, void* stream, pds_kernel_times* out,
                                 int32_t reset) {
  if (!plan || !out) return fail(PDS_EINVAL, "plan or out is NULL");
  std::string err;
  pds_status st =
      pds::plan_kernel_times(*plan, static_cast<cudaStream_t>(stream), out, reset != 0, &err);
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

size_t pds_gemm_workspace_bytes(int32_t M, int32_t N) {
  if (M < 1 || N < 1) return 0;
  return pds::tc_gemm_scratch_bytes(M, (N + 127) / 128);
}

pds_status pds_gemm_bf16(const uint16_t* A, const uint16_t* W, float* C, int32_t M, int32_t N,
                         int32_t K, void* workspace, size_t workspace_bytes, void* stream) {
  if (!A || !W || !C || !workspace) return fail(PDS_EINVAL, "pds_gemm_bf16: NULL operand");
  if (M < 1 || N < 128 || K < 64) return fail(PDS_EINVAL, "pds_gemm_bf16: bad size");
  if (N % 128 || K % 64)
    return fail(PDS_DECLINED, "declined: pds_gemm_bf16 needs N % 128 == 0 and K % 64 == 0");
  if (!aligned16(A) || !aligned16(W) || !aligned16(C) || !aligned16(workspace))
    return fail(PDS_EINVAL, "pds_gemm_bf16: operand not 16-byte aligned");
  if (workspace_bytes < pds_gemm_workspace_bytes(M, N))
    return fail(PDS_EINVAL, "pds_gemm_bf16: workspace smaller than pds_gemm_workspace_bytes");
  std::string err;
  pds_status st = pds::run_gemm_plain(A, W, C, M, N, K, static_cast<char*>(workspace),
                                      workspace_bytes, static_cast<cudaStream_t>(stream), &err);
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

pds_status pds_gemm_bf16_noalloc(const uint16_t* A, const uint16_t* W, float* C, int32_t M,
                                 int32_t N, int32_t K, void* stream) {
  if (!A || !W || !C) return fail(PDS_EINVAL, "pds_gemm_bf16_noalloc: NULL operand");
  if (M < 1 || N < 128 || K < 64) return fail(PDS_EINVAL, "pds_gemm_bf16_noalloc: bad size");
  if (N % 128 || K % 64)
    return fail(PDS_DECLINED,
                "declined: pds_gemm_bf16_noalloc needs N % 128 == 0 and K % 64 == 0");
  if (!aligned16(A) || !aligned16(W) || !aligned16(C))
    return fail(PDS_EINVAL, "pds_gemm_bf16_noalloc: operand not 16-byte aligned");
  const size_t tiles = static_cast<size_t>((M + 127) / 128) * (N / 128);
  if (tiles > pds::tc_gemm_noalloc_max_tiles())
    return fail(PDS_EINVAL, "pds_gemm_bf16_noalloc: ceil(M/128) * (N/128) = " +
                                std::to_string(tiles) + " output tiles, more than the " +
                                std::to_string(pds::tc_gemm_noalloc_max_tiles()) +
                                " its static scratch holds");
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return fail(PDS_ELAUNCH, "pds_gemm_bf16_noalloc: no CUDA device");
  std::string err;
  pds_status st = pds::tc_gemm_plain_noalloc(A, W, C, M, N, K, sms,
                                             static_cast<cudaStream_t>(stream), &err);
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

size_t pds_attention_workspace_bytes(int32_t batch, int32_t start_pos, int32_t n_heads,
                                     int32_t head_dim) {
  if (batch < 1 || start_pos < 0 || n_heads < 1 || (head_dim != 64 && head_dim != 128)) return 0;
  return pds::tc_attention_scratch_bytes(batch, start_pos, n_heads, head_dim);
}

pds_status pds_attention(const uint16_t* q, const uint16_t* k, const uint16_t* v, uint16_t* o,
                         int32_t batch, int32_t start_pos, int32_t n_heads, int32_t n_kv_heads,
                         int32_t head_dim, float softcap, int32_t window, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o) return fail(PDS_EINVAL, "pds_attention: NULL operand");
  if (batch < 1 || start_pos < 0 || n_heads < 1 || n_kv_heads < 1)
    return fail(PDS_EINVAL, "pds_attention: bad size");
  if (!(softcap >= 0.f) || !std::isfinite(softcap) || window < 0)
    return fail(PDS_EINVAL, "pds_attention: softcap and window must be >= 0");
  if (n_heads % n_kv_heads != 0 || (head_dim != 64 && head_dim != 128))
    return fail(PDS_DECLINED, "declined: pds_attention needs H % Hkv == 0 and hd in {64, 128}");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (workspace && !aligned16(workspace)))
    return fail(PDS_EINVAL, "pds_attention: operand not 16-byte aligned");
  if (!workspace) workspace_bytes = 0;
  std::string err;
  pds_status st = pds::run_attention(q, k, v, o, batch, start_pos, n_heads, n_kv_heads, head_dim,
                                     softcap, window, static_cast<char*>(workspace),
                                     workspace_bytes, static_cast<cudaStream_t>(stream), &err);
  if (st != PDS_OK) return fail(st, err);
  return PDS_OK;
}

// ------------------------------------------------------ cached decoding

namespace {

// The turns of a spec's pairs; false (with a message) for a bad one.  A null
// spec is no rotation.
pds_status make_turns(const char* fn, const pds_rope_spec* spec, int hd, bool inverse,
                      pds::RopeTurns* r) {
  *r = pds::RopeTurns{};
  if (!spec) return PDS_OK;
  const pds_rope_spec& p = *spec;
  const std::string name = fn;
  if (!(p.theta > 0.f) || !std::isfinite(p.theta))
    return fail(PDS_EINVAL, name + ": rope theta must be > 0");
  if (p.layout != PDS_ROPE_NEOX && p.layout != PDS_ROPE_NORM)
    return fail(PDS_EINVAL, name + ": rope layout must be PDS_ROPE_NEOX or PDS_ROPE_NORM");
  if (p.rot_dim < 0 || p.rot_dim > hd)
    return fail(PDS_EINVAL, name + ": rot_dim must be 0 .. head_dim");
  const int rot = p.rot_dim ? p.rot_dim : hd;
  if (rot % 16) return fail(PDS_DECLINED, "declined: " + name + " needs rot_dim % 16 == 0");
  if (!std::isfinite(p.mscale) || p.mscale < 0.f)
    return fail(PDS_EINVAL, name + ": rope mscale must be 0 or > 0");
  if (p.scaling != PDS_ROPE_UNSCALED && p.scaling != PDS_ROPE_LINEAR && p.scaling != PDS_ROPE_YARN)
    return fail(PDS_EINVAL, name + ": unknown rope scaling");
  if (p.scaling != PDS_ROPE_UNSCALED && (!(p.factor > 0.f) || !std::isfinite(p.factor)))
    return fail(PDS_EINVAL, name + ": rope factor must be > 0");
  double lo = 0.0, hi = 0.0;
  if (p.scaling == PDS_ROPE_YARN) {
    if (!(p.theta > 1.f) || p.orig_context < 1 || !(p.beta_slow > 0.f) ||
        !(p.beta_fast > p.beta_slow) || !std::isfinite(p.beta_fast))
      return fail(PDS_EINVAL, name + ": YaRN needs theta > 1, orig_context >= 1, beta_fast > beta_slow > 0");
    auto edge = [&](double beta) {
      return rot * std::log(p.orig_context / (2.0 * M_PI * beta)) / (2.0 * std::log(double{p.theta}));
    };
    lo = std::max(0.0, std::floor(edge(p.beta_fast)));
    hi = std::min(rot - 1.0, std::ceil(edge(p.beta_slow)));
  }
  // theta^(-2i/rot) in float64, eight neighbours from one power
  const double next = std::pow(double{p.theta}, -2.0 / rot);
  double omega = 1.0;
  for (int i = 0; i < rot / 2; ++i) {
    omega = i % 8 ? omega * next : std::pow(double{p.theta}, -2.0 * i / rot);
    double w = omega;
    if (p.freq_factors) {
      const float f = p.freq_factors[i];
      if (!(f > 0.f) || !std::isfinite(f))
        return fail(PDS_EINVAL, name + ": freq_factors must be finite and > 0");
      w /= f;
    }
    if (p.scaling == PDS_ROPE_LINEAR) w /= p.factor;
    if (p.scaling == PDS_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
      w *= (1.0 - ramp) + ramp / p.factor;
    }
    // positions are whole numbers: whole turns per position drop out
    const double turns = w / (2.0 * M_PI);
    r->turns[i] = static_cast<uint64_t>(std::ldexp(turns - std::floor(turns), 64));
  }
  r->rot_dim = rot;
  r->layout = p.layout;
  r->mscale = p.mscale > 0.f ? p.mscale : 1.0f;
  r->sign = inverse ? -1.0f : 1.0f;
  return PDS_OK;
}

// Whether the rows of a cache, `width` elements each, are apart: from the smallest
// stride on each one steps over all that lies within the ones before it (sizes of
// one have none).
bool rows_apart(const pds_cache& c, int64_t ss, int64_t rs, int64_t hs) {
  struct Dim {
    int64_t stride, size;
  } dims[3] = {{ss, c.n_seqs}, {rs, c.capacity}, {hs, c.n_kv_heads}};
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  int64_t extent = c.head_dim;
  for (const Dim& d : dims) {
    if (d.size == 1) continue;
    int64_t span;
    if (d.stride < extent || __builtin_mul_overflow(d.stride, d.size - 1, &span) ||
        __builtin_add_overflow(span, extent, &extent))
      return false;
  }
  return extent <= INT64_MAX / 2;  // in bytes
}

// The kernels' view of a cache, or the reason it is refused.
pds_status make_view(const char* fn, const pds_cache* cache, pds::CacheView* v) {
  const std::string name = fn;
  if (!cache) return fail(PDS_EINVAL, name + ": cache is NULL");
  const pds_cache& c = *cache;
  if (c.format != PDS_KV_BF16 && c.format != PDS_KV_E4M3 && c.format != PDS_KV_INT4)
    return fail(PDS_EINVAL, name + ": unknown cache format");
  if (c.reserved != 0) return fail(PDS_EINVAL, name + ": cache.reserved must be 0");
  if (c.n_seqs < 1 || c.capacity < 1 || c.n_kv_heads < 1 || c.head_dim < 1)
    return fail(PDS_EINVAL, name + ": every cache size must be positive");
  if (c.head_dim != 64 && c.head_dim != 128)
    return fail(PDS_DECLINED, "declined: " + name + " needs head_dim 64 or 128");
  if (c.n_seqs > 4096 || c.n_kv_heads > 1024 || c.capacity > (1 << 30))
    return fail(PDS_DECLINED, "declined: " + name +
                                  " serves at most 4096 sequences, 1024 kv heads and 2^30 rows");
  if (!c.k || !c.v || !c.lens) return fail(PDS_EINVAL, name + ": cache k / v / lens is NULL");
  if (!aligned16(c.k) || !aligned16(c.v))
    return fail(PDS_EINVAL, name + ": cache k / v not 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(c.lens) & 3u)
    return fail(PDS_EINVAL, name + ": cache lens not 4-byte aligned");
  if (c.format != PDS_KV_BF16) {
    if (!c.k_scale || !c.v_scale) return fail(PDS_EINVAL, name + ": cache scale words are NULL");
    if ((reinterpret_cast<uintptr_t>(c.k_scale) | reinterpret_cast<uintptr_t>(c.v_scale)) & 3u)
      return fail(PDS_EINVAL, name + ": cache scale words not 4-byte aligned");
  }
  int64_t hs = c.head_stride, rs = c.row_stride, ss = c.seq_stride;
  if (hs == 0 && rs == 0 && ss == 0) {
    hs = c.head_dim;
    rs = hs * c.n_kv_heads;
    ss = rs * c.capacity;
  }
  const int per16 = c.format == PDS_KV_BF16 ? 8 : c.format == PDS_KV_E4M3 ? 16 : 32;
  if (hs < c.head_dim || rs < c.head_dim || (c.n_seqs > 1 ? ss < c.head_dim : ss < 0))
    return fail(PDS_EINVAL, name + ": a cache stride is smaller than a head's row");
  if (hs % per16 || rs % per16 || ss % per16)
    return fail(PDS_EINVAL, name + ": cache strides must be multiples of 16 bytes");
  if (!rows_apart(c, ss, rs, hs))
    return fail(PDS_EINVAL, name + ": cache strides let rows overlap");
  // half bytes: elements to bytes
  auto bytes = [&](int64_t e) { return c.format == PDS_KV_BF16 ? 2 * e : c.format == PDS_KV_E4M3 ? e : e / 2; };
  *v = pds::CacheView{static_cast<char*>(c.k), static_cast<char*>(c.v), c.k_scale, c.v_scale,
                      c.lens, bytes(ss), bytes(rs), bytes(hs), c.n_seqs, c.capacity, c.n_kv_heads};
  return PDS_OK;
}

// A row stride in elements: 0 is packed.
pds_status row_stride(const char* fn, int64_t packed, int64_t* stride) {
  if (*stride == 0) *stride = packed;
  if (*stride < packed || *stride % 8)
    return fail(PDS_EINVAL, std::string(fn) + ": row strides must be 0, or multiples of 8 and no "
                                              "smaller than a packed row");
  return PDS_OK;
}

// The status word and SM count of the current device, looked up once per
// device; ptr has to be memory of that device.
constexpr int kMaxDevices = 64;
pds_status device_facts(const char* fn, const void* ptr, uint32_t** status, int* sms) {
  static pds::DeviceFacts facts[kMaxDevices];
  const std::string name = fn;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return fail(PDS_ELAUNCH, name + ": no CUDA device");
  }
  cudaPointerAttributes at{};
  if (cudaPointerGetAttributes(&at, ptr) != cudaSuccess) {
    cudaGetLastError();
    return fail(PDS_ELAUNCH, name + ": no CUDA device");
  }
  if ((at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged) ||
      (at.type == cudaMemoryTypeDevice && at.device != dev))
    return fail(PDS_EINVAL, name + ": a buffer is not memory of the current device");
  std::string err;
  auto lookup = [&](uint32_t** word, int* n) {
    *word = pds::component_status(&err);
    if (!*word) return false;
    const cudaError_t ce = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
    if (ce != cudaSuccess) err = cudaGetErrorString(ce);
    return ce == cudaSuccess && *n > 0;
  };
  if (!facts[dev].get(lookup, status, sms)) {
    cudaGetLastError();
    return fail(PDS_ELAUNCH, name + ": status word or SM count: " + err);
  }
  return PDS_OK;
}

pds_status launched(const char* fn, cudaError_t ce) {
  if (ce == cudaSuccess) return PDS_OK;
  return fail(PDS_ELAUNCH, std::string(fn) + " launch: " + cudaGetErrorString(ce));
}

}  // namespace

pds_status pds_rope(const pds_rope_spec* spec, const uint16_t* x, uint16_t* y, int32_t rows,
                    int32_t n_heads, int32_t head_dim, int64_t x_stride, int64_t y_stride,
                    const int32_t* positions, int32_t start_pos, int32_t inverse, void* stream) try {
  if (!spec || !x || !y) return fail(PDS_EINVAL, "pds_rope: NULL operand");
  if (rows < 1 || n_heads < 1 || head_dim < 1) return fail(PDS_EINVAL, "pds_rope: bad size");
  if (head_dim % 16 || head_dim > 256 || n_heads > (1 << 20))
    return fail(PDS_DECLINED, "declined: pds_rope needs head_dim % 16 == 0, head_dim <= 256");
  if (!aligned16(x) || !aligned16(y) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return fail(PDS_EINVAL, "pds_rope: operand not aligned");
  const int64_t packed = static_cast<int64_t>(n_heads) * head_dim;
  pds_status rc;
  if ((rc = row_stride("pds_rope", packed, &x_stride)) != PDS_OK ||
      (rc = row_stride("pds_rope", packed, &y_stride)) != PDS_OK)
    return rc;
  if (x == y && x_stride != y_stride)
    return fail(PDS_EINVAL, "pds_rope: in place needs one stride");
  pds::RopeTurns turns;
  if ((rc = make_turns("pds_rope", spec, head_dim, inverse != 0, &turns)) != PDS_OK) return rc;
  uint32_t* status;
  int sms;
  if ((rc = device_facts("pds_rope", x, &status, &sms)) != PDS_OK) return rc;
  return launched("pds_rope", pds::launch_rope(turns, x, y, rows, n_heads, head_dim, x_stride,
                                               y_stride, positions, start_pos,
                                               static_cast<cudaStream_t>(stream)));
} catch (...) {  // a message could not be allocated
  return PDS_ENOMEM;
}

pds_status pds_cache_write(const pds_cache* cache, const pds_rope_spec* spec, const uint16_t* k,
                           const uint16_t* v, int32_t n_tokens, int64_t k_stride,
                           int64_t v_stride, const int32_t* parents, const int32_t* positions,
                           void* stream) try {
  pds::CacheView view;
  pds_status rc = make_view("pds_cache_write", cache, &view);
  if (rc != PDS_OK) return rc;
  if (!k || !v) return fail(PDS_EINVAL, "pds_cache_write: NULL operand");
  if (!aligned16(k) || !aligned16(v) ||
      ((reinterpret_cast<uintptr_t>(parents) | reinterpret_cast<uintptr_t>(positions)) & 3u))
    return fail(PDS_EINVAL, "pds_cache_write: operand not aligned");
  if (n_tokens < 1) return fail(PDS_EINVAL, "pds_cache_write: n_tokens must be >= 1");
  if (n_tokens > cache->capacity)
    return fail(PDS_DECLINED, "declined: pds_cache_write: more tokens than the cache's capacity");
  if (parents && n_tokens > pds::kMaxDraftTokens)
    return fail(PDS_DECLINED, "declined: pds_cache_write: at most 256 tokens with parents");
  if (static_cast<int64_t>(cache->n_seqs) * n_tokens > INT32_MAX)
    return fail(PDS_DECLINED, "declined: pds_cache_write: too many rows");
  const int64_t packed = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
  if ((rc = row_stride("pds_cache_write", packed, &k_stride)) != PDS_OK ||
      (rc = row_stride("pds_cache_write", packed, &v_stride)) != PDS_OK)
    return rc;
  pds::RopeTurns turns;
  if ((rc = make_turns("pds_cache_write", spec, cache->head_dim, false, &turns)) != PDS_OK)
    return rc;
  uint32_t* status;
  int sms;
  if ((rc = device_facts("pds_cache_write", cache->k, &status, &sms)) != PDS_OK) return rc;
  return launched("pds_cache_write",
                  pds::launch_cache_write(view, cache->format, cache->head_dim, turns, k, v,
                                          n_tokens, k_stride, v_stride, parents, positions, status,
                                          static_cast<cudaStream_t>(stream)));
} catch (...) {  // a message could not be allocated
  return PDS_ENOMEM;
}

pds_status pds_cache_read(const pds_cache* cache, int32_t first_row, int32_t rows,
                          uint16_t* k_out, uint16_t* v_out, void* stream) try {
  pds::CacheView view;
  pds_status rc = make_view("pds_cache_read", cache, &view);
  if (rc != PDS_OK) return rc;
  if (!k_out && !v_out) return fail(PDS_EINVAL, "pds_cache_read: k_out and v_out are NULL");
  if (!aligned16(k_out) || !aligned16(v_out))
    return fail(PDS_EINVAL, "pds_cache_read: output not 16-byte aligned");
  if (rows < 1 || first_row < PDS_AT_LENS)
    return fail(PDS_EINVAL, "pds_cache_read: rows must be >= 1 and first_row >= 0 or PDS_AT_LENS");
  if (static_cast<int64_t>(first_row > 0 ? first_row : 0) + rows > cache->capacity)
    return fail(PDS_DECLINED, "declined: pds_cache_read: rows past the cache's capacity");
  uint32_t* status;
  int sms;
  if ((rc = device_facts("pds_cache_read", cache->k, &status, &sms)) != PDS_OK) return rc;
  return launched("pds_cache_read",
                  pds::launch_cache_read(view, cache->format, cache->head_dim, first_row, rows,
                                         k_out, v_out, status, static_cast<cudaStream_t>(stream)));
} catch (...) {  // a message could not be allocated
  return PDS_ENOMEM;
}

size_t pds_attention_tree_workspace_bytes(const pds_cache* cache, int32_t n_tokens,
                                          int32_t n_heads) {
  if (!cache || n_tokens < 1 || n_tokens > pds::kMaxDraftTokens || n_heads < 1 ||
      n_heads > 8192 || cache->n_seqs < 1 || cache->n_seqs > 4096 || cache->n_kv_heads < 1 ||
      n_heads % cache->n_kv_heads || (cache->head_dim != 64 && cache->head_dim != 128))
    return 0;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return pds::tree_attention_ws_bytes(cache->format, cache->head_dim, cache->n_seqs, n_tokens,
                                      n_heads, cache->n_kv_heads, sms);
}

pds_status pds_attention_tree(const pds_cache* cache, const uint16_t* q, uint16_t* o,
                              int32_t n_tokens, int32_t n_heads, int64_t q_stride,
                              int64_t o_stride, const int32_t* parents, float softcap,
                              int32_t window, int32_t max_len, void* workspace,
                              size_t workspace_bytes, void* stream) try {
  pds::TreeAttnCall a{};
  pds_status rc = make_view("pds_attention_tree", cache, &a.cache);
  if (rc != PDS_OK) return rc;
  if (!q || !o) return fail(PDS_EINVAL, "pds_attention_tree: NULL operand");
  if (n_tokens < 1 || n_heads < 1) return fail(PDS_EINVAL, "pds_attention_tree: bad size");
  if (!(softcap >= 0.f) || !std::isfinite(softcap) || window < 0 || max_len < 0)
    return fail(PDS_EINVAL, "pds_attention_tree: softcap, window and max_len must be >= 0");
  if (n_heads % cache->n_kv_heads || n_heads > 8192)
    return fail(PDS_DECLINED, "declined: pds_attention_tree needs H % Hkv == 0, H <= 8192");
  if (n_tokens > pds::kMaxDraftTokens)
    return fail(PDS_DECLINED, "declined: pds_attention_tree takes at most 256 tokens");
  if (n_tokens > cache->capacity)
    return fail(PDS_DECLINED, "declined: pds_attention_tree: more tokens than the cache's capacity");
  if (!aligned16(q) || !aligned16(o) || (workspace && !aligned16(workspace)) ||
      (reinterpret_cast<uintptr_t>(parents) & 3u))
    return fail(PDS_EINVAL, "pds_attention_tree: operand not aligned");
  const int64_t packed = static_cast<int64_t>(n_heads) * cache->head_dim;
  if ((rc = row_stride("pds_attention_tree", packed, &q_stride)) != PDS_OK ||
      (rc = row_stride("pds_attention_tree", packed, &o_stride)) != PDS_OK)
    return rc;
  if (static_cast<int64_t>(cache->n_seqs) * n_tokens * n_heads > INT32_MAX)
    return fail(PDS_DECLINED, "declined: pds_attention_tree: too many query rows");
  if (q == o)  // (its blocks read rows of q after others have written theirs of o)
    return fail(PDS_EINVAL, "pds_attention_tree: q and o are the same buffer");
  if ((rc = device_facts("pds_attention_tree", cache->k, &a.status, &a.num_sms)) != PDS_OK)
    return rc;
  if (workspace && workspace_bytes < pds::tree_attention_ws_bytes(
                                         cache->format, cache->head_dim, cache->n_seqs, n_tokens,
                                         n_heads, cache->n_kv_heads, a.num_sms))
    return fail(PDS_EINVAL,
                "pds_attention_tree: workspace smaller than pds_attention_tree_workspace_bytes");
  a.format = cache->format;
  a.head_dim = cache->head_dim;
  a.q = q;
  a.o = o;
  a.q_stride = q_stride;
  a.o_stride = o_stride;
  a.parents = parents;
  a.n_tokens = n_tokens;
  a.n_heads = n_heads;
  const int32_t room = cache->capacity - n_tokens;
  a.max_len = max_len > 0 ? std::min(max_len, room) : room;
  a.softcap = softcap;
  a.window = window;
  a.ws = static_cast<char*>(workspace);
  std::string err;
  rc = pds::tree_attention(a, static_cast<cudaStream_t>(stream), &err);
  if (rc != PDS_OK) return fail(rc, err);
  return PDS_OK;
} catch (...) {  // a message could not be allocated
  return PDS_ENOMEM;
}

}  // extern "C"
