// C-ABI entry points of libgdn.so: host-side validation, then dispatch to the
// kernels. Nothing is launched when validation fails. The declarations, with
// the passages each operation follows, are in include/gdn.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "gdn.h"
#include "gdn_common.cuh"
#include "launch.h"

namespace {

using gdn::kHeadDim;

bool valid_dtype(gdn_dtype t) { return t == GDN_BF16 || t == GDN_F32; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes) == 0;
}
bool stride_ok(int64_t stride_elems, gdn_dtype t) {
  return (stride_elems * gdn::elem_bytes(t)) % 16 == 0;
}
gdn_status from_cuda(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// [a, a+na) and [b, b+nb) overlap without being identical ranges
bool partial_overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  if (a0 == b0 && na == nb) return false;
  return a0 < b0 + nb && b0 < a0 + na;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

struct Extent { const void* p; size_t n; };
// an output over an input or another output
template <size_t I, size_t O>
bool outputs_overlap(const Extent (&in)[I], const Extent (&out)[O]) {
  for (size_t i = 0; i < O; ++i) {
    for (const Extent& b : in)
      if (overlap(out[i].p, out[i].n, b.p, b.n)) return true;
    for (size_t j = i + 1; j < O; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
}

// Checks shared by the prefill and decode recurrences.
gdn_status check_recurrence(const void* q, const void* k, const void* v,
                            gdn_dtype qkv_dtype, int64_t qs, int64_t ks,
                            int64_t vs, const void* g, const void* beta,
                            gdn_dtype gate_dtype, int H_k, int H_v, void* o,
                            gdn_dtype o_dtype, bool have_tokens) {
  if (!valid_dtype(qkv_dtype) || !valid_dtype(gate_dtype) || !valid_dtype(o_dtype))
    return GDN_ERR_INVALID_ARG;
  if (H_k <= 0 || H_v <= 0 || H_v % H_k != 0) return GDN_ERR_INVALID_ARG;
  if (qs < (int64_t)H_k * kHeadDim || ks < (int64_t)H_k * kHeadDim ||
      vs < (int64_t)H_v * kHeadDim)
    return GDN_ERR_INVALID_ARG;
  if (!have_tokens) return GDN_OK;
  if (!q || !k || !v || !g || !beta || !o) return GDN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o))
    return GDN_ERR_MISALIGNED;
  if (!stride_ok(qs, qkv_dtype) || !stride_ok(ks, qkv_dtype) || !stride_ok(vs, qkv_dtype))
    return GDN_ERR_MISALIGNED;
  const int gb = gdn::elem_bytes(gate_dtype);
  if (!aligned_to(g, gb) || !aligned_to(beta, gb)) return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

}  // namespace

extern "C" {

const char* gdn_status_string(gdn_status s) {
  switch (s) {
    case GDN_OK: return "GDN_OK";
    case GDN_ERR_INVALID_ARG: return "GDN_ERR_INVALID_ARG: invalid argument";
    case GDN_ERR_UNSUPPORTED: return "GDN_ERR_UNSUPPORTED: unsupported shape or option";
    case GDN_ERR_MISALIGNED: return "GDN_ERR_MISALIGNED: pointer or stride not 16-byte aligned";
    case GDN_ERR_CUDA: return "GDN_ERR_CUDA: CUDA launch failed";
    case GDN_ERR_TIMEOUT: return "GDN_ERR_TIMEOUT: a bounded wait in a kernel gave up";
  }
  return "unknown gdn_status";
}

const char* gdn_version(void) { return "0.1.0"; }

gdn_status gdn_conv1d_silu(const void* x, int64_t x_row_stride,
                           gdn_dtype x_dtype, const void* w, gdn_dtype w_dtype,
                           const void* bias, int channels, int l2norm_channels,
                           float l2_eps, const int32_t* cu_seqlens, int N,
                           int64_t T_total, const void* conv_state_in,
                           void* conv_state_out, void* y, int64_t y_row_stride,
                           gdn_dtype y_dtype, cudaStream_t stream) {
  if (!valid_dtype(x_dtype) || !valid_dtype(w_dtype) || !valid_dtype(y_dtype))
    return GDN_ERR_INVALID_ARG;
  if (N < 0 || T_total < 0 || channels <= 0 || channels % 8 != 0)
    return GDN_ERR_INVALID_ARG;
  if (l2norm_channels < 0 || l2norm_channels % kHeadDim != 0 ||
      l2norm_channels > channels || !(l2_eps >= 0.f))
    return GDN_ERR_INVALID_ARG;
  if (N == 0) return T_total == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens || !w) return GDN_ERR_INVALID_ARG;
  if (T_total > 0) {
    if (!x || !y) return GDN_ERR_INVALID_ARG;
    if (x_row_stride < channels || y_row_stride < channels) return GDN_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y)) return GDN_ERR_MISALIGNED;
    if (!stride_ok(x_row_stride, x_dtype) || !stride_ok(y_row_stride, y_dtype))
      return GDN_ERR_MISALIGNED;
  }
  if (!aligned16(w) || (bias && !aligned16(bias)) ||
      (conv_state_in && !aligned16(conv_state_in)) ||
      (conv_state_out && !aligned16(conv_state_out)))
    return GDN_ERR_MISALIGNED;
  const size_t cs_bytes = (size_t)N * 3 * channels * gdn::elem_bytes(x_dtype);
  if (partial_overlap(conv_state_in, cs_bytes, conv_state_out, cs_bytes))
    return GDN_ERR_INVALID_ARG;
  gdn::ConvArgs a{x, x_row_stride, x_dtype, w, w_dtype, bias, channels,
                  l2norm_channels, l2_eps, cu_seqlens, N, T_total,
                  conv_state_in, conv_state_out, y, y_row_stride, y_dtype,
                  stream};
  return from_cuda(gdn::launch_conv1d_silu(a));
}

size_t gdn_chunked_prefill_workspace(int N, int64_t T_total, int H_k, int H_v) {
  (void)H_k;
  if (N <= 0 || T_total <= 0 || H_v <= 0) return 0;
  return gdn::prefill_pc_workspace(N, T_total, H_v);
}

gdn_status gdn_chunked_prefill(const void* q, const void* k, const void* v,
                               gdn_dtype qkv_dtype, int64_t q_row_stride,
                               int64_t k_row_stride, int64_t v_row_stride,
                               const void* g, const void* beta,
                               gdn_dtype gate_dtype, const float* state_in,
                               float* state_out, const int32_t* cu_seqlens,
                               int N, int64_t T_total, int H_k, int H_v,
                               float scale, void* o, gdn_dtype o_dtype,
                               void* workspace, size_t workspace_bytes,
                               cudaStream_t stream) {
  if (N < 0 || T_total < 0) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_recurrence(q, k, v, qkv_dtype, q_row_stride, k_row_stride,
                                   v_row_stride, g, beta, gate_dtype, H_k, H_v,
                                   o, o_dtype, T_total > 0);
  if (st != GDN_OK) return st;
  if (N == 0) return T_total == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens) return GDN_ERR_INVALID_ARG;
  if ((state_in && !aligned16(state_in)) || (state_out && !aligned16(state_out)))
    return GDN_ERR_MISALIGNED;
  const size_t st_bytes = (size_t)N * H_v * kHeadDim * kHeadDim * sizeof(float);
  if (partial_overlap(state_in, st_bytes, state_out, st_bytes)) return GDN_ERR_INVALID_ARG;
  if (qkv_dtype == GDN_BF16 && T_total > 0) {
    if (workspace_bytes < gdn_chunked_prefill_workspace(N, T_total, H_k, H_v) ||
        (workspace_bytes > 0 && !workspace))
      return GDN_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return GDN_ERR_MISALIGNED;
  }
  gdn::RecurArgs a{q, k, v, qkv_dtype, q_row_stride, k_row_stride, v_row_stride,
                   g, beta, gate_dtype, state_in, state_out, cu_seqlens, N,
                   T_total, H_k, H_v, scale, o, o_dtype, workspace,
                   workspace_bytes, stream};
  return from_cuda(qkv_dtype == GDN_BF16 ? gdn::launch_prefill_pc(a)
                                         : gdn::launch_prefill_chunked_f32(a));
}

gdn_status gdn_prefill_layer(const void* x, int64_t x_row_stride, const void* conv_w,
                             gdn_dtype w_dtype, const void* conv_bias,
                             const void* conv_state_in, void* conv_state_out,
                             const void* g, const void* beta, gdn_dtype gate_dtype,
                             const float* state_in, float* state_out,
                             const int32_t* cu_seqlens, int N, int64_t T_total, int H_k,
                             int H_v, float scale, float l2_eps, const void* z,
                             const void* norm_w, float norm_eps, void* y, gdn_dtype y_dtype,
                             void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!valid_dtype(w_dtype) || !valid_dtype(gate_dtype) || !valid_dtype(y_dtype))
    return GDN_ERR_INVALID_ARG;
  if (N < 0 || T_total < 0 || H_k <= 0 || H_v <= 0 || H_v % H_k != 0 || !(l2_eps >= 0.f) ||
      !(norm_eps >= 0.f))
    return GDN_ERR_INVALID_ARG;
  const int64_t C = 2 * (int64_t)H_k * kHeadDim + (int64_t)H_v * kHeadDim;
  if (x_row_stride < C) return GDN_ERR_INVALID_ARG;
  if (N == 0) return T_total == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens || !conv_w || !norm_w) return GDN_ERR_INVALID_ARG;
  if (T_total > 0 && (!x || !g || !beta || !z || !y)) return GDN_ERR_INVALID_ARG;
  if ((x && !aligned16(x)) || !aligned16(conv_w) || (conv_bias && !aligned16(conv_bias)) ||
      (conv_state_in && !aligned16(conv_state_in)) ||
      (conv_state_out && !aligned16(conv_state_out)) || (z && !aligned16(z)) ||
      !aligned16(norm_w) || (y && !aligned16(y)) || (state_in && !aligned16(state_in)) ||
      (state_out && !aligned16(state_out)))
    return GDN_ERR_MISALIGNED;
  if (!stride_ok(x_row_stride, GDN_BF16)) return GDN_ERR_MISALIGNED;
  const int gb = gdn::elem_bytes(gate_dtype);
  if ((g && !aligned_to(g, gb)) || (beta && !aligned_to(beta, gb))) return GDN_ERR_MISALIGNED;
  const size_t st_bytes = (size_t)N * H_v * kHeadDim * kHeadDim * sizeof(float);
  if (partial_overlap(state_in, st_bytes, state_out, st_bytes)) return GDN_ERR_INVALID_ARG;
  const size_t cs_bytes = (size_t)N * 3 * C * 2;
  if (partial_overlap(conv_state_in, cs_bytes, conv_state_out, cs_bytes))
    return GDN_ERR_INVALID_ARG;
  if (T_total > 0) {
    if (workspace_bytes < gdn_prefill_layer_workspace(N, T_total, H_k, H_v) || !workspace)
      return GDN_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return GDN_ERR_MISALIGNED;
  }
  gdn::LayerPrefillArgs a{x, x_row_stride, conv_w, w_dtype, conv_bias, conv_state_in,
                          conv_state_out, g, beta, gate_dtype, state_in, state_out,
                          cu_seqlens, N, T_total, H_k, H_v, scale, l2_eps, z, norm_w,
                          norm_eps, y, y_dtype, workspace, workspace_bytes, stream};
  return from_cuda(gdn::launch_prefill_layer(a));
}

size_t gdn_prefill_layer_workspace(int N, int64_t T_total, int H_k, int H_v) {
  if (N < 0 || T_total < 0 || H_k <= 0 || H_v <= 0 || H_v % H_k != 0) return 0;
  if (T_total == 0) return 0;
  return gdn::prefill_layer_workspace(N, T_total, H_k, H_v);
}

gdn_status gdn_chunked_prefill_status(const void* workspace, cudaStream_t stream) {
  if (workspace && !aligned16(workspace)) return GDN_ERR_MISALIGNED;
  int word = 0;
  if (gdn::prefill_abort_word(workspace, stream, &word) != cudaSuccess) return GDN_ERR_CUDA;
  return word ? GDN_ERR_TIMEOUT : GDN_OK;
}

void gdn_set_wait_limit_ns(uint64_t ns) { gdn::set_wait_limit_ns(ns); }

gdn_status gdn_stepwise_prefill(const void* q, const void* k, const void* v,
                                gdn_dtype qkv_dtype, int64_t q_row_stride,
                                int64_t k_row_stride, int64_t v_row_stride,
                                const void* g, const void* beta,
                                gdn_dtype gate_dtype, const float* state_in,
                                float* state_out, const int32_t* cu_seqlens,
                                int N, int64_t T_total, int H_k, int H_v,
                                float scale, void* o, gdn_dtype o_dtype,
                                cudaStream_t stream) {
  if (N < 0 || T_total < 0) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_recurrence(q, k, v, qkv_dtype, q_row_stride, k_row_stride,
                                   v_row_stride, g, beta, gate_dtype, H_k, H_v,
                                   o, o_dtype, T_total > 0);
  if (st != GDN_OK) return st;
  if (N == 0) return T_total == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens) return GDN_ERR_INVALID_ARG;
  if ((state_in && !aligned16(state_in)) || (state_out && !aligned16(state_out)))
    return GDN_ERR_MISALIGNED;
  const size_t st_bytes = (size_t)N * H_v * kHeadDim * kHeadDim * sizeof(float);
  if (partial_overlap(state_in, st_bytes, state_out, st_bytes)) return GDN_ERR_INVALID_ARG;
  gdn::RecurArgs a{q, k, v, qkv_dtype, q_row_stride, k_row_stride, v_row_stride,
                   g, beta, gate_dtype, state_in, state_out, cu_seqlens, N,
                   T_total, H_k, H_v, scale, o, o_dtype, nullptr, 0, stream};
  return from_cuda(gdn::launch_prefill_stepwise(a));
}

gdn_status gdn_chunked_prefill_noalloc(const void* q, const void* k, const void* v,
                                       gdn_dtype qkv_dtype, int64_t q_row_stride,
                                       int64_t k_row_stride, int64_t v_row_stride,
                                       const void* g, const void* beta,
                                       gdn_dtype gate_dtype, const float* state_in,
                                       float* state_out, const int32_t* cu_seqlens,
                                       int N, int64_t T_total, int H_k, int H_v,
                                       float scale, void* o, gdn_dtype o_dtype,
                                       cudaStream_t stream) {
  if (N < 0 || T_total < 0) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_recurrence(q, k, v, qkv_dtype, q_row_stride, k_row_stride,
                                   v_row_stride, g, beta, gate_dtype, H_k, H_v,
                                   o, o_dtype, T_total > 0);
  if (st != GDN_OK) return st;
  if (N == 0) return T_total == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu_seqlens) return GDN_ERR_INVALID_ARG;
  if ((state_in && !aligned16(state_in)) || (state_out && !aligned16(state_out)))
    return GDN_ERR_MISALIGNED;
  const size_t st_bytes = (size_t)N * H_v * kHeadDim * kHeadDim * sizeof(float);
  if (partial_overlap(state_in, st_bytes, state_out, st_bytes)) return GDN_ERR_INVALID_ARG;
  if (qkv_dtype == GDN_BF16 && T_total > 0 &&
      gdn_chunked_prefill_workspace(N, T_total, H_k, H_v) > gdn::prefill_noalloc_scratch_bytes())
    return GDN_ERR_UNSUPPORTED;
  gdn::RecurArgs a{q, k, v, qkv_dtype, q_row_stride, k_row_stride, v_row_stride,
                   g, beta, gate_dtype, state_in, state_out, cu_seqlens, N,
                   T_total, H_k, H_v, scale, o, o_dtype, nullptr, 0, stream};
  return from_cuda(qkv_dtype == GDN_BF16 ? gdn::launch_prefill_pc_noalloc(a)
                                         : gdn::launch_prefill_chunked_f32(a));
}

size_t gdn_chunked_prefill_noalloc_scratch_bytes(void) {
  return gdn::prefill_noalloc_scratch_bytes();
}

gdn_status gdn_decode_step(const void* q, const void* k, const void* v,
                           gdn_dtype qkv_dtype, int64_t q_row_stride,
                           int64_t k_row_stride, int64_t v_row_stride,
                           const void* g, const void* beta,
                           gdn_dtype gate_dtype, float* state, int N, int H_k,
                           int H_v, float scale, void* o, gdn_dtype o_dtype,
                           cudaStream_t stream) {
  if (N < 0) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_recurrence(q, k, v, qkv_dtype, q_row_stride, k_row_stride,
                                   v_row_stride, g, beta, gate_dtype, H_k, H_v,
                                   o, o_dtype, N > 0);
  if (st != GDN_OK) return st;
  if (N == 0) return GDN_OK;
  if (!state) return GDN_ERR_INVALID_ARG;
  if (!aligned16(state)) return GDN_ERR_MISALIGNED;
  gdn::RecurArgs a{q, k, v, qkv_dtype, q_row_stride, k_row_stride, v_row_stride,
                   g, beta, gate_dtype, state, state, nullptr, N, N, H_k, H_v,
                   scale, o, o_dtype, nullptr, 0, stream};
  return from_cuda(gdn::launch_decode_step(a));
}

gdn_status gdn_decode_layer_step(const void* x, int64_t x_row_stride, gdn_dtype x_dtype,
                                 const void* conv_w, gdn_dtype w_dtype,
                                 const void* conv_bias, void* conv_state,
                                 const void* g, const void* beta, gdn_dtype gate_dtype,
                                 float* state, const int32_t* state_idx, int N, int P,
                                 int H_k, int H_v, float scale, float l2_eps,
                                 const void* z, const void* norm_w, float norm_eps,
                                 void* y, gdn_dtype y_dtype, cudaStream_t stream) {
  if (!valid_dtype(x_dtype) || !valid_dtype(w_dtype) || !valid_dtype(gate_dtype) ||
      !valid_dtype(y_dtype))
    return GDN_ERR_INVALID_ARG;
  if (N < 0 || P < 0 || H_k <= 0 || H_v <= 0 || H_v % H_k != 0 || !(l2_eps >= 0.f) ||
      !(norm_eps >= 0.f))
    return GDN_ERR_INVALID_ARG;
  if (H_v / H_k > 8) return GDN_ERR_UNSUPPORTED;
  const int64_t C = 2 * (int64_t)H_k * kHeadDim + (int64_t)H_v * kHeadDim;
  if (x_row_stride < C) return GDN_ERR_INVALID_ARG;
  if (N == 0) return GDN_OK;
  if (P == 0 || !x || !conv_w || !conv_state || !g || !beta || !state || !state_idx || !z ||
      !norm_w || !y)
    return GDN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(conv_w) || (conv_bias && !aligned16(conv_bias)) ||
      !aligned16(conv_state) || !aligned16(state) || !aligned16(z) || !aligned16(norm_w) ||
      !aligned16(y) || !aligned_to(state_idx, 4))
    return GDN_ERR_MISALIGNED;
  if (!stride_ok(x_row_stride, x_dtype)) return GDN_ERR_MISALIGNED;
  const int gb = gdn::elem_bytes(gate_dtype);
  if (!aligned_to(g, gb) || !aligned_to(beta, gb)) return GDN_ERR_MISALIGNED;
  gdn::DecodeLayerArgs a{x, x_row_stride, x_dtype, conv_w, w_dtype, conv_bias, conv_state,
                         g, beta, gate_dtype, state, state_idx, N, P, H_k, H_v, scale,
                         l2_eps, z, norm_w, norm_eps, y, y_dtype, stream};
  return from_cuda(gdn::launch_decode_layer(a));
}

gdn_status gdn_gated_rmsnorm(const void* x, gdn_dtype x_dtype, const void* z,
                             gdn_dtype z_dtype, const void* w,
                             gdn_dtype w_dtype, int64_t rows, int dim,
                             float eps, void* y, gdn_dtype y_dtype,
                             cudaStream_t stream) {
  if (!valid_dtype(x_dtype) || !valid_dtype(z_dtype) || !valid_dtype(w_dtype) ||
      !valid_dtype(y_dtype) || rows < 0 || !(eps >= 0.f))
    return GDN_ERR_INVALID_ARG;
  if (dim != kHeadDim) return GDN_ERR_UNSUPPORTED;
  if (rows == 0) return GDN_OK;
  if (!x || !z || !w || !y) return GDN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(z) || !aligned16(w) || !aligned16(y))
    return GDN_ERR_MISALIGNED;
  if (x == y && x_dtype != y_dtype) return GDN_ERR_INVALID_ARG;
  gdn::NormArgs a{x, x_dtype, z, z_dtype, w, w_dtype, rows, dim, eps, y, y_dtype,
                  stream};
  return from_cuda(gdn::launch_gated_rmsnorm(a));
}

// ---------------------------------------------------------- global attention

namespace {

constexpr int kAttnHeadDim = 256;

gdn_status check_attn_common(int H_q, int H_kv, int head_dim, int rope_dims, float rope_base,
                             float eps, gdn_dtype w_dtype) {
  if (head_dim != kAttnHeadDim) return GDN_ERR_UNSUPPORTED;
  if (H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0) return GDN_ERR_INVALID_ARG;
  if (rope_dims < 0 || rope_dims > 64 || rope_dims % 2 != 0) return GDN_ERR_UNSUPPORTED;
  if (rope_dims > 0 && !(rope_base > 1.0f)) return GDN_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !valid_dtype(w_dtype)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

bool attn_stride_ok(int64_t stride, int H) {
  return stride >= (int64_t)H * kAttnHeadDim && stride % 8 == 0;
}

}  // namespace

size_t gdn_attention_prefill_workspace(int64_t T_total, int H_q, int head_dim) {
  if (T_total < 0 || H_q <= 0 || head_dim != kAttnHeadDim) return 0;
  return gdn::attention_prefill_workspace(T_total, H_q);
}

gdn_status gdn_attention_prefill(const void* q, int64_t q_row_stride, const void* k,
                                 int64_t k_row_stride, const void* v, int64_t v_row_stride,
                                 const void* gate, int64_t gate_row_stride,
                                 const void* q_norm_w, const void* k_norm_w, gdn_dtype w_dtype,
                                 const int32_t* cu_seqlens, const int32_t* positions,
                                 const int32_t* pos0, int N, int64_t T_total, int H_q, int H_kv,
                                 int head_dim, float eps, int rope_dims, float rope_base,
                                 float scale, void* o, void* k_rot, void* v_h, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  gdn_status st = check_attn_common(H_q, H_kv, head_dim, rope_dims, rope_base, eps, w_dtype);
  if (st != GDN_OK) return st;
  if ((H_q / H_kv) % 2 != 0) return GDN_ERR_UNSUPPORTED;   // query heads go in pairs
  if (N < 0 || T_total < 0 || T_total > (int64_t)1 << 30) return GDN_ERR_INVALID_ARG;
  if (N == 0 && T_total > 0) return GDN_ERR_INVALID_ARG;
  if (!attn_stride_ok(q_row_stride, H_q) || !attn_stride_ok(gate_row_stride, H_q) ||
      !attn_stride_ok(k_row_stride, H_kv) || !attn_stride_ok(v_row_stride, H_kv))
    return GDN_ERR_MISALIGNED;
  if (T_total == 0) return GDN_OK;
  if (!q || !k || !v || !gate || !q_norm_w || !k_norm_w || !cu_seqlens || !o || !k_rot ||
      !v_h || !workspace)
    return GDN_ERR_INVALID_ARG;
  if (workspace_bytes < gdn::attention_prefill_workspace(T_total, H_q)) return GDN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(gate) || !aligned16(o) ||
      !aligned16(k_rot) || !aligned16(v_h) || !aligned16(workspace))
    return GDN_ERR_MISALIGNED;
  const int wb = gdn::elem_bytes(w_dtype);
  if (!aligned_to(q_norm_w, wb) || !aligned_to(k_norm_w, wb)) return GDN_ERR_MISALIGNED;
  gdn::AttnPrefillArgs a{q, k, v, gate, q_row_stride, k_row_stride, v_row_stride,
                         gate_row_stride, q_norm_w, k_norm_w, w_dtype, cu_seqlens, positions,
                         pos0, N, T_total, H_q, H_kv, eps, rope_dims, rope_base, scale, o,
                         k_rot, v_h, workspace, stream};
  return from_cuda(gdn::launch_attention_prefill(a));
}

size_t gdn_attention_decode_workspace(int N, int H_q, int L_max, int head_dim) {
  if (N < 0 || H_q <= 0 || L_max <= 0 || head_dim != kAttnHeadDim) return 0;
  return gdn::attention_decode_workspace(N, H_q, L_max);
}

gdn_status gdn_attention_decode(const void* q, int64_t q_row_stride, const void* k,
                                int64_t k_row_stride, const void* v, int64_t v_row_stride,
                                const void* gate, int64_t gate_row_stride,
                                const void* q_norm_w, const void* k_norm_w, gdn_dtype w_dtype,
                                void* k_cache, void* v_cache, const int32_t* cache_idx,
                                int32_t* cache_len, const int32_t* positions, int N, int P,
                                int L_max, int H_q, int H_kv, int head_dim, float eps,
                                int rope_dims, float rope_base, float scale, void* o,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  gdn_status st = check_attn_common(H_q, H_kv, head_dim, rope_dims, rope_base, eps, w_dtype);
  if (st != GDN_OK) return st;
  const int G = H_q / H_kv;
  if (G != 1 && G != 2 && G != 4 && G != 6 && G != 8) return GDN_ERR_UNSUPPORTED;
  if (N < 0 || N > 65535 || P < 0 || L_max <= 0 || H_q > 65535) return GDN_ERR_INVALID_ARG;
  if (!attn_stride_ok(q_row_stride, H_q) || !attn_stride_ok(gate_row_stride, H_q) ||
      !attn_stride_ok(k_row_stride, H_kv) || !attn_stride_ok(v_row_stride, H_kv))
    return GDN_ERR_MISALIGNED;
  if (N == 0) return GDN_OK;
  if (P == 0) return GDN_ERR_INVALID_ARG;
  if (!q || !k || !v || !gate || !q_norm_w || !k_norm_w || !k_cache || !v_cache ||
      !cache_len || !o || !workspace)
    return GDN_ERR_INVALID_ARG;
  if (workspace_bytes < gdn::attention_decode_workspace(N, H_q, L_max))
    return GDN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(gate) || !aligned16(o) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace))
    return GDN_ERR_MISALIGNED;
  const int wb = gdn::elem_bytes(w_dtype);
  if (!aligned_to(q_norm_w, wb) || !aligned_to(k_norm_w, wb)) return GDN_ERR_MISALIGNED;
  gdn::AttnDecodeArgs a{q, k, v, gate, q_row_stride, k_row_stride, v_row_stride,
                        gate_row_stride, q_norm_w, k_norm_w, w_dtype, k_cache, v_cache,
                        cache_idx, cache_len, positions, N, P, L_max, H_q, H_kv, eps,
                        rope_dims, rope_base, scale, o, workspace, stream};
  return from_cuda(gdn::launch_attention_decode(a));
}

// ------------------------------------------------------------ paged cache

namespace {

bool valid_dtype3(gdn_dtype t) { return valid_dtype(t) || t == GDN_F16; }
bool half_dtype(gdn_dtype t) { return t == GDN_F16 || t == GDN_BF16; }
bool paged_dim(int d) { return d == 64 || d == 128 || d == 256; }

// a cache and its strides: rows of D values, 16-byte aligned, inside int32 slots
gdn_status check_cache(const void* base, const gdn::PageStrides& s, int num_pages, int page_size,
                       int D) {
  if (!base || num_pages <= 0 || page_size <= 0) return GDN_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size > INT32_MAX) return GDN_ERR_INVALID_ARG;
  if (s.page < 0 || s.token < 0 || s.head < 0) return GDN_ERR_INVALID_ARG;
  if ((num_pages > 1 && s.page < D) || (page_size > 1 && s.token < D) || s.head < D)
    return GDN_ERR_INVALID_ARG;
  if (!aligned16(base) || s.page % 8 != 0 || s.token % 8 != 0 || s.head % 8 != 0)
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

}  // namespace

gdn_status gdn_page_plan(const int32_t* lens, const int32_t* want, int N,
                         int32_t* block_table, int64_t table_row_stride, int max_pages,
                         int32_t* free_pages, const int32_t* free_count, int num_pages,
                         int page_size, int64_t token_capacity, int32_t* new_lens,
                         int32_t* cu_new, int32_t* slot_map, int32_t* positions,
                         int32_t* new_count, int32_t* info, cudaStream_t stream) {
  if (N < 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0 || token_capacity < 0 ||
      token_capacity > (int64_t)1 << 30 || table_row_stride < max_pages)
    return GDN_ERR_INVALID_ARG;
  if (N > gdn::kPlanMaxRequests) return GDN_ERR_UNSUPPORTED;
  if ((int64_t)num_pages * page_size > INT32_MAX || (int64_t)max_pages * page_size > INT32_MAX ||
      num_pages > 1 << 30 || (int64_t)N * max_pages > INT32_MAX)
    return GDN_ERR_INVALID_ARG;
  if (!free_pages || !free_count || !cu_new || !new_count || (token_capacity > 0 && !slot_map))
    return GDN_ERR_INVALID_ARG;
  if (N > 0 && (!lens || !want || !block_table || !new_lens)) return GDN_ERR_INVALID_ARG;
  const Extent in[] = {{lens, (size_t)N * 4}, {want, (size_t)N * 4}, {free_count, 4}};
  const Extent out[] = {
      {new_lens, (size_t)N * 4}, {cu_new, (size_t)(N + 1) * 4},
      {slot_map, (size_t)token_capacity * 4}, {positions, (size_t)token_capacity * 4},
      {new_count, 4}, {info, 16}, {free_pages, (size_t)num_pages * 4},
      {block_table, N > 0 ? ((size_t)(N - 1) * table_row_stride + max_pages) * 4 : 0}};
  for (const auto& a : in)
    if (!aligned_to(a.p, 4)) return GDN_ERR_MISALIGNED;
  for (const auto& a : out)
    if (!aligned_to(a.p, 4)) return GDN_ERR_MISALIGNED;
  if (!aligned16(slot_map) || !aligned16(positions)) return GDN_ERR_MISALIGNED;
  if (outputs_overlap(in, out)) return GDN_ERR_INVALID_ARG;
  gdn::PagePlanArgs a{lens, want, N, block_table, table_row_stride, max_pages, free_pages,
                      free_count, num_pages, page_size, token_capacity, new_lens, cu_new,
                      slot_map, positions, new_count, info, stream};
  return from_cuda(gdn::launch_page_plan(a));
}

gdn_status gdn_rope_inv_freq(int rope_dims, double base, double factor, double context,
                             double beta_fast, double beta_slow, double* out,
                             cudaStream_t stream) {
  if (rope_dims < 0 || rope_dims % 2 != 0 || rope_dims > 256) return GDN_ERR_UNSUPPORTED;
  if (!(base > 1.0) || !(factor >= 1.0) || !(context >= 0.0) ||
      (context > 0.0 && !(beta_fast > beta_slow)))
    return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(base) || !std::isfinite(factor) || !std::isfinite(context) ||
      (context > 0.0 && !(std::isfinite(beta_fast) && std::isfinite(beta_slow))))
    return GDN_ERR_INVALID_ARG;
  if (rope_dims == 0) return GDN_OK;
  if (!out) return GDN_ERR_INVALID_ARG;
  if (!aligned_to(out, 8)) return GDN_ERR_MISALIGNED;
  return from_cuda(gdn::launch_rope_inv_freq(rope_dims, base, factor, context, beta_fast,
                                             beta_slow, out, stream));
}

gdn_status gdn_qk_norm_rope(const void* q, int64_t q_row_stride, const void* k,
                            int64_t k_row_stride, const void* v, int64_t v_row_stride,
                            gdn_dtype x_dtype, const void* q_norm_w, const void* k_norm_w,
                            gdn_dtype w_dtype, float eps, const int32_t* positions, int axes,
                            const double* inv_freq, int rope_dims, int interleaved,
                            float rope_scale, const int32_t* slot_map, int64_t T, int H_q,
                            int H_kv, int head_dim, void* q_out, void* k_cache,
                            int64_t k_page_stride, int64_t k_token_stride,
                            int64_t k_head_stride, void* v_cache, int64_t v_page_stride,
                            int64_t v_token_stride, int64_t v_head_stride, int num_pages,
                            int page_size, gdn_dtype out_dtype, cudaStream_t stream) {
  if (!paged_dim(head_dim)) return GDN_ERR_UNSUPPORTED;
  if (rope_dims < 0 || rope_dims % 2 != 0 || rope_dims > head_dim) return GDN_ERR_UNSUPPORTED;
  if (!half_dtype(out_dtype)) return GDN_ERR_UNSUPPORTED;
  if (!valid_dtype3(x_dtype) || !valid_dtype3(w_dtype) || !(eps >= 0.f) || T < 0 ||
      T > (int64_t)1 << 30)
    return GDN_ERR_INVALID_ARG;
  if ((!q && !k) || (!k) != (!v)) return T == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if ((q && (H_q <= 0 || H_q > 1 << 16)) || (k && (H_kv <= 0 || H_kv > 1 << 16)))
    return GDN_ERR_INVALID_ARG;
  if (rope_dims > 0 && axes != 1 && axes != 3) return GDN_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)H_q * head_dim, kv_row = (int64_t)H_kv * head_dim;
  if ((q && q_row_stride < q_row) || (k && (k_row_stride < kv_row || v_row_stride < kv_row)))
    return GDN_ERR_INVALID_ARG;
  if ((q && !stride_ok(q_row_stride, x_dtype)) ||
      (k && (!stride_ok(k_row_stride, x_dtype) || !stride_ok(v_row_stride, x_dtype))))
    return GDN_ERR_MISALIGNED;
  const gdn::PageStrides ks{k_page_stride, k_token_stride, k_head_stride},
      vs{v_page_stride, v_token_stride, v_head_stride};
  if (k) {
    gdn_status st = check_cache(k_cache, ks, num_pages, page_size, head_dim);
    if (st == GDN_OK) st = check_cache(v_cache, vs, num_pages, page_size, head_dim);
    if (st != GDN_OK) return st;
    if (!slot_map && T > (int64_t)num_pages * page_size) return GDN_ERR_INVALID_ARG;
  }
  if (T == 0) return GDN_OK;
  if ((q && !q_out) || (rope_dims > 0 && (!positions || !inv_freq))) return GDN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || (q && !aligned16(q_out)))
    return GDN_ERR_MISALIGNED;
  const int wb = gdn::elem_bytes(w_dtype);
  if (!aligned_to(q_norm_w, wb) || !aligned_to(k_norm_w, wb) || !aligned_to(positions, 4) ||
      !aligned_to(inv_freq, 8) || !aligned_to(slot_map, 4))
    return GDN_ERR_MISALIGNED;
  if (q) {
    const size_t xb = (size_t)gdn::elem_bytes(x_dtype);
    const size_t in = ((size_t)(T - 1) * q_row_stride + q_row) * xb;
    const size_t out = (size_t)T * q_row * 2;
    const bool same = q == q_out && x_dtype == out_dtype && q_row_stride == q_row;
    if (!same && overlap(q, in, q_out, out)) return GDN_ERR_INVALID_ARG;
    const Extent small[] = {{q_norm_w, (size_t)head_dim * wb}, {k_norm_w, (size_t)head_dim * wb},
                            {positions, rope_dims > 0 ? (size_t)axes * T * 4 : 0},
                            {inv_freq, (size_t)rope_dims * 4}, {slot_map, (size_t)T * 4}};
    for (const Extent& e : small)
      if (overlap(e.p, e.n, q_out, out)) return GDN_ERR_INVALID_ARG;
    if (k) {
      const size_t kn = ((size_t)(T - 1) * k_row_stride + kv_row) * xb;
      const size_t vn = ((size_t)(T - 1) * v_row_stride + kv_row) * xb;
      if (overlap(k, kn, q_out, out) || overlap(v, vn, q_out, out)) return GDN_ERR_INVALID_ARG;
    }
  }
  gdn::NormRopeArgs a{q, k, v, q_row_stride, k_row_stride, v_row_stride, x_dtype, q_norm_w,
                      k_norm_w, w_dtype, eps, positions, axes, inv_freq, rope_dims, interleaved,
                      rope_scale, slot_map, T, H_q, H_kv, head_dim, q_out, k_cache, v_cache, ks,
                      vs, num_pages, page_size, out_dtype, stream};
  return from_cuda(gdn::launch_qk_norm_rope(a));
}

size_t gdn_paged_attention_decode_workspace(int H_q, int H_kv, int head_dim) {
  if (H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || !paged_dim(head_dim)) return 0;
  return gdn::paged_decode_workspace(H_q / H_kv, head_dim);
}

gdn_status gdn_paged_attention_decode(const void* q, int64_t q_row_stride, const void* k_cache,
                                      int64_t k_page_stride, int64_t k_token_stride,
                                      int64_t k_head_stride, const void* v_cache,
                                      int64_t v_page_stride, int64_t v_token_stride,
                                      int64_t v_head_stride, gdn_dtype kv_dtype, int num_pages,
                                      int page_size, const int32_t* block_table,
                                      int64_t table_row_stride, int max_pages,
                                      const int32_t* kv_lens, const void* gate,
                                      int64_t gate_row_stride, int N, int H_q, int H_kv,
                                      int head_dim, float scale, void* o, gdn_dtype o_dtype,
                                      float* lse, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream) {
  if (!paged_dim(head_dim) || !half_dtype(kv_dtype)) return GDN_ERR_UNSUPPORTED;
  if (H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || H_q > 65535 || N < 0 || N > 65535 ||
      !valid_dtype3(o_dtype) || !(scale == scale))
    return GDN_ERR_INVALID_ARG;
  if (H_q / H_kv > 16) return GDN_ERR_UNSUPPORTED;
  // units of work are counted in 64 bits, times a few thousand
  if ((double)N * H_kv * max_pages * page_size > 9e15) return GDN_ERR_UNSUPPORTED;
  const int64_t row = (int64_t)H_q * head_dim;
  if (q_row_stride < row || (gate && gate_row_stride < row) || max_pages <= 0 ||
      table_row_stride < max_pages || (int64_t)max_pages * page_size > INT32_MAX)
    return GDN_ERR_INVALID_ARG;
  const gdn::PageStrides ks{k_page_stride, k_token_stride, k_head_stride},
      vs{v_page_stride, v_token_stride, v_head_stride};
  gdn_status st = check_cache(k_cache, ks, num_pages, page_size, head_dim);
  if (st == GDN_OK) st = check_cache(v_cache, vs, num_pages, page_size, head_dim);
  if (st != GDN_OK) return st;
  if (N == 0) return GDN_OK;
  if (!q || !block_table || !kv_lens || !o || !workspace) return GDN_ERR_INVALID_ARG;
  if (workspace_bytes < gdn::paged_decode_workspace(H_q / H_kv, head_dim))
    return GDN_ERR_INVALID_ARG;
  if (!aligned16(q) || q_row_stride % 8 != 0 || !aligned16(gate) ||
      (gate && gate_row_stride % 8 != 0) || !aligned16(o) || !aligned16(workspace) ||
      !aligned_to(block_table, 4) || !aligned_to(kv_lens, 4) || !aligned_to(lse, 4))
    return GDN_ERR_MISALIGNED;
  const Extent in[] = {{q, ((size_t)(N - 1) * q_row_stride + row) * 2},
                       {gate, ((size_t)(N - 1) * gate_row_stride + row) * 2},
                       {kv_lens, (size_t)N * 4},
                       {block_table, ((size_t)(N - 1) * table_row_stride + max_pages) * 4}};
  const Extent out[] = {{o, (size_t)N * row * gdn::elem_bytes(o_dtype)},
                        {lse, (size_t)N * H_q * 4},
                        {workspace, gdn::paged_decode_workspace(H_q / H_kv, head_dim)}};
  if (outputs_overlap(in, out)) return GDN_ERR_INVALID_ARG;
  gdn::PagedDecodeArgs a{q, q_row_stride, k_cache, v_cache, ks, vs, kv_dtype, num_pages,
                         page_size, block_table, table_row_stride, max_pages, kv_lens, gate,
                         gate_row_stride, N, H_q, H_kv, head_dim, scale, o, o_dtype, lse,
                         workspace, stream};
  return from_cuda(gdn::launch_paged_decode(a));
}

gdn_status gdn_attention_status(const void* workspace, cudaStream_t stream) {
  if (!workspace) return GDN_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return GDN_ERR_MISALIGNED;
  int word = 0;
  if (gdn::attention_status_word(workspace, stream, &word) != cudaSuccess) return GDN_ERR_CUDA;
  if (word == 1) return GDN_ERR_TIMEOUT;
  if (word == 2) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

}  // extern "C"
