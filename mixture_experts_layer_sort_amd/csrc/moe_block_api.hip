// C ABI entry points of the scored routing and of the end of an expert block,
// with their gradients: host-side argument checks, then launches on the caller's
// stream.  Nothing here allocates device memory, synchronises or reads device data.
#include <cmath>

#include "../../include/moe.h"
#include "moe_norm.h"
#include "moe_router.h"

using namespace moe;

namespace {

moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
template <class... P>
bool aligned_to(size_t n, const P*... p) {  // null is
  return (aligned(p, n) && ...);
}

moe_status check_router(const moe_router* r, int32_t T) {
  if (!r || T < 0) return MOE_ERR_INVALID_ARG;
  const int E = r->num_experts, k = r->top_k, G = r->num_groups;
  if (E < 1 || E > 1024 || k < 1 || k > 32 || k > E) return MOE_ERR_UNSUPPORTED;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (G < 1 || G > E || E % G) return MOE_ERR_UNSUPPORTED;
  if (r->topk_groups < 1 || r->topk_groups > G || r->topk_groups * (E / G) < k) return MOE_ERR_UNSUPPORTED;
  if (r->group_top != 1 && r->group_top != 2) return MOE_ERR_UNSUPPORTED;
  if (r->group_top > E / G) return MOE_ERR_UNSUPPORTED;
  if (r->renormalise != 0 && r->renormalise != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(r->scale)) return MOE_ERR_INVALID_ARG;
  return (long long)T * k > (1LL << 24) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_stride(int64_t stride, int32_t E) {
  if (stride < E) return MOE_ERR_INVALID_ARG;
  return stride > (1LL << 32) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

RouterArgs router_args(const moe_router* r, int32_t T, const float* logits, int64_t stride) {
  RouterArgs a = {};
  a.logits = logits, a.ldl = stride;
  a.T = T, a.E = r->num_experts, a.k = r->top_k;
  a.softmax = r->score == MOE_SCORE_SOFTMAX, a.renorm = r->renormalise != 0;
  a.scale = r->scale;
  return a;
}

moe_status check_norm(int32_t T, int32_t H, int32_t k) {
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (H < 8 || H > 16384 || H % 8 || k < 0 || k > 32) return MOE_ERR_UNSUPPORTED;
  return T > (1 << 24) || (long long)T * k > (1LL << 24) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_route_scores(const moe_router* r, int32_t T, const float* logits, int64_t logits_stride,
                            const float* bias, int32_t* topk_ids, float* topk_w, hipStream_t stream) {
  moe_status st = check_router(r, T);
  if (st != MOE_OK || T == 0) return st;
  if (!logits || !topk_ids || !topk_w || !aligned_to(4, logits, bias, topk_ids, topk_w)) return MOE_ERR_INVALID_ARG;
  if ((st = check_stride(logits_stride, r->num_experts)) != MOE_OK) return st;
  RouterArgs a = router_args(r, T, logits, logits_stride);
  a.bias = bias;
  a.G = r->num_groups, a.KG = r->topk_groups, a.top = r->group_top;
  a.ids = topk_ids, a.w = topk_w;
  return launched(launch_route_scores(a, stream));
}

moe_status moe_route_scores_backward(const moe_router* r, int32_t T, const float* logits, int64_t logits_stride,
                                     const int32_t* topk_ids, const float* d_topk_w, const uint8_t* token_mask,
                                     int32_t accumulate, float* d_logits, int64_t d_logits_stride,
                                     hipStream_t stream) {
  moe_status st = check_router(r, T);
  if (st != MOE_OK || T == 0) return st;
  if (!logits || !topk_ids || !d_topk_w || !d_logits) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(4, logits, topk_ids, d_topk_w, d_logits)) return MOE_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if ((st = check_stride(logits_stride, r->num_experts)) != MOE_OK) return st;
  if ((st = check_stride(d_logits_stride, r->num_experts)) != MOE_OK) return st;
  RouterArgs a = router_args(r, T, logits, logits_stride);
  a.ids = const_cast<int32_t*>(topk_ids);
  a.d_w = d_topk_w, a.mask = token_mask;
  a.accumulate = accumulate != 0;
  a.d_logits = d_logits, a.ldd = d_logits_stride;
  return launched(launch_route_scores_backward(a, stream));
}

moe_status moe_combine_norm(int32_t T, int32_t H, int32_t k, const uint16_t* y, const float* topk_w,
                            const uint16_t* shared, const float* shared_gate, const uint16_t* residual,
                            const uint16_t* post_weight, const uint16_t* next_weight, float eps, float scale,
                            uint16_t* out, uint16_t* normed, hipStream_t stream) {
  const moe_status st = check_norm(T, H, k);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f && std::isfinite(eps)) || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if ((k > 0) != (y != nullptr) || (k > 0) != (topk_w != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!out || (k == 0 && !shared) || (shared_gate && !shared)) return MOE_ERR_INVALID_ARG;
  if ((next_weight != nullptr) != (normed != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(16, y, shared, residual, post_weight, next_weight, out, normed)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(4, topk_w, shared_gate)) return MOE_ERR_INVALID_ARG;
  NormArgs a = {};
  a.T = T, a.H = H, a.k = k;
  a.y = y, a.w = topk_w, a.shared = shared, a.gate = shared_gate, a.residual = residual;
  a.post = post_weight, a.next = next_weight, a.eps = eps, a.scale = scale;
  a.out = out, a.normed = normed;
  return launched(launch_combine_norm(a, stream));
}

size_t moe_combine_norm_backward_workspace_bytes(int32_t max_T, int32_t H) {
  if (max_T < 1 || check_norm(max_T, H, 0) != MOE_OK) return 0;
  return norm_backward_bytes(max_T, H);
}

moe_status moe_combine_norm_backward(int32_t T, int32_t H, int32_t k, const uint16_t* y, const float* topk_w,
                                     const uint16_t* shared, const float* shared_gate, const uint16_t* out,
                                     const uint16_t* post_weight, const uint16_t* next_weight, float eps, float scale,
                                     const uint16_t* d_out, const uint16_t* d_normed, uint16_t* d_residual,
                                     uint16_t* d_y, float* d_topk_w, uint16_t* d_shared, float* d_gate,
                                     float* d_post_weight, float* d_next_weight, void* ws, size_t ws_bytes,
                                     hipStream_t stream) {
  const moe_status st = check_norm(T, H, k);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f && std::isfinite(eps)) || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if ((k > 0) != (y != nullptr) || (k > 0) != (topk_w != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((k == 0 && !shared) || (shared_gate && !shared)) return MOE_ERR_INVALID_ARG;
  if ((next_weight != nullptr) != (d_normed != nullptr) || (next_weight && !out)) return MOE_ERR_INVALID_ARG;
  if (!d_out && !d_normed) return MOE_ERR_INVALID_ARG;
  if ((next_weight != nullptr) != (d_next_weight != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((post_weight != nullptr) != (d_post_weight != nullptr)) return MOE_ERR_INVALID_ARG;
  if (((d_y || d_topk_w) && k == 0) || (d_shared && !shared) || (d_gate && !shared_gate)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(16, y, shared, out, post_weight, next_weight, d_out, d_normed, d_residual, d_y, d_shared))
    return MOE_ERR_INVALID_ARG;
  if (!aligned_to(4, topk_w, shared_gate, d_topk_w, d_gate, d_post_weight, d_next_weight)) return MOE_ERR_INVALID_ARG;
  if (post_weight || next_weight) {
    if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < norm_backward_bytes(T, H)) return MOE_ERR_WORKSPACE;
  }
  NormArgs a = {};
  a.T = T, a.H = H, a.k = k;
  a.y = y, a.w = topk_w, a.shared = shared, a.gate = shared_gate;
  a.post = post_weight, a.next = next_weight, a.eps = eps, a.scale = scale;
  a.out = const_cast<uint16_t*>(out);
  a.d_out = d_out, a.d_normed = d_normed, a.d_residual = d_residual, a.d_y = d_y, a.d_w = d_topk_w;
  a.d_shared = d_shared, a.d_gate = d_gate, a.d_post = d_post_weight, a.d_next = d_next_weight;
  a.part = (float*)ws;
  return launched(launch_combine_norm_backward(a, stream));
}

}  // extern "C"
