// C ABI of the operators around the experts' products (routing, gradient norm, AdamW): argument
// checks on the host, then launches on the caller's stream (no allocation, no synchronisation).
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "internal.h"

using namespace ftmoe;

namespace {

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline ftmoe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FTMOE_OK : FTMOE_CUDA_ERROR; }

bool half_dtype(int32_t d) { return d == FTMOE_OUT_BF16 || d == FTMOE_OUT_FP16; }
bool any_dtype(int32_t d) { return half_dtype(d) || d == FTMOE_OUT_FP32; }
bool aligned(const void* p, int32_t dtype) { return (uintptr_t)p % (dtype == FTMOE_OUT_FP32 ? 4 : 2) == 0; }
bool aligned4(const void* p) { return (uintptr_t)p % 4 == 0; }
bool aligned8(const void* p) { return (uintptr_t)p % 8 == 0; }

constexpr int64_t kMaxDim = (int64_t)1 << 31;
// elements of a tensor: its units of work fit 30 bits
constexpr int64_t kMaxElements = (int64_t)1 << 42;

ftmoe_status check_router(const ftmoe_router* r) {
  if (!r || r->num_experts <= 0 || r->topk <= 0 || r->groups <= 0 || r->num_experts % r->groups != 0 ||
      r->group_topk <= 0 || r->group_topk > r->groups || (r->group_best != 1 && r->group_best != 2) ||
      (r->score != FTMOE_SCORE_SOFTMAX && r->score != FTMOE_SCORE_SIGMOID) || (r->renormalize != 0 && r->renormalize != 1) ||
      !(r->scale >= 1e-30f) || !(r->scale <= 1e30f) || r->topk > (int64_t)r->group_topk * (r->num_experts / r->groups))
    return FTMOE_INVALID_ARG;
  if (r->num_experts > kRouteMaxExperts || r->topk > kRouteMaxTopk || r->groups > kRouteMaxGroups) return FTMOE_UNSUPPORTED;
  return FTMOE_OK;
}

bool check_grads(const ftmoe_grad_list* list) {
  if (!list || list->count < 0 || !any_dtype(list->dtype) || (list->count > 0 && !list->grads)) return false;
  for (int i = 0; i < list->count; ++i) {
    const ftmoe_grad& g = list->grads[i];
    if (g.n < 0 || g.n >= kMaxElements || (g.n > 0 && (!g.grad || !aligned(g.grad, list->dtype)))) return false;
  }
  return true;
}

}  // namespace

extern "C" {

ftmoe_status ftmoe_route_tokens(const void* logits, int32_t dtype, int64_t tokens, int64_t ld,
                                const ftmoe_router* router, const float* bias, const int32_t* tokens_dev,
                                int32_t* expert_ids, float* weights, void* stream) {
  if (tokens < 0 || tokens >= kMaxDim || !any_dtype(dtype)) return FTMOE_INVALID_ARG;
  const ftmoe_status st = check_router(router);
  if (st != FTMOE_OK) return st;
  if (ld < router->num_experts || ld >= kMaxDim) return FTMOE_INVALID_ARG;
  if (tokens == 0) return FTMOE_OK;
  if (!logits || !expert_ids || !weights || !aligned(logits, dtype) || !aligned4(bias) || !aligned4(tokens_dev) ||
      !aligned4(expert_ids) || !aligned4(weights))
    return FTMOE_INVALID_ARG;
  RouteArgs a = {};
  a.logits = logits;
  a.dtype = dtype;
  a.tokens = tokens;
  a.ld = ld;
  a.router = *router;
  a.bias = bias;
  a.tokens_dev = tokens_dev;
  a.ids_out = expert_ids;
  a.weights_out = weights;
  return from_cuda(launch_route(a, as_stream(stream)));
}

ftmoe_status ftmoe_route_tokens_backward(const void* logits, int32_t dtype, int64_t tokens, int64_t ld,
                                         const ftmoe_router* router, const int32_t* expert_ids, const float* weights,
                                         const float* dweights, void* dlogits, int32_t dlogits_dtype,
                                         int64_t ld_dlogits, void* stream) {
  if (tokens < 0 || tokens >= kMaxDim || !any_dtype(dtype) || !any_dtype(dlogits_dtype)) return FTMOE_INVALID_ARG;
  const ftmoe_status st = check_router(router);
  if (st != FTMOE_OK) return st;
  if (ld < router->num_experts || ld >= kMaxDim || ld_dlogits < router->num_experts || ld_dlogits >= kMaxDim)
    return FTMOE_INVALID_ARG;
  if (tokens == 0) return FTMOE_OK;
  if (!logits || !expert_ids || !weights || !dweights || !dlogits || !aligned(logits, dtype) || !aligned4(expert_ids) ||
      !aligned4(weights) || !aligned4(dweights) || !aligned(dlogits, dlogits_dtype))
    return FTMOE_INVALID_ARG;
  RouteArgs a = {};
  a.logits = logits;
  a.dtype = dtype;
  a.tokens = tokens;
  a.ld = ld;
  a.router = *router;
  a.ids = expert_ids;
  a.weights = weights;
  a.dweights = dweights;
  a.dlogits = dlogits;
  a.dlogits_dtype = dlogits_dtype;
  a.ld_dlogits = ld_dlogits;
  return from_cuda(launch_route_backward(a, as_stream(stream)));
}

size_t ftmoe_grad_norm_workspace_bytes(const ftmoe_grad_list* list) {
  return check_grads(list) ? grad_norm_workspace(*list) : 0;
}

ftmoe_status ftmoe_grad_norm(const ftmoe_grad_list* list, float scale, float max_norm, void* workspace,
                             size_t workspace_bytes, float* result, void* stream) {
  if (!check_grads(list) || !(scale > 0.0f) || !(scale < INFINITY) || !(max_norm > 0.0f)) return FTMOE_INVALID_ARG;
  if (!workspace || !aligned8(workspace) || !result || !aligned4(result)) return FTMOE_INVALID_ARG;
  if (workspace_bytes < grad_norm_workspace(*list)) return FTMOE_WORKSPACE_TOO_SMALL;
  return from_cuda(launch_grad_norm(*list, scale, max_norm, static_cast<double*>(workspace), result, as_stream(stream)));
}

ftmoe_status ftmoe_adamw_step(const ftmoe_adamw_list* list, const ftmoe_adamw* opt, void* stream) {
  if (!list || !opt || list->count < 0 || !any_dtype(list->param_dtype) || !any_dtype(list->grad_dtype) ||
      (list->copy_dtype != -1 && !half_dtype(list->copy_dtype)) ||
      (list->moments != FTMOE_MOMENTS_FP32 && list->moments != FTMOE_MOMENTS_8BIT) || (list->count > 0 && !list->tensors))
    return FTMOE_INVALID_ARG;
  if (!(std::fabs(opt->lr) <= FLT_MAX) || !(std::fabs(opt->weight_decay) <= FLT_MAX) || !(opt->eps >= 1e-30) || !(opt->eps <= 1e30) ||
      !(opt->beta1 >= 0.0) || !(opt->beta1 < 1.0) || !(opt->beta2 >= 0.0) || !(opt->beta2 < 1.0) ||
      (!opt->step_dev && opt->step < 1))
    return FTMOE_INVALID_ARG;
  if (!aligned4(opt->lr_dev) || !aligned8(opt->step_dev) || !aligned4(opt->grad_scale)) return FTMOE_INVALID_ARG;
  const bool narrow = list->moments == FTMOE_MOMENTS_8BIT;
  for (int i = 0; i < list->count; ++i) {
    const ftmoe_adamw_tensor& t = list->tensors[i];
    if (t.n < 0 || t.n >= kMaxElements) return FTMOE_INVALID_ARG;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.m || !t.v || (narrow && (!t.m_scales || !t.v_scales)) ||
        (!narrow && (t.m_scales || t.v_scales)) || (list->copy_dtype == -1) != (t.copy == nullptr))
      return FTMOE_INVALID_ARG;
    if (!aligned(t.param, list->param_dtype) || !aligned(t.grad, list->grad_dtype) ||
        (!narrow && (!aligned4(t.m) || !aligned4(t.v))) || !aligned(t.copy, list->copy_dtype))
      return FTMOE_INVALID_ARG;
  }
  AdamwConstants c = {};
  c.lr = (float)opt->lr;
  c.beta1 = (float)opt->beta1;
  c.beta2 = (float)opt->beta2;
  c.rest1 = (float)(1.0 - opt->beta1);
  c.rest2 = (float)(1.0 - opt->beta2);
  c.eps = (float)opt->eps;
  c.weight_decay = (float)opt->weight_decay;
  c.ln_beta1 = (float)std::log(opt->beta1);
  c.ln_beta2 = (float)std::log(opt->beta2);
  if (!opt->step_dev) {
    c.correction1 = (float)(1.0 / (1.0 - std::pow(opt->beta1, (double)opt->step)));
    c.correction2 = (float)(1.0 / std::sqrt(1.0 - std::pow(opt->beta2, (double)opt->step)));
  }
  c.one = 1.0f;
  c.seed = opt->seed;
  c.step = opt->step;
  c.lr_dev = opt->lr_dev;
  c.step_dev = opt->step_dev;
  c.grad_scale = opt->grad_scale;
  return from_cuda(launch_adamw(*list, c, as_stream(stream)));
}

}  // extern "C"
