// Routing of fp32 logits, and the choice by the logits' type (each in a translation unit of its own).
#include "route_forward.cuh"

namespace ftmoe {

cudaError_t launch_route(const RouteArgs& a, cudaStream_t st) {
  if (a.dtype == FTMOE_OUT_BF16) return launch_route_bf16(a, st);
  if (a.dtype == FTMOE_OUT_FP16) return launch_route_fp16(a, st);
  return route::launch_as<ElemF32>(a, st);
}

}  // namespace ftmoe
