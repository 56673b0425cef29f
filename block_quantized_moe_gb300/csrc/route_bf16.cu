// Routing of bf16 logits.
#include "route_forward.cuh"

namespace ftmoe {

cudaError_t launch_route_bf16(const RouteArgs& a, cudaStream_t st) { return route::launch_as<ElemBf16>(a, st); }

}  // namespace ftmoe
