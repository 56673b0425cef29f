// Routing of fp16 logits.
#include "route_forward.cuh"

namespace ftmoe {

cudaError_t launch_route_fp16(const RouteArgs& a, cudaStream_t st) { return route::launch_as<ElemF16>(a, st); }

}  // namespace ftmoe
