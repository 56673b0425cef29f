// Gradient of the routing weights: a closed form in the saved weights (see
// ftmoe_route_tokens_backward), so that only plain softmax reads every logit. Half a warp a token
// (a warp above 16 slots or 512 experts) puts the chosen experts' terms in a row of shared memory
// (zero otherwise, and again after it) and writes the row of dlogits whole. An expert that is
// chosen twice gets both terms.
// Measured on GB300: 32,768 tokens of 256 experts, plain softmax, bf16: 11.8 us (36 MB, 5.3 us of
// memory; a warp a token 13.6, a quarter of a warp 17). Latency bounds it: issue slots are 53% busy, and
// most stalls wait for shared memory and exchanges. (The next row is read before its routes are known;
// read only where one is active, behind its ids, the kernel takes 15.5 us.) Sigmoid, renormalised, top-8,
// fp32 logits and bf16 gradients: 13.5 us, most stalls wait for the chosen logits.
#include "route.cuh"

namespace ftmoe {

namespace route {

constexpr int kThreads = 256;  // (a row of shared memory a token: 32 KB for 1,024 experts, 16 tokens of 512)
constexpr int kBlocksPerSm = 4;

// what a lane reads of a token's routes: its slot
struct Slot {
  int id;
  float w, dw;
  __device__ __forceinline__ void load(const RouteArgs& a, int64_t token, int lane, int topk) {
    id = -1;
    w = dw = 0.0f;
    if (lane < topk && token < a.tokens) {
      const int64_t at = token * topk + lane;
      id = a.ids[at];
      w = a.weights[at];
      dw = a.dweights[at];
    }
  }
};

// over the kLanes lanes of a token
template <int kLanes>
__device__ __forceinline__ float token_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <int kLanes>
__device__ __forceinline__ float token_top(float v) {
  if constexpr (kLanes == 32) {
    return warp_top(v);
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}

template <typename Elem, typename Out, int kPer, int kLanes>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ float4 rows[];
  pdl_wait();
  pdl_trigger();
  const int warp_lane = threadIdx.x & 31, first = warp_lane & ~(kLanes - 1);  // the token's first lane
  const int lane = warp_lane - first;
  const uint32_t lanes = (kLanes < 32 ? (1u << kLanes) - 1u : kFull) << first;
  const int E = a.router.num_experts, topk = a.router.topk, e0 = lane * kPer;
  float* const part = reinterpret_cast<float*>(rows) + (threadIdx.x / kLanes) * (kLanes * kPer);
  const bool softmax = a.router.score == FTMOE_SCORE_SOFTMAX, whole = softmax && !a.router.renormalize;
  const float per_scale = 1.0f / a.router.scale;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / kLanes);
  int64_t token = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  Row<Elem, kPer> next_row;
  Slot next;
#pragma unroll
  for (int j = 0; j < kPer; ++j) part[lane + kLanes * j] = 0.0f;  // and again after each token
  __syncwarp();
  next.load(a, token, lane, topk);
  if (whole && token < a.tokens) next_row.load(static_cast<const typename Elem::T*>(a.logits) + token * a.ld, lane, E, a.vec);
  // (the lanes of a warp go round together: its first token is there as long as any is)
  for (; token - first / kLanes < a.tokens; token += stride) {
    const bool there = token < a.tokens;
    const typename Elem::T* row = static_cast<const typename Elem::T*>(a.logits) + token * a.ld;
    Slot s = next;
    const Row<Elem, kPer> this_row = next_row;
    next.load(a, token + stride, lane, topk);
    if (whole && token + stride < a.tokens) next_row.load(row + stride * a.ld, lane, E, a.vec);
    if (s.id >= E) raise_error(FTMOE_ERR_EXPERT_ID_RANGE);
    if (s.id < 0 || s.id >= E) s.id = -1, s.w = 0.0f, s.dw = 0.0f;
    float r = s.w * s.dw;
    const float total = token_sum<kLanes>(r);
    if (a.router.renormalize) r = fmaf(-s.w, total * per_scale, r);
    if (!softmax && s.id >= 0) r *= 1.0f / (1.0f + expf(taken(Elem::get(row[s.id]))));
    // the terms in the row. An id that occurs twice (a lane reads another's number in its place): each
    // of its lanes puts their sum there
    const bool active = s.id >= 0;
    if (active) part[s.id] = __int_as_float(lane);
    __syncwarp();
    const bool second = active && __float_as_int(part[s.id]) != lane;
    if (__any_sync(kFull, second)) {
      const uint32_t same = __match_any_sync(kFull, active ? s.id + (first << 16) : -1);
      float all = 0.0f;
      for (int t = 0; t < topk; ++t) {
        const float other = __shfl_sync(kFull, r, first + t);
        all += (same >> (first + t)) & 1u ? other : 0.0f;
      }
      r = all;
    }
    __syncwarp();
    if (active) part[s.id] = r;
    __syncwarp();

    float d[kPer];
    if constexpr (kPer >= 4) {
#pragma unroll
      for (int j = 0; j < kPer; j += 4) {
        const float4 q = *reinterpret_cast<const float4*>(part + e0 + j);
        d[j] = q.x, d[j + 1] = q.y, d[j + 2] = q.z, d[j + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) d[j] = part[e0 + j];
    }
    __syncwarp();
    if (active) part[s.id] = 0.0f;
    __syncwarp();
    const bool any = (__ballot_sync(kFull, active) & lanes) != 0u;
    if (whole) {
      float x[kPer], top = -INFINITY, sum = 0.0f;
      this_row.get_taken(x);
#pragma unroll
      for (int j = 0; j < kPer; ++j) top = fmaxf(top, x[j]);
      top = token_top<kLanes>(top);
#pragma unroll
      for (int j = 0; j < kPer; ++j) sum += x[j] = exp2_fast((x[j] - top) * kLog2e);
      const float f = total * reciprocal(token_sum<kLanes>(sum));
      if (any && top > -INFINITY) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) d[j] = fmaf(-x[j], f, d[j]);
      }
    }
    typename Out::T* out = static_cast<typename Out::T*>(a.dlogits) + token * a.ld_dlogits;
    if constexpr (kPer >= 8) {
#pragma unroll
      for (int c = 0; c < kPer; c += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = d[c + j];
        const int n = there ? E - e0 - c : 0;
        if (n > 0) elem_store8<Out>(out + e0 + c, a.vec_out, n, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (there && e0 + j < E) out[e0 + j] = Out::put(d[j]);
    }
  }
}

}  // namespace route

cudaError_t launch_route_backward(RouteArgs a, cudaStream_t st) {
  using namespace route;
  OverlapLaunch overlap;
  a.vec_out = elem_vec_ok(a.dlogits, a.ld_dlogits, a.dlogits_dtype == FTMOE_OUT_FP32 ? 4 : 2);
  // half a warp a token where its slots and experts fit: two tokens share what a warp does once
  const bool half = a.router.topk <= 16 && a.router.num_experts <= 512;
  return with_elem(a.dtype, [&](auto elem) {
    return with_elem(a.dlogits_dtype, [&](auto out) {
      using E = decltype(elem);
      using Out = decltype(out);
      return with_per(half ? 2 * a.router.num_experts : a.router.num_experts, [&](auto per) {
        constexpr int kPer = decltype(per)::value;
        a.vec = Row<E, kPer>::vec_ok(a.logits, a.ld, a.router.num_experts);
        const int64_t tokens = kThreads / (half ? 16 : 32);  // of a block at a time
        return launch_kernel(half ? route_backward_kernel<E, Out, kPer, 16> : route_backward_kernel<E, Out, kPer, 32>,
                             dim3((unsigned)std::min<int64_t>(cdiv(a.tokens, tokens), 152 * kBlocksPerSm)), dim3(kThreads),
                             kThreads * kPer * sizeof(float), st, true, a);
      });
    });
  });
}

FTMOE_DEFINE_ERR_READER(read_err_route)

}  // namespace ftmoe
