// Routing of tokens to experts from the router's logits, and its gradient.
//
// Forward, per token, with x its logits: s = softmax(x) or 1 / (1 + exp(-x)), value = s + bias;
// groups of consecutive experts are ranked by the sum of their 1 or 2 best values and all but the
// best groups left out; the top-k values are chosen, largest first, ties to the lower expert; the
// weights are the chosen s times the scale, renormalised to sum to it where asked.
//
// A warp per token; lane l holds the experts [l * kPer, (l + 1) * kPer), so that the lowest lane with the
// largest key is the lowest expert. Keys are order-preserving integers of fp32 values (0: never
// chosen); each of the k steps is a warp maximum (one instruction), a vote and the owner's rescan.
// Without a bias the logits themselves are the order and nothing is rounded. With one, the order of
// s + bias is that of 64 bits: fp32 values are off by less than kTolerance, so wherever two values
// that the choice depends on are nearer than that, the token's near values are taken again in 64 bits
// (route_exact), unless the logits and biases are the same, which is a tie in any precision.
//
// Backward: a closed form in the saved weights (see ftmoe_route_tokens_backward), so that only plain
// softmax reads every logit. A warp per token puts the chosen experts' terms in a row of shared
// memory and writes the row of dlogits whole.
#include <cfloat>

#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"

namespace ftmoe {

namespace route {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xffffffffu;

// fp32 -> integer of the same order, > 0 for every number; -0 and +0 are one
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (int32_t)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((int32_t)key < 0 ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// NaN and -inf take no part (-inf); +inf counts as the largest finite number
__device__ __forceinline__ float taken(float x) { return x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY; }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// a lane's logits; -inf past the last expert
template <typename Elem, int kPer>
__device__ __forceinline__ void load_row(const typename Elem::T* row, int lane, int E, bool vec, float (&x)[kPer]) {
  const int e0 = lane * kPer;
  if constexpr (kPer >= 8) {
#pragma unroll
    for (int c = 0; c < kPer; c += 8) {
      const int n = E - e0 - c;
      const Raw8<Elem> raw = raw_load8<Elem>(row + e0 + c, vec, n < 0 ? 0 : n);
      float v[8];
      raw_get8<Elem>(raw, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[c + j] = j < n ? taken(v[j]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) x[j] = e0 + j < E ? taken(Elem::get(row[e0 + j])) : -INFINITY;
  }
}

// largest logit of the row and the sum of exp(x - max) (softmax scores)
template <int kPer>
__device__ __forceinline__ void softmax_stats(const float (&x)[kPer], float& top, float& sum) {
  float m = x[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) m = fmaxf(m, x[j]);
  top = warp_max(m);
  float s = 0.0f;
  if (top > -INFINITY) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s += expf(x[j] - top);
  }
  sum = warp_sum(s);
}

// scores in fp32 (0 where an expert takes no part)
template <int kPer>
__device__ __forceinline__ void scores(const float (&x)[kPer], int32_t score, float top, float sum, float (&s)[kPer]) {
  if (score == FTMOE_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[j] = sigmoid(x[j]);
  } else {
    const float r = 1.0f / sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[j] = top > -INFINITY ? expf(x[j] - top) * r : 0.0f;
  }
}

// the two largest of two pairs
template <typename F>
__device__ __forceinline__ void merge2(F& a1, F& a2, F b1, F b2) {
  const F low = a1 < b1 ? a1 : b1;
  a1 = a1 < b1 ? b1 : a1;
  const F second = a2 < b2 ? b2 : a2;
  a2 = low < second ? second : low;
}
template <typename F>
__device__ __forceinline__ F group_score(F a1, F a2, int best) {
  return best == 2 && a2 > -INFINITY ? a1 + a2 : a1;
}

// Scores of the groups: the group's on each of its lanes where whole lanes make up a group and their
// number is a power of two (`lanes` > 0), else group g's on lane g.
template <int kPer, typename F>
__device__ __forceinline__ F group_scores(const F (&v)[kPer], int lane, int groups, int size, int lanes, int best) {
  F mine = -INFINITY;
  if (lanes > 0) {
    F a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) merge2(a1, a2, v[j], (F)-INFINITY);
    for (int o = 1; o < lanes; o <<= 1) merge2(a1, a2, __shfl_xor_sync(kFull, a1, o), __shfl_xor_sync(kFull, a2, o));
    mine = lane < groups * lanes ? group_score(a1, a2, best) : -INFINITY;
  } else {
    for (int g = 0; g < groups; ++g) {
      F a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int at = lane * kPer + j - g * size;
        merge2(a1, a2, at >= 0 && at < size ? v[j] : (F)-INFINITY, (F)-INFINITY);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) merge2(a1, a2, __shfl_xor_sync(kFull, a1, o), __shfl_xor_sync(kFull, a2, o));
      if (lane == g) mine = group_score(a1, a2, best);
    }
  }
  return mine;
}

// bit g: group g is among the group_topk best. gap: how far the worst of them is from the best of
// the others (infinite where there is none, or none that could be chosen)
template <typename F>
__device__ __forceinline__ uint32_t kept_groups(F mine, int lane, int groups, int lanes, int keep, F& gap) {
  const int step = lanes > 0 ? lanes : 1, me = lane / step;
  int rank = 0;
  for (int g = 0; g < groups; ++g) {
    const F other = __shfl_sync(kFull, mine, g * step);
    rank += other > mine || (other == mine && g < me);
  }
  const bool lead = lane % step == 0 && me < groups, in = lead && rank < keep;
  F worst = in ? mine : (F)INFINITY, next = lead && !in ? mine : (F)-INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const F w = __shfl_xor_sync(kFull, worst, o), n = __shfl_xor_sync(kFull, next, o);
    worst = w < worst ? w : worst;
    next = n > next ? n : next;
  }
  gap = next > -INFINITY ? worst - next : (F)INFINITY;
  uint32_t mask = 0;
  for (int g = 0; g < groups; ++g) mask |= (__shfl_sync(kFull, (int)in, g * step) != 0 ? 1u : 0u) << g;
  return mask;
}

// whether this bit's group holds expert e
__device__ __forceinline__ bool in_groups(uint32_t mask, int e, int size) { return (mask >> (e / size)) & 1u; }

__device__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// The choice of one token with the values in 64 bits: all of them, or (near != 0, sigmoid scores, groups
// settled by `groups_kept`) those within `window` of the values of the slots in `near`; the others
// are further from what decides than fp32 is off. Lane t gets the expert of slot t, -1 for none.
template <typename Elem, int kPer>
__device__ __noinline__ int route_exact(const RouteArgs& a, const typename Elem::T* row, int lane, uint32_t near,
                                        float slot_value, float window, uint32_t groups_kept) {
  const int E = a.router.num_experts, size = E / a.router.groups;
  float x[kPer];
  load_row<Elem, kPer>(row, lane, E, a.vec, x);
  float top = 0.0f, sum = 1.0f;
  double sum64 = 0.0;
  double v[kPer];
  if (a.router.score == FTMOE_SCORE_SOFTMAX) {
    softmax_stats(x, top, sum);
#pragma unroll 1
    for (int j = 0; j < kPer; ++j) sum64 += x[j] > -INFINITY ? exp((double)x[j] - (double)top) : 0.0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum64 += __shfl_xor_sync(kFull, sum64, o);
  }
#pragma unroll 1
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * kPer + j;
    const float b = a.bias != nullptr && e < E ? taken(a.bias[e]) : 0.0f;
    v[j] = -INFINITY;
    bool wanted = x[j] > -INFINITY && b > -INFINITY;
    if (near != 0) {
      if (wanted) wanted = in_groups(groups_kept, e, size);
      const float approx = sigmoid(x[j]) + b;
      if (wanted) v[j] = approx;
      bool close = false;
      for (int t = 0; t < a.router.topk; ++t) {
        const float c = __shfl_sync(kFull, slot_value, t);
        close = close || (((near >> t) & 1u) && fabsf(approx - c) <= window);
      }
      wanted = wanted && close;
      if (!__any_sync(kFull, wanted)) continue;
    }
    if (wanted)
      v[j] = (a.router.score == FTMOE_SCORE_SIGMOID ? sigmoid64(x[j]) : exp((double)x[j] - (double)top) / sum64) + (double)b;
  }
  if (near == 0 && a.router.groups > 1) {
    double gap;
    const double mine = group_scores<kPer, double>(v, lane, a.router.groups, size, 0, a.router.group_best);
    groups_kept = kept_groups<double>(mine, lane, a.router.groups, 0, a.router.group_topk, gap);
#pragma unroll 1
    for (int j = 0; j < kPer; ++j) {
      if (x[j] > -INFINITY && !in_groups(groups_kept, lane * kPer + j, size)) v[j] = -INFINITY;
      else if (a.bias == nullptr) v[j] = x[j];  // the order is the logits'
    }
  }
  int mine = -1;
  for (int t = 0; t < a.router.topk; ++t) {
    double best = -INFINITY;
    int at = E;
#pragma unroll 1
    for (int j = 0; j < kPer; ++j)
      if (v[j] > best) best = v[j], at = lane * kPer + j;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double other = __shfl_xor_sync(kFull, best, o);
      const int other_at = __shfl_xor_sync(kFull, at, o);
      if (other > best || (other == best && other_at < at)) best = other, at = other_at;
    }
    if (!(best > -INFINITY)) break;
    if (lane == t) mine = at;
#pragma unroll 1
    for (int j = 0; j < kPer; ++j)
      if (lane * kPer + j == at) v[j] = -INFINITY;
  }
  return mine;
}

// How far apart two fp32 values have to be for their order to be that of 64 bits: s is within
// 2^-20 of the largest score (expf and the quotient: under 4 units of 2^-24 of s each, the softmax's
// sum under 8, its argument's rounding |x - top| exp(x - top) 2^-24 < 2^-25 of the largest score), the
// sum with the bias within 2^-24 of itself; twice that for two values, and as much again to spare.
__device__ __forceinline__ float tolerance(float largest_score, float v) {
  return 0x1p-18f * largest_score + 0x1p-21f * fabsf(v);
}

template <typename Elem, int kPer>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t token = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const int E = a.router.num_experts, topk = a.router.topk, size = E / a.router.groups;
  int32_t* ids = a.ids_out + token * topk;
  float* weights = a.weights_out + token * topk;
  if (a.tokens_dev != nullptr && token >= *a.tokens_dev) {
    if (lane < topk) ids[lane] = -1, weights[lane] = 0.0f;
    return;
  }
  const typename Elem::T* row = static_cast<const typename Elem::T*>(a.logits) + token * a.ld;
  float x[kPer];
  load_row<Elem, kPer>(row, lane, E, a.vec, x);

  const bool softmax = a.router.score == FTMOE_SCORE_SOFTMAX, biased = a.bias != nullptr;
  const bool scored_groups = a.router.groups > 1 && (biased || a.router.group_best == 2);
  float top = 0.0f, sum = 1.0f;
  if (softmax && (biased || scored_groups || !a.router.renormalize)) softmax_stats(x, top, sum);

  // values: the order of the experts (-inf: never chosen)
  uint32_t key[kPer];
  int chosen = -1;       // lane t: expert of slot t
  bool exact = false;    // chosen in 64 bits already
  {
    float v[kPer];
    if (biased || scored_groups) {
      scores(x, a.router.score, top, sum, v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int e = lane * kPer + j;
        const float b = biased && e < E ? taken(a.bias[e]) : 0.0f;
        v[j] = x[j] > -INFINITY ? v[j] + b : -INFINITY;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = x[j];
    }
    const float largest_score = softmax ? 1.0f / sum : 1.0f;
    uint32_t groups_kept = 1u;
    if (a.router.groups > 1) {
      float gap, mine = group_scores<kPer, float>(v, lane, a.router.groups, size, a.group_lanes, a.router.group_best);
      groups_kept = kept_groups<float>(mine, lane, a.router.groups, a.group_lanes, a.router.group_topk, gap);
      if (scored_groups) {
        const float most = warp_max(mine > -INFINITY ? fabsf(mine) : 0.0f);
        exact = gap <= 2.0f * tolerance(largest_score, most);
        if (!biased) {
#pragma unroll
          for (int j = 0; j < kPer; ++j) v[j] = x[j];
        }
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (lane * kPer + j < E && !in_groups(groups_kept, lane * kPer + j, size)) v[j] = -INFINITY;
    }
    if (exact) {
      chosen = route_exact<Elem, kPer>(a, row, lane, 0u, 0.0f, 0.0f, 0u);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) key[j] = v[j] > -INFINITY ? key_of(v[j]) : 0u;
      uint32_t slot_key = 0u, best = 0u;
#pragma unroll
      for (int j = 0; j < kPer; ++j) best = max(best, key[j]);
      for (int t = 0; t < topk; ++t) {
        const uint32_t most = __reduce_max_sync(kFull, best);
        if (most == 0u) break;
        const int owner = __ffs(__ballot_sync(kFull, best == most)) - 1;
        int at = 0;
        if (lane == owner) {
#pragma unroll
          for (int j = kPer - 1; j >= 0; --j) at = key[j] == most ? j : at;
          best = 0u;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            key[j] = j == at ? 0u : key[j];
            best = max(best, key[j]);
          }
        }
        at = __shfl_sync(kFull, at, owner);
        if (lane == t) chosen = owner * kPer + at, slot_key = most;
      }
      if (biased) {
        // pairs of neighbours in the order, and the last chosen against the best of the rest
        const float value = chosen >= 0 ? value_of(slot_key) : 0.0f;
        const float tol = tolerance(largest_score, value);
        const float cx = chosen >= 0 ? taken(Elem::get(row[chosen])) : 0.0f, cb = chosen >= 0 ? taken(a.bias[chosen]) : 0.0f;
        const int next = __shfl_down_sync(kFull, chosen, 1);
        const float next_value = __shfl_down_sync(kFull, value, 1), next_x = __shfl_down_sync(kFull, cx, 1),
                    next_b = __shfl_down_sync(kFull, cb, 1);
        bool close = lane + 1 < topk && next >= 0 && value - next_value <= tol && (cx != next_x || cb != next_b);
        const float last = __shfl_sync(kFull, value, topk - 1), last_tol = __shfl_sync(kFull, tol, topk - 1);
        const uint32_t from = __shfl_sync(kFull, chosen, topk - 1) >= 0 ? max(key_of(last - last_tol), 1u) : 0xffffffffu;
        if (__any_sync(kFull, best >= from)) {
          const float lx = __shfl_sync(kFull, cx, topk - 1), lb = __shfl_sync(kFull, cb, topk - 1);
          bool other = false;
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            if (key[j] >= from) other = other || taken(Elem::get(row[lane * kPer + j])) != lx || taken(a.bias[lane * kPer + j]) != lb;
          other = __any_sync(kFull, other);
          if (lane == topk - 1) close = other;
        }
        const uint32_t near = __ballot_sync(kFull, close);
        if (near != 0u) {
          const float widest = 2.0f * warp_max(chosen >= 0 ? tol : 0.0f);
          chosen = route_exact<Elem, kPer>(a, row, lane, softmax ? 0u : near, value, widest, groups_kept);
        }
      }
    }
  }

  const bool active = chosen >= 0;
  const float cx = active ? taken(Elem::get(row[chosen])) : -INFINITY;
  float u = 0.0f;
  if (a.router.renormalize) {
    // shares of the chosen scores, scaled so that the largest does not underflow:
    // softmax exp(x - most), sigmoid exp(-t) s with t = min(most, 0)
    const float most = warp_max(cx);
    const float t = fminf(most, 0.0f);
    if (active) u = softmax ? expf(cx - most) : 1.0f / (expf(t) + expf(t - cx));
    const float total = warp_sum(u);
    u = active ? u / total : 0.0f;
  } else if (active) {
    u = softmax ? expf(cx - top) / sum : sigmoid(cx);
  }
  if (lane < topk) {
    ids[lane] = chosen;
    weights[lane] = a.router.scale * u;
  }
}

template <typename Elem, typename Out, int kPer>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float rows[];
  const int lane = threadIdx.x & 31;
  const int64_t token = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const int E = a.router.num_experts, topk = a.router.topk;
  float* part = rows + (threadIdx.x >> 5) * (32 * kPer);
  const typename Elem::T* row = static_cast<const typename Elem::T*>(a.logits) + token * a.ld;
  const bool softmax = a.router.score == FTMOE_SCORE_SOFTMAX;

  int id = lane < topk ? a.ids[token * topk + lane] : -1;
  if (id >= E) {
    raise_error(FTMOE_ERR_EXPERT_ID_RANGE);
    id = -1;
  }
  const float w = id >= 0 ? a.weights[token * topk + lane] : 0.0f, dw = id >= 0 ? a.dweights[token * topk + lane] : 0.0f;
  float r = w * dw;
  const float total = warp_sum(r);
  if (a.router.renormalize) r = r - w * (total / a.router.scale);
  if (!softmax && id >= 0) r *= 1.0f / (1.0f + expf(taken(Elem::get(row[id]))));
  // an id that occurs twice: the first of its lanes gets the sum
  const uint32_t same = __match_any_sync(kFull, id);
  if (__any_sync(kFull, id >= 0 && (same & (same - 1u)) != 0u)) {
    float all = 0.0f;
    for (int t = 0; t < topk; ++t) {
      const float other = __shfl_sync(kFull, r, t);
      all += (same >> t) & 1u ? other : 0.0f;
    }
    r = all;
  }
  const bool lead = id >= 0 && (same & ((1u << lane) - 1u)) == 0u;

#pragma unroll
  for (int j = 0; j < kPer; ++j) part[lane + 32 * j] = 0.0f;
  __syncwarp();
  if (lead) part[id] = r;
  __syncwarp();

  const int e0 = lane * kPer;
  float d[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) d[j] = part[e0 + j];
  if (softmax && !a.router.renormalize && __any_sync(kFull, id >= 0)) {
    float x[kPer], top, sum;
    load_row<Elem, kPer>(row, lane, E, a.vec, x);
    softmax_stats(x, top, sum);
    const float f = total / sum;
    if (top > -INFINITY) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) d[j] -= expf(x[j] - top) * f;
    }
  }
  typename Out::T* out = static_cast<typename Out::T*>(a.dlogits) + token * a.ld_dlogits;
  if constexpr (kPer >= 8) {
#pragma unroll
    for (int c = 0; c < kPer; c += 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = d[c + j];
      const int n = E - e0 - c;
      if (n > 0) elem_store8<Out>(out + e0 + c, a.vec_out, n, v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (e0 + j < E) out[e0 + j] = Out::put(d[j]);
  }
}

// experts per lane: the smallest power of two that covers them
template <typename F>
inline cudaError_t with_per(int32_t E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace route

cudaError_t launch_route(RouteArgs a, cudaStream_t st) {
  using namespace route;
  OverlapLaunch overlap;
  a.vec = elem_vec_ok(a.logits, a.ld, a.dtype == FTMOE_OUT_FP32 ? 4 : 2);
  return with_elem(a.dtype, [&](auto elem) {
    return with_per(a.router.num_experts, [&](auto per) {
      constexpr int kPer = decltype(per)::value;
      const int size = a.router.num_experts / a.router.groups, lanes = size / kPer;
      a.group_lanes = size % kPer == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
      return launch_kernel(route_kernel<decltype(elem), kPer>, dim3((unsigned)cdiv(a.tokens, kWarps)), dim3(kThreads), 0,
                           st, true, a);
    });
  });
}

cudaError_t launch_route_backward(RouteArgs a, cudaStream_t st) {
  using namespace route;
  OverlapLaunch overlap;
  a.vec = elem_vec_ok(a.logits, a.ld, a.dtype == FTMOE_OUT_FP32 ? 4 : 2);
  a.vec_out = elem_vec_ok(a.dlogits, a.ld_dlogits, a.dlogits_dtype == FTMOE_OUT_FP32 ? 4 : 2);
  return with_elem(a.dtype, [&](auto elem) {
    return with_elem(a.dlogits_dtype, [&](auto out) {
      return with_per(a.router.num_experts, [&](auto per) {
        constexpr int kPer = decltype(per)::value;
        return launch_kernel(route_backward_kernel<decltype(elem), decltype(out), kPer>,
                             dim3((unsigned)cdiv(a.tokens, kWarps)), dim3(kThreads), kWarps * 32 * kPer * sizeof(float), st,
                             true, a);
      });
    });
  });
}

FTMOE_DEFINE_ERR_READER(read_err_route)

}  // namespace ftmoe
