// Routing of tokens to experts from the router's logits, and its gradient.
//
// Forward, per token, with x its logits: s = softmax(x) or 1 / (1 + exp(-x)), value = s + bias;
// groups of consecutive experts are ranked by the sum of their 1 or 2 best values and all but the
// best groups left out; the top-k values are chosen, largest first, ties to the lower expert; the
// weights are the chosen s times the scale, renormalised to sum to it where asked.
//
// A warp per token, the next token's logits on their way meanwhile; lane l holds the experts
// [l * kPer, (l + 1) * kPer). Keys are order-preserving integers of fp32 values. Top-k: the k-th largest of
// the 32 lanes' maxima is a threshold that at least k keys reach, and, for a small k, few more do (8 of 256: 9 or
// 10 on average); they go to a lane each, in the experts' order, and a count of the larger ones is a key's
// place. That is 6 instructions a step of the threshold and 4 a candidate, against about 70 for each of k
// steps that take the largest key out of its lane's registers; the latter is kept for k > kFewTopk,
// where the candidates would pass 32 too often.
// Without a bias the logits themselves are the order and nothing is rounded. With one, the order of
// s + bias is that of 64 bits: fp32 values are off by less than half of tolerance(), so the
// threshold is lowered by that much, and where two neighbours in the order are nearer than that
// (and not the same logit and bias, a tie in any precision) the candidates' values are taken again in 64 bits.
// More candidates than lanes, and group scores nearer than that, take the whole token again (route_exact).
//
// Backward: a closed form in the saved weights (see ftmoe_route_tokens_backward), so that only plain
// softmax reads every logit. A warp per token puts the chosen experts' terms in a row of shared
// memory and writes the row of dlogits whole.
#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"

namespace ftmoe {

namespace route {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 4;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kFewTopk = 12;  // 16 of 256 would have 21 candidates on average, 20 of 256 30

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// NaN and -inf take no part (-inf); +inf counts as the largest finite number
__device__ __forceinline__ float taken(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Scores for the order alone, by the hardware's exponential and reciprocal. exp(-x) is off by the
// argument's rounding (|x| log2(e) 2^-24 ln 2 of it) and 2 units of the exponential: s by s (1 - s) of
// that, at most 0.23 * 2^-24 + 2^-24, and by 2^-23 s of the sum's rounding and the reciprocal: under 2^-21.5.
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return reciprocal(1.0f + exp2_fast(x * -kLog2e)); }

// How far apart two fp32 values have to be for their order to be that of 64 bits: s is within
// 2^-21 of the largest score (sigmoid_fast as above, the largest score taken as 1; softmax: exponentials of arguments
// rounded by |x - top| 2^-23, which times exp(x - top) is below 2^-24 of the largest, and 2 units of
// the exponential, a sum of 32 terms a lane at most and 5 levels, its reciprocal: 2^-21 of s), the sum with
// the bias within 2^-24 of itself; twice that for two values, and as much again to spare.
__device__ __forceinline__ float tolerance(float largest_score, float v) {
  return 0x1p-19f * largest_score + 0x1p-21f * fabsf(v);
}

// a lane's logits as they lie in memory
template <typename Elem, int kPer>
struct Row {
  Raw8<Elem> raw[kPer >= 8 ? kPer / 8 : 1];
  __device__ __forceinline__ void load(const typename Elem::T* row, int lane, int E, bool vec) {
    const int e0 = lane * kPer;
    if constexpr (kPer >= 8) {
#pragma unroll
      for (int c = 0; c < kPer; c += 8) raw[c / 8] = raw_load8<Elem>(row + e0 + c, vec, E - e0 - c);
    } else {
      raw[0] = raw_load8<Elem>(row + e0, false, min(E - e0, kPer));
    }
  }
  // -inf for experts that take no part, and past the last
  __device__ __forceinline__ void get(int lane, int E, float (&x)[kPer]) const {
#pragma unroll
    for (int c = 0; c < kPer; c += 8) {
      float v[8];
      raw_get8<Elem>(raw[c / 8], v);
#pragma unroll
      for (int j = c; j < kPer && j < c + 8; ++j) x[j] = taken(v[j - c]);
    }
    if (lane * kPer + kPer > E) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] = lane * kPer + j < E ? x[j] : -INFINITY;
    }
  }
};

// largest logit of the row and the sum of exp(x - max) (softmax scores)
template <int kPer>
__device__ __forceinline__ void softmax_stats(const float (&x)[kPer], float& top, float& sum) {
  float m = x[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) m = fmaxf(m, x[j]);
  top = warp_top(m);
  float s = 0.0f;
  if (top > -INFINITY) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s += exp2_fast((x[j] - top) * kLog2e);
  }
  sum = warp_sum(s);
}

// scores for the order (0 where an expert takes no part)
template <int kPer>
__device__ __forceinline__ void scores(const float (&x)[kPer], bool softmax, float top, float largest, float (&s)[kPer]) {
  if (softmax) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[j] = exp2_fast((x[j] - top) * kLog2e) * largest;
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[j] = sigmoid_fast(x[j]);
  }
}

// the two largest of two pairs
__device__ __forceinline__ void merge2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}
__device__ __forceinline__ void add2(float& a1, float& a2, float v) {
  a2 = fmaxf(a2, fminf(a1, v));
  a1 = fmaxf(a1, v);
}
__device__ __forceinline__ float group_score(float a1, float a2, int best) {
  return best == 2 && a2 > -INFINITY ? a1 + a2 : a1;
}

// The group's score on each of its lanes, where `lanes` whole lanes (a power of two) make up a group.
template <int kPer>
__device__ __forceinline__ float lane_group_scores(const float (&v)[kPer], int lane, int groups, int lanes, int best) {
  float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
  for (int j = 0; j < kPer; ++j) add2(a1, a2, v[j]);
  for (int o = 1; o < lanes; o <<= 1) merge2(a1, a2, __shfl_xor_sync(kFull, a1, o), __shfl_xor_sync(kFull, a2, o));
  return lane < groups * lanes ? group_score(a1, a2, best) : -INFINITY;
}

// Group g's score on lane g, groups of any size.
template <int kPer>
__device__ __forceinline__ float any_group_scores(const float (&v)[kPer], int lane, int groups, int size, int best) {
  float mine = -INFINITY;
  for (int g = 0; g < groups; ++g) {
    float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = lane * kPer + j - g * size;
      add2(a1, a2, at >= 0 && at < size ? v[j] : -INFINITY);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) merge2(a1, a2, __shfl_xor_sync(kFull, a1, o), __shfl_xor_sync(kFull, a2, o));
    if (lane == g) mine = group_score(a1, a2, best);
  }
  return mine;
}

// Whether this lane's group is among the `keep` best (lanes of a group next to each other, `lanes` of
// them); how far the worst of those is from the best of the others (infinite where there is none).
__device__ __forceinline__ bool keep_groups(float mine, int lane, int lanes, int keep, float& gap) {
  float last = -INFINITY;
  bool in = false;
  for (int t = 0; t < keep; ++t) {
    const float most = warp_top(mine);
    if (!(most > -INFINITY)) break;
    const int first = __ffs(__ballot_sync(kFull, mine == most)) - 1;
    last = most;
    if ((uint32_t)(lane - first) < (uint32_t)lanes) in = true, mine = -INFINITY;
  }
  const float next = warp_top(mine);
  gap = next > -INFINITY && last > -INFINITY ? last - next : INFINITY;
  return in;
}

// fp64 -> integer of the same order (-0 and +0 are one): compared without the few fp64 units
__device__ __forceinline__ int64_t key_of(double v) {
  const int64_t b = __double_as_longlong(v + 0.0);
  return b ^ (int64_t)((uint64_t)(b >> 63) >> 1);
}
__device__ __forceinline__ double value_of(int64_t key) {
  return __longlong_as_double(key ^ (int64_t)((uint64_t)(key >> 63) >> 1));
}
constexpr int64_t kNever64 = (int64_t)0x800fffffffffffffull;  // key of -inf

__device__ __forceinline__ double score64(bool softmax, double x, double top, double sum) {
  const double e = exp(softmax ? x - top : -x);
  return softmax ? e / sum : 1.0 / (1.0 + e);
}

// The choice of one token with all its values in 64 bits. Lane t gets the expert of slot t, -1 for
// none. (Any router, any number of equal values; a few microseconds.)
template <typename Elem, int kPer>
__device__ __noinline__ int route_exact(const RouteArgs& a, const typename Elem::T* row, int lane) {
  constexpr int kUnroll = kPer < 4 ? kPer : 4;
  const int E = a.router.num_experts, size = E / a.router.groups;
  const bool softmax = a.router.score == FTMOE_SCORE_SOFTMAX;
  const bool scored = a.bias != nullptr || (a.router.groups > 1 && a.router.group_best == 2);
  int64_t key[kPer];
  double sum = 1.0;
  float top = -INFINITY;
  if (softmax && scored) {
    for (int j = 0; j < kPer; ++j) top = fmaxf(top, lane * kPer + j < E ? taken(Elem::get(row[lane * kPer + j])) : -INFINITY);
    top = warp_top(top);
    sum = 0.0;
#pragma unroll(kUnroll)
    for (int j = 0; j < kPer; ++j) {
      const float x = lane * kPer + j < E ? taken(Elem::get(row[lane * kPer + j])) : -INFINITY;
      sum += x > -INFINITY ? exp((double)x - (double)top) : 0.0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
#pragma unroll(kUnroll)
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * kPer + j;
    const float x = e < E ? taken(Elem::get(row[e])) : -INFINITY;
    double v = (double)x;
    if (scored) v = score64(softmax, v, (double)top, sum) + (a.bias != nullptr && e < E ? (double)taken(a.bias[e]) : 0.0);
    key[j] = x > -INFINITY && v > -INFINITY ? key_of(v) : kNever64;
  }
  if (a.router.groups > 1) {
    int64_t mine = kNever64;
    for (int g = 0; g < a.router.groups; ++g) {
      int64_t a1 = kNever64, a2 = kNever64;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int at = lane * kPer + j - g * size;
        if (at >= 0 && at < size) {
          a2 = max(a2, min(a1, key[j]));
          a1 = max(a1, key[j]);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const int64_t b1 = __shfl_xor_sync(kFull, a1, o), b2 = __shfl_xor_sync(kFull, a2, o);
        a2 = max(min(a1, b1), max(a2, b2));
        a1 = max(a1, b1);
      }
      if (lane == g) mine = a.router.group_best == 2 && a2 > kNever64 ? key_of(value_of(a1) + value_of(a2)) : a1;
    }
    int rank = 0;
    for (int g = 0; g < a.router.groups; ++g) {
      const int64_t other = __shfl_sync(kFull, mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    const uint32_t kept = __ballot_sync(kFull, lane < a.router.groups && rank < a.router.group_topk);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = lane * kPer + j;
      if (e < E && !((kept >> (e / size)) & 1u)) key[j] = kNever64;
      else if (a.bias == nullptr && key[j] > kNever64) key[j] = key_of((double)taken(Elem::get(row[e])));  // the order is the logits'
    }
  }
  int mine = -1;
  for (int t = 0; t < a.router.topk; ++t) {
    int64_t best = kNever64;
    int at = E;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (key[j] > best) best = key[j], at = lane * kPer + j;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const int64_t other = __shfl_xor_sync(kFull, best, o);
      const int other_at = __shfl_xor_sync(kFull, at, o);
      if (other > best || (other == best && other_at < at)) best = other, at = other_at;
    }
    if (best <= kNever64) break;
    if (lane == t) mine = at;
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (lane * kPer + j == at) key[j] = kNever64;
  }
  return mine;
}

// an expert that may be among the chosen, a lane each
struct Candidate {
  float v, x, b;
  int32_t expert;
};

// Top-k of the values v by up to 32 candidates, in the order of 64 bits. Lane t gets the
// candidate of slot t (expert -1: none); false: there are more candidates.
template <typename Elem, int kPer>
__device__ __forceinline__ bool choose_few(const float (&v)[kPer], const float (&x)[kPer], const RouteArgs& a,
                                           const typename Elem::T* row, bool biased, bool softmax, float top,
                                           float largest_score, int topk, int lane, Candidate* shared, Candidate& mine) {
  // the threshold (equal maxima go together: it is then lower than it need be)
  float best = v[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) best = fmaxf(best, v[j]);
  float from = -INFINITY;
#pragma unroll 2
  for (int t = 0; t < topk; ++t) {
    from = warp_top(best);
    best = best == from ? -INFINITY : best;
  }
  if (biased) from -= tolerance(largest_score, from);
  from = fmaxf(from, -FLT_MAX);
  // places of this lane's candidates: after those of the lanes below
  int count = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) count += v[j] >= from;
  const uint32_t below = (1u << lane) - 1u;
  int at = 0, total = 0;
#pragma unroll
  for (int bit = 0; (1 << bit) <= kPer; ++bit) {
    const uint32_t lanes = __ballot_sync(kFull, (count >> bit) & 1);
    at += __popc(lanes & below) << bit;
    total += __popc(lanes) << bit;
  }
  if (total > 32) return false;
  int32_t* experts = reinterpret_cast<int32_t*>(shared + 32);
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (v[j] >= from) experts[at++] = lane * kPer + j;
  __syncwarp();
  mine = {-INFINITY, -INFINITY, 0.0f, -1};
  if (lane < total) {
    mine.expert = experts[lane];
    mine.x = taken(Elem::get(row[mine.expert]));
    mine.v = mine.x;
    if (biased) {
      mine.b = taken(__ldg(a.bias + mine.expert));
      mine.v = (softmax ? exp2_fast((mine.x - top) * kLog2e) * largest_score : sigmoid_fast(mine.x)) + mine.b;
    }
  }
  // a candidate's place: how many are larger, and where values are equal how many of those are lower experts
  int place = 0;
#pragma unroll 4
  for (int i = 0; i < total; ++i) place += __shfl_sync(kFull, mine.v, i) > mine.v;
  const uint32_t places = __reduce_or_sync(kFull, lane < total ? 1u << place : 0u);
  if (places != (uint32_t)((1ull << total) - 1ull)) {
    for (int i = 0; i < total; ++i) place += __shfl_sync(kFull, mine.v, i) == mine.v && i < lane;
  }
  if (lane < total) shared[place] = mine;
  __syncwarp();
  if (lane < total) mine = shared[lane];
  if (biased) {
    const float next = __shfl_down_sync(kFull, mine.v, 1);
    bool near = lane < topk && lane + 1 < total && mine.v - next <= tolerance(largest_score, mine.v);
    if (__any_sync(kFull, near)) {
      const float next_x = __shfl_down_sync(kFull, mine.x, 1), next_b = __shfl_down_sync(kFull, mine.b, 1);
      near = near && (next_x != mine.x || next_b != mine.b);
      if (__any_sync(kFull, near)) {
        double sum = 1.0;
        if (softmax) {
          sum = 0.0;
#pragma unroll 1
          for (int j = 0; j < kPer; ++j) sum += x[j] > -INFINITY ? exp((double)x[j] - (double)top) : 0.0;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        }
        const int64_t key = key_of(score64(softmax, (double)mine.x, (double)top, sum) + (double)mine.b);
        place = 0;
        for (int i = 0; i < total; ++i) {
          const int64_t other = __shfl_sync(kFull, key, i);
          const int expert = __shfl_sync(kFull, mine.expert, i);
          place += other > key || (other == key && expert < mine.expert);
        }
        __syncwarp();
        if (lane < total) shared[place] = mine;
        __syncwarp();
        if (lane < total) mine = shared[lane];
      }
    }
  }
  if (lane >= topk) mine.expert = -1;
  return true;
}

// Top-k a step at a time; `near` where two neighbours in the order have to be taken in 64 bits.
template <int kPer>
__device__ __forceinline__ int choose_many(float (&v)[kPer], bool biased, float largest_score, int topk, int lane, bool& near) {
  int chosen = -1;
  float slot = -INFINITY, best = v[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) best = fmaxf(best, v[j]);
  for (int t = 0; t < topk; ++t) {
    const float most = warp_top(best);
    if (!(most > -INFINITY)) break;
    const int owner = __ffs(__ballot_sync(kFull, best == most)) - 1;
    int at = 0;
    if (lane == owner) {
#pragma unroll
      for (int j = kPer - 1; j >= 0; --j) at = v[j] == most ? j : at;
      best = -INFINITY;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        v[j] = j == at ? -INFINITY : v[j];
        best = fmaxf(best, v[j]);
      }
    }
    at = __shfl_sync(kFull, at, owner);
    if (lane == t) chosen = owner * kPer + at, slot = most;
  }
  near = false;
  if (biased) {
    // pairs of neighbours in the order, and the last chosen against the best of the rest (whatever it is)
    const int next = __shfl_down_sync(kFull, chosen, 1);
    const float next_value = __shfl_down_sync(kFull, slot, 1), last = __shfl_sync(kFull, slot, topk - 1);
    bool close = lane + 1 < topk && next >= 0 && slot - next_value <= tolerance(largest_score, slot);
    if (last > -INFINITY) close = close || (best > -INFINITY && last - best <= tolerance(largest_score, last));
    near = __any_sync(kFull, close);
  }
  return chosen;
}

// A block takes consecutive tokens; its warps take them one by one, so that a token that has to be
// taken in 64 bits holds up none of the others.
template <typename Elem, int kPer, bool kFew>
__global__ void __launch_bounds__(kThreads, kPer <= 8 ? kBlocksPerSm : 2) route_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ Candidate candidates[kWarps][32 + 8];  // (the last 8: 32 experts)
  __shared__ int taken_tokens;
  if (threadIdx.x == 0) taken_tokens = kWarps;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  using T = typename Elem::T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.router.num_experts, topk = a.router.topk;
  const bool softmax = a.router.score == FTMOE_SCORE_SOFTMAX, biased = a.bias != nullptr;
  const bool scored_groups = a.router.groups > 1 && (biased || a.router.group_best == 2);
  int64_t active_tokens = a.tokens;
  if (a.tokens_dev != nullptr) {
    const int64_t n = *a.tokens_dev;
    active_tokens = n < 0 ? 0 : n < active_tokens ? n : active_tokens;
  }
  const int64_t first = a.tokens * blockIdx.x / gridDim.x;
  const int tokens = (int)(a.tokens * (blockIdx.x + 1) / gridDim.x - first);
  const int active = (int)(active_tokens <= first ? 0 : active_tokens - first < tokens ? active_tokens - first : tokens);
  const T* const rows = static_cast<const T*>(a.logits) + first * a.ld;
  float bias[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) bias[j] = biased && lane * kPer + j < E ? taken(a.bias[lane * kPer + j]) : 0.0f;

  int token = warp;
  Row<Elem, kPer> next;
  if (token < active) next.load(rows + token * a.ld, lane, E, a.vec);
  while (token < tokens) {
    int after = 0;
    if (lane == 0) after = atomicAdd(&taken_tokens, 1);
    after = __shfl_sync(kFull, after, 0);
    int chosen = -1;    // lane t: expert of slot t
    float weight = 0.0f;
    if (token < active) {
      const T* const row = rows + token * a.ld;
      float x[kPer];
      next.get(lane, E, x);
      if (after < active) next.load(rows + after * a.ld, lane, E, a.vec);

      float top = 0.0f, sum = 1.0f;
      if (softmax && (biased || scored_groups || !a.router.renormalize)) softmax_stats(x, top, sum);
      const float largest_score = softmax ? 1.0f / sum : 1.0f;
      float v[kPer];       // the order of the experts (-inf: never chosen)
      bool exact = false;  // the token has to be taken in 64 bits
      if (biased || scored_groups) {
        scores(x, softmax, top, largest_score, v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = x[j] > -INFINITY ? v[j] + bias[j] : -INFINITY;
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = x[j];
      }
      if (a.router.groups > 1) {
        float gap, mine;
        uint32_t kept;  // bit j: expert j of the lane may be chosen
        if (a.group_lanes > 0) {
          mine = lane_group_scores(v, lane, a.router.groups, a.group_lanes, a.router.group_best);
          kept = keep_groups(mine, lane, a.group_lanes, a.router.group_topk, gap) ? 0xffffffffu : 0u;
        } else {
          const int size = E / a.router.groups;
          mine = any_group_scores(v, lane, a.router.groups, size, a.router.group_best);
          const uint32_t groups = __ballot_sync(kFull, keep_groups(mine, lane, 1, a.router.group_topk, gap));
          kept = 0u;
          int group = lane * kPer / size, rest = lane * kPer - group * size;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            kept |= (group < 32 ? (groups >> group) & 1u : 0u) << j;
            if (++rest == size) rest = 0, ++group;
          }
        }
        if (scored_groups) {
          const float most = warp_top(mine > -INFINITY ? fabsf(mine) : 0.0f);
          exact = gap <= 2.0f * tolerance(largest_score, most);
          if (!biased) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = x[j];
          }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = (kept >> j) & 1u ? v[j] : -INFINITY;
      }
      float cx = -INFINITY;  // the chosen's logit
      if constexpr (kFew) {
        Candidate c;
        if (!exact) {
          exact = !choose_few<Elem, kPer>(v, x, a, row, biased, softmax, top, largest_score, topk, lane, candidates[warp], c);
          chosen = c.expert;
          cx = c.x;
        }
      } else {
        bool near;
        chosen = choose_many(v, biased, largest_score, topk, lane, near);
        exact = exact || near;
        if (chosen >= 0) cx = taken(Elem::get(row[chosen]));
      }
      if (exact) {
        chosen = route_exact<Elem, kPer>(a, row, lane);
        cx = chosen >= 0 ? taken(Elem::get(row[chosen])) : -INFINITY;
      }
      if (chosen < 0) cx = -INFINITY;

      if (a.router.renormalize) {
        // shares of the chosen scores, scaled so that the largest does not underflow:
        // softmax exp(x - most), sigmoid exp(-t) s with t = min(most, 0)
        const float most = warp_top(cx), t = fminf(most, 0.0f);
        float u = 0.0f;
        if (chosen >= 0) u = softmax ? exp2_fast((cx - most) * kLog2e) : reciprocal(exp2_fast(t * kLog2e) + exp2_fast((t - cx) * kLog2e));
        weight = u;
        for (int o = 1; o < topk; o <<= 1) u += __shfl_xor_sync(kFull, u, o);
        weight = chosen >= 0 ? weight * (a.router.scale / u) : 0.0f;
      } else if (chosen >= 0) {
        weight = a.router.scale * (softmax ? exp2_fast((cx - top) * kLog2e) * largest_score : sigmoid(cx));
      }
    }
    if (lane < topk) {
      const int64_t at = (first + token) * topk + lane;
      a.ids_out[at] = chosen;
      a.weights_out[at] = weight;
    }
    token = after;
  }
}

// what a lane reads of a token's routes: its slot
struct Slot {
  int id;
  float w, dw;
  __device__ __forceinline__ void load(const RouteArgs& a, int64_t token, int lane, int topk) {
    id = -1;
    w = dw = 0.0f;
    if (lane < topk) {
      const int64_t at = token * topk + lane;
      id = a.ids[at];
      w = a.weights[at];
      dw = a.dweights[at];
    }
  }
};

template <typename Elem, typename Out, int kPer>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const __grid_constant__ RouteArgs a) {
  extern __shared__ float4 rows[];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int E = a.router.num_experts, topk = a.router.topk, e0 = lane * kPer;
  float* const part = reinterpret_cast<float*>(rows) + (threadIdx.x >> 5) * (32 * kPer);
  const bool softmax = a.router.score == FTMOE_SCORE_SOFTMAX, whole = softmax && !a.router.renormalize;
  const float per_scale = 1.0f / a.router.scale;
  const int64_t stride = (int64_t)gridDim.x * kWarps;
  int64_t token = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  Row<Elem, kPer> next_row;
  Slot next;
  if (token < a.tokens) {
    next.load(a, token, lane, topk);
    if (whole) next_row.load(static_cast<const typename Elem::T*>(a.logits) + token * a.ld, lane, E, a.vec);
  }
  for (; token < a.tokens; token += stride) {
    const typename Elem::T* row = static_cast<const typename Elem::T*>(a.logits) + token * a.ld;
    Slot s = next;
    const Row<Elem, kPer> this_row = next_row;
    if (token + stride < a.tokens) {
      next.load(a, token + stride, lane, topk);
      if (whole) next_row.load(row + stride * a.ld, lane, E, a.vec);
    }
    if (s.id >= E) raise_error(FTMOE_ERR_EXPERT_ID_RANGE);
    if (s.id < 0 || s.id >= E) s.id = -1, s.w = 0.0f, s.dw = 0.0f;
    float r = s.w * s.dw;
    const float total = warp_sum(r);
    if (a.router.renormalize) r = fmaf(-s.w, total * per_scale, r);
    if (!softmax && s.id >= 0) r *= 1.0f / (1.0f + expf(taken(Elem::get(row[s.id]))));
    // an id that occurs twice: the first of its lanes gets the sum
    const uint32_t same = __match_any_sync(kFull, s.id);
    if (__any_sync(kFull, s.id >= 0 && (same & (same - 1u)) != 0u)) {
      float all = 0.0f;
      for (int t = 0; t < topk; ++t) {
        const float other = __shfl_sync(kFull, r, t);
        all += (same >> t) & 1u ? other : 0.0f;
      }
      r = all;
    }
    const bool lead = s.id >= 0 && (same & ((1u << lane) - 1u)) == 0u;

    float d[kPer];
    if constexpr (kPer >= 4) {
#pragma unroll
      for (int j = 0; j < kPer; j += 4) *reinterpret_cast<float4*>(part + e0 + j) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) part[e0 + j] = 0.0f;
    }
    __syncwarp();
    if (lead) part[s.id] = r;
    __syncwarp();
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
    if (whole && __any_sync(kFull, s.id >= 0)) {
      float x[kPer], top = -INFINITY, sum = 0.0f;
      this_row.get(lane, E, x);
#pragma unroll
      for (int j = 0; j < kPer; ++j) top = fmaxf(top, x[j]);
      top = warp_top(top);
      if (top > -INFINITY) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += x[j] = exp2_fast((x[j] - top) * kLog2e);
        const float f = total / warp_sum(sum);
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
        const int n = E - e0 - c;
        if (n > 0) elem_store8<Out>(out + e0 + c, a.vec_out, n, v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (e0 + j < E) out[e0 + j] = Out::put(d[j]);
    }
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
      // one token a block where there are few, else as many blocks as fit at once, of equal shares
      const unsigned blocks = (unsigned)std::min<int64_t>(a.tokens, 152 * kBlocksPerSm);
      return launch_kernel(a.router.topk <= kFewTopk ? route_kernel<decltype(elem), kPer, true> : route_kernel<decltype(elem), kPer, false>,
                           dim3(blocks), dim3(kThreads), 0, st, true, a);
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
                             dim3((unsigned)std::min<int64_t>(cdiv(a.tokens, kWarps), 152 * kBlocksPerSm)), dim3(kThreads),
                             kWarps * 32 * kPer * sizeof(float), st, true, a);
      });
    });
  });
}

FTMOE_DEFINE_ERR_READER(read_err_route)

}  // namespace ftmoe
