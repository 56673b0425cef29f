// Routing of tokens to experts from the router's logits.
//
// Per token, with x its logits: s = softmax(x) or 1 / (1 + exp(-x)), value = s + bias;
// groups of consecutive experts are ranked by the sum of their 1 or 2 best values and all but the
// best groups left out; the top-k values are chosen, largest first, ties to the lower expert; the
// weights are the chosen s times the scale, renormalised to sum to it where asked.
//
// A warp per token, the next token's logits on their way meanwhile; lane l holds the experts
// [l * kPer, (l + 1) * kPer). Top-k (choose_top): each lane keeps its three best values, and each of the
// k steps takes the largest of the lanes' best. Where a lane gives all three (3% of tokens for 8 of 256
// normal logits, 6 to 10% where half of the groups are left; four values a lane cost every token as much
// as that) or values are too near (below), choose_few takes over: the k-th largest of the lanes' maxima is
// a threshold that at least k values reach and few more do; they go to a lane each and are ranked by a
// count. (Where fewer than k lanes are left, or lanes have equal maxima, the threshold falls, at worst to
// the lowest number.) A choice of more than kFewTopk, which would have too many for both, takes the
// largest out of its lane's registers step by step (choose_many).
// Without a bias the logits themselves are the order and nothing is rounded. With one, the order of
// s + bias is that of 64 bits: fp32 values are off by less than half of tolerance(), and where two
// neighbours in the order are nearer than that (and not the same logit and bias, a tie in any
// precision) the candidates' values are taken again in 64 bits, a lane each; groups at the border
// likewise (settle_groups), where the sizes of their values (not of their sums) leave it open. More
// candidates than lanes take the whole token again (route_exact).
//
// Measured on GB300, a call among others: 32,768 tokens of 256 experts, top-8 of 4 of 8 groups, sigmoid
// and bias 28 us; without bias and groups 17.5 us (k = 1: 12 us), where the logits are 33.5 MB, 5 us of
// memory. Instructions bound it (683 and 440 a token, issued in 72% of the cycles), most of them on the
// half-rate ALU pipe; a step is about 15 (steps that rescan the owner's registers took 70 each, 94 us
// in all; the threshold for every token 42 us). One token, or eight: 2 to 3 us, launch and latency.
// Slow are the routers and rows that go to 64 bits whole (32,768 tokens, sigmoid, bias): kept groups of
// fewer lanes than k that hold more than 32 experts (512 experts, 2 of 8 groups, top-10: 71% of tokens,
// 0.91 ms; all groups 40 us; 1,024, 1 of 8, top-12: every token, 2.3 ms), rows of more than 32 equal logits
// under one bias, or with k above kFewTopk of any equal ones (256 experts, top-16, bf16: 0.40 ms; without
// a bias 54 us).
#pragma once

#include "route.cuh"

namespace ftmoe {

namespace route {

constexpr int kThreads = 512, kWarps = kThreads / 32;  // at most: see launch_as
constexpr int kBlocksPerSm = 2;                        // (four of 256 threads are 2 to 5% slower)
constexpr int kFewTopk = 12;  // 16 of 256 would have 21 candidates on average, 20 of 256 30

// How far apart two fp32 values have to be for their order to be that of 64 bits: scores are off by
// at most 2^-21.5 (sigmoid_fast), or 45 * 2^-24 = 2^-18.5 of the largest (softmax: arguments rounded by
// |x - top| 2^-23, which times exp(x - top) is below 2^-24 of the largest; 4 half steps of the
// exponential; 37 of a sum of 32 terms a lane and 5 levels; 3 of its reciprocal and the product),
// and sums with the bias by 2^-24 of themselves; twice that for two values, and some to spare.
// unit: see score_unit.
__device__ __forceinline__ float tolerance(float unit, float v) { return 0x1p-19f * unit + 0x1p-21f * fabsf(v); }
__device__ __forceinline__ float score_unit(bool softmax, float largest_score) { return softmax ? 4.0f * largest_score : 1.0f; }

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

__device__ __forceinline__ float score_fast(float x, bool softmax, float top, float largest) {
  return softmax ? exp2_fast((x - top) * kLog2e) * largest : sigmoid_fast(x);
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
// (a sum is at least the lowest number: -inf is the score of a group of which nothing can be chosen)
__device__ __forceinline__ float group_score(float a1, float a2, int best) {
  return best == 2 && a2 > -INFINITY ? fmaxf(a1 + a2, -FLT_MAX) : a1;
}

// How far a group's score may be from its score in 64 bits: its values are off by half of tolerance() each, by
// their own sizes and not by their sum's (which biases of both signs leave small), and the sum by a rounding.
__device__ __forceinline__ float group_slack(float unit, float a1, float a2, int best) {
  const float size = best == 2 && a2 > -INFINITY ? fmaxf(fabsf(a1), fabsf(a2)) : fabsf(a1);
  return a1 > -INFINITY ? tolerance(unit, size) : 0.0f;
}

// Group g's two best values on lane g, groups of any size.
template <int kPer>
__device__ __forceinline__ void any_groups_best(const float (&v)[kPer], int lane, int groups, int size, float& g1, float& g2) {
  g1 = g2 = -INFINITY;
  for (int g = 0; g < groups; ++g) {
    float a1 = -INFINITY, a2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int at = lane * kPer + j - g * size;
      add2(a1, a2, at >= 0 && at < size ? v[j] : -INFINITY);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) merge2(a1, a2, __shfl_xor_sync(kFull, a1, o), __shfl_xor_sync(kFull, a2, o));
    if (lane == g) g1 = a1, g2 = a2;
  }
}

// Whether this lane's group is among the `keep` best (lanes of a group next to each other, `lanes` of them).
__device__ __forceinline__ bool keep_groups(float mine, int lane, int lanes, int keep) {
  bool in = false;
  const uint32_t below = (1u << (lane & ~(lanes - 1))) - 1u;  // the lanes of lower groups
  for (int t = 0; t < keep; ++t) {
    const float most = warp_top(mine);  // (-inf: groups of no expert that could be chosen)
    const uint32_t all = __ballot_sync(kFull, mine == most);  // (by every lane, so not behind a condition)
    const bool is = mine == most && (all & below) == 0u;
    in = in || is;
    mine = is ? -INFINITY : mine;
  }
  return in;
}

// The border between the groups kept and the others: the least that the score of a kept one may be in 64 bits, and
// the most that one of the others may be (-inf where there is none).
struct Border {
  float low, high;
  __device__ __forceinline__ Border(float mine, float slack, bool kept) {
    low = -warp_top(kept ? slack - mine : -INFINITY);
    high = warp_top(kept ? -INFINITY : mine + slack);
  }
  __device__ __forceinline__ bool unsure() const { return high > -INFINITY && low <= high; }
};

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

// the three largest of a lane's values (of a lane of fewer, -inf for the others)
struct Best3 {
  float a, b, c;
};
template <int kPer>
__device__ __forceinline__ Best3 best3(const float (&v)[kPer]) {
  Best3 t = {v[0], -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 1; j < kPer; ++j) {
    if (j > 1) t.c = fmaxf(t.c, fminf(t.b, v[j]));
    t.b = fmaxf(t.b, fminf(t.a, v[j]));
    t.a = fmaxf(t.a, v[j]);
  }
  return t;
}

// Top-k from the lanes' three best values: each step takes the largest of the lanes' best, and its lane's
// next moves up. Lane t gets the expert of slot t (-1: none) and its value; rest: the best value left.
// false: a lane gave three, and what it has left is not known (3% of tokens for 8 of 256 experts), or
// two that are equal, or there are not enough (-inf comes from the lowest lane again and again).
// (A step is a maximum and a vote over the warp, 24 cycles each; selects rather than branches, and
// no first-set-bit, which runs at a quarter of the vote's rate. The experts' places in their lanes are
// found at the end, for all slots at once, by an exchange for each of a lane's values.)
template <int kPer>
__device__ __forceinline__ bool choose_top(const float (&v)[kPer], Best3 t, int topk, int lane, int& expert, float& value, float& rest) {
  const uint32_t below = (1u << lane) - 1u;
  const bool twins = t.a == t.b;
  uint32_t givers = 0u;  // lane t: those whose best was the largest at slot t (the lowest gave it)
  int given = 0;         // values that this lane gave
  value = -INFINITY;
#pragma unroll 4
  for (int n = 0; n < topk; ++n) {
    const float most = warp_top(t.a);
    const bool is = t.a == most;
    const uint32_t alike = __ballot_sync(kFull, is);  // (by every lane, so not behind a condition)
    const bool first = is && (alike & below) == 0u;
    givers = lane == n ? alike : givers;
    value = lane == n ? most : value;
    given += first ? 1 : 0;
    t.a = first ? t.b : t.a;
    t.b = first ? t.c : t.b;  // (what follows the third value is never used: see below)
  }
  if (__any_sync(kFull, given > 2 || (given == 2 && twins))) return false;
  rest = warp_top(t.a);
  const int giver = __ffs(givers) - 1;
  int at = 0;
#pragma unroll
  for (int j = kPer - 1; j >= 0; --j) at = __shfl_sync(kFull, v[j], giver) == value ? j : at;
  expert = value > -INFINITY ? giver * kPer + at : -1;
  return true;
}

// an expert that may be among the chosen, a lane each
struct Candidate {
  float v, x, b;
  int32_t expert;
};

// Writes this lane's candidates, the elements j with bit j of `mask`, behind those of the lanes below; how many
// there are in all (nothing is written where there are more than 32).
__device__ __forceinline__ int gather_candidates(uint32_t mask, int lane, int first, int32_t* experts) {
  const int count = __popc(mask);
  const uint32_t below = (1u << lane) - 1u;
  int at = 0, total = 0;
#pragma unroll
  for (int bit = 0; bit < 6; ++bit) {
    const uint32_t lanes = __ballot_sync(kFull, (count >> bit) & 1);
    at += __popc(lanes & below) << bit;
    total += __popc(lanes) << bit;
  }
  __syncwarp();  // (the last ones have been read)
  if (total <= 32) {
    for (; mask != 0u; mask &= mask - 1u) experts[at++] = first + __ffs(mask) - 1;
  }
  __syncwarp();
  return total;
}

template <int kPer>
__device__ __forceinline__ double softmax_sum64(const float (&x)[kPer], float top) {
  double sum = 0.0;
#pragma unroll 1
  for (int j = 0; j < kPer; ++j) sum += x[j] > -INFINITY ? exp((double)x[j] - (double)top) : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  return sum;
}

// The groups to keep where the border is unsure: a kept group that may be below one of the others and another that may
// be above a kept one are compared by their best values in 64 bits, taken of every expert that may be
// one of them. kept: whether this lane's group is, in fp32 and then in 64 bits. false: they are more than 32.
template <typename Elem, int kPer>
__device__ __forceinline__ bool settle_groups(const float (&v)[kPer], const float (&x)[kPer], const RouteArgs& a,
                                              const typename Elem::T* row, bool softmax, float unit, float top, float g1,
                                              float g2, float mine, float slack, Border border, int lane, int32_t* experts,
                                              bool& kept) {
  const int lanes = a.group_lanes, groups = a.router.groups, best = a.router.group_best;
  const bool open = kept ? mine - slack <= border.high : mine > -INFINITY && mine + slack >= border.low;
  // (the values that make up the score; without a bias they are logits, and the order is theirs)
  const float least = best == 2 && g2 > -INFINITY ? g2 : g1;
  const float from = a.bias != nullptr ? least - tolerance(unit, least) : least;
  uint32_t mask = 0u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) mask |= (open && v[j] > -INFINITY && v[j] >= from ? 1u : 0u) << j;
  const int total = gather_candidates(mask, lane, lane * kPer, experts);
  if (total > 32) return false;
  const double sum = softmax ? softmax_sum64(x, top) : 1.0;
  int64_t key = kNever64;
  int group = -1;
  if (lane < total) {
    const int e = experts[lane];
    key = key_of(score64(softmax, (double)taken(Elem::get(row[e])), (double)top, sum) + (a.bias != nullptr ? (double)taken(a.bias[e]) : 0.0));
    group = e / (lanes * kPer);
  }
  int64_t a1 = kNever64, a2 = kNever64;
  for (int i = 0; i < total; ++i) {
    const int64_t other = __shfl_sync(kFull, key, i);
    const int of = __shfl_sync(kFull, group, i);
    if (of == lane / lanes) {
      a2 = max(a2, min(a1, other));
      a1 = max(a1, other);
    }
  }
  int64_t score = best == 2 && a2 > kNever64 ? key_of(value_of(a1) + value_of(a2)) : a1;
  if (!open) score = kept ? INT64_MAX : kNever64;
  int rank = 0;
  for (int g = 0; g < groups; ++g) {
    const int64_t other = __shfl_sync(kFull, score, g * lanes);
    rank += other > score || (other == score && g < lane / lanes);
  }
  kept = rank < a.router.group_topk;
  return true;
}

// Top-k of the values v by up to 32 candidates, in the order of 64 bits. Lane t gets the
// candidate of slot t (expert -1: none); false: there are more candidates.
template <typename Elem, int kPer>
__device__ __forceinline__ bool choose_few(const float (&v)[kPer], const float (&x)[kPer], const RouteArgs& a,
                                           const typename Elem::T* row, bool biased, bool softmax, float top,
                                           float largest_score, int topk, int lane, Candidate* shared, Candidate& mine) {
  const float unit = score_unit(softmax, largest_score);
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
  if (biased) from -= tolerance(unit, from);
  from = fmaxf(from, -FLT_MAX);
  uint32_t mask = 0u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) mask |= (v[j] >= from ? 1u : 0u) << j;
  int32_t* experts = reinterpret_cast<int32_t*>(shared + 32);
  const int total = gather_candidates(mask, lane, lane * kPer, experts);
  if (total > 32) return false;
  mine = {-INFINITY, -INFINITY, 0.0f, -1};
  if (lane < total) {
    mine.expert = experts[lane];
    mine.x = taken(Elem::get(row[mine.expert]));
    mine.v = mine.x;
    if (biased) {
      mine.b = taken(a.bias[mine.expert]);
      mine.v = score_fast(mine.x, softmax, top, largest_score) + mine.b;
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
    // (pairs beyond the last slot too: one that is not the same may follow several that are)
    bool near = lane + 1 < total && mine.v - next <= tolerance(unit, mine.v);
    if (__any_sync(kFull, near)) {
      const float next_x = __shfl_down_sync(kFull, mine.x, 1), next_b = __shfl_down_sync(kFull, mine.b, 1);
      near = near && (next_x != mine.x || next_b != mine.b);
      if (__any_sync(kFull, near)) {
        const double sum = softmax ? softmax_sum64(x, top) : 1.0;
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
__device__ __forceinline__ int choose_many(float (&v)[kPer], bool biased, float unit, int topk, int lane, bool& near) {
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
    bool close = lane + 1 < topk && next >= 0 && slot - next_value <= tolerance(unit, slot);
    if (last > -INFINITY) close = close || (best > -INFINITY && last - best <= tolerance(unit, last));
    near = __any_sync(kFull, close);
  }
  return chosen;
}

// A block takes consecutive tokens; its warps take them one by one, so that a token that has to be
// taken in 64 bits holds up none of the others.
template <typename Elem, int kPer, bool kFew, bool kBiased>
__global__ void __launch_bounds__(kThreads, kPer <= 8 ? kBlocksPerSm : 1) route_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ Candidate candidates[kWarps][32 + 8];  // (the last 8: 32 experts)
  __shared__ int taken_tokens;
  if (threadIdx.x == 0) taken_tokens = (int)blockDim.x >> 5;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  using T = typename Elem::T;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.router.num_experts, topk = a.router.topk;
  const bool softmax = a.router.score == FTMOE_SCORE_SOFTMAX, biased = kFew ? kBiased : a.bias != nullptr;
  const bool grouped = a.router.groups > 1, lane_groups = a.group_lanes > 0;
  const bool scored_groups = grouped && (biased || a.router.group_best == 2);
  const bool all_scores = softmax && (biased || scored_groups || !a.router.renormalize);
  int64_t active_tokens = a.tokens;
  if (a.tokens_dev != nullptr) {
    const int64_t n = *a.tokens_dev;
    active_tokens = n < 0 ? 0 : n < active_tokens ? n : active_tokens;
  }
  const int64_t first = a.tokens * blockIdx.x / gridDim.x;
  const int tokens = (int)(a.tokens * (blockIdx.x + 1) / gridDim.x - first);
  const int active = (int)(active_tokens <= first ? 0 : active_tokens - first < tokens ? active_tokens - first : tokens);
  const T* const rows = static_cast<const T*>(a.logits) + first * a.ld;
  int32_t* const ids_out = a.ids_out + first * topk + lane;
  float* const weights_out = a.weights_out + first * topk + lane;
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
      next.get_taken(x);
      if (after < active) next.load(rows + after * a.ld, lane, E, a.vec);

      float top = 0.0f, sum = 1.0f;
      if (all_scores) softmax_stats(x, top, sum);
      const float largest_score = softmax ? reciprocal(sum) : 1.0f, unit = score_unit(softmax, largest_score);
      float v[kPer];  // the order of the experts (-inf: never chosen)
      if (biased) {
        scores(x, softmax, top, largest_score, v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = x[j] > -INFINITY ? v[j] + bias[j] : -INFINITY;
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = x[j];
      }
      bool exact = false;    // the token has to be taken in 64 bits
      bool kept = true;      // this lane's experts may be chosen
      Best3 best;
      if (!grouped) {
        if constexpr (kFew) best = best3(v);
      } else if (lane_groups) {
        best = best3(v);
        float g1 = best.a, g2 = best.b;
        for (int o = 1; o < a.group_lanes; o <<= 1) merge2(g1, g2, __shfl_xor_sync(kFull, g1, o), __shfl_xor_sync(kFull, g2, o));
        const bool inside = lane < a.router.groups * a.group_lanes;
        float h1 = g1, h2 = g2;
        if (!biased && scored_groups) {  // (scores grow with the logits)
          h1 = g1 > -INFINITY ? score_fast(g1, softmax, top, largest_score) : -INFINITY;
          h2 = g2 > -INFINITY ? score_fast(g2, softmax, top, largest_score) : -INFINITY;
        }
        const float mine = inside ? group_score(h1, h2, a.router.group_best) : -INFINITY;
        kept = keep_groups(mine, lane, a.group_lanes, a.router.group_topk);
        if (scored_groups) {
          const float slack = inside ? group_slack(unit, h1, h2, a.router.group_best) : 0.0f;
          const Border border(mine, slack, kept);
          if (border.unsure())
            exact = !settle_groups<Elem, kPer>(v, x, a, row, softmax, unit, top, g1, g2, mine, slack, border, lane,
                                               reinterpret_cast<int32_t*>(candidates[warp] + 32), kept);
        }
        if (!kept) best = {-INFINITY, -INFINITY, -INFINITY};
      } else {
        const int size = E / a.router.groups;
        float s[kPer], g1, g2;
        if (!biased && scored_groups) scores(x, softmax, top, largest_score, s);
#pragma unroll
        for (int j = 0; j < kPer; ++j) s[j] = !biased && scored_groups && x[j] > -INFINITY ? s[j] : v[j];
        any_groups_best(s, lane, a.router.groups, size, g1, g2);
        const float mine = group_score(g1, g2, a.router.group_best);
        const bool in = keep_groups(mine, lane, 1, a.router.group_topk);
        const uint32_t groups = __ballot_sync(kFull, in);
        exact = scored_groups && Border(mine, group_slack(unit, g1, g2, a.router.group_best), in).unsure();
        int group = lane * kPer / size, rest = lane * kPer - group * size;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          v[j] = group < 32 && (groups >> group) & 1u ? v[j] : -INFINITY;
          if (++rest == size) rest = 0, ++group;
        }
        best = best3(v);
      }
      float cx = -INFINITY;  // the chosen's logit
      if constexpr (kFew) {
        if (!exact) {
          float rest;
          float value;
          bool fine = choose_top(v, best, topk, lane, chosen, value, rest);
          if (fine) {
            cx = value;
            if (biased) {
              // (a neighbour as near as that, the best of the rest after the last)
              const float below = __shfl_down_sync(kFull, value, 1);
              if (chosen >= 0) cx = taken(Elem::get(row[chosen]));
              fine = !__any_sync(kFull, chosen >= 0 && value - (lane + 1 < topk ? below : rest) <= tolerance(unit, value));
            }
          }
          if (!fine) {
            Candidate c;
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] = kept ? v[j] : -INFINITY;
            exact = !choose_few<Elem, kPer>(v, x, a, row, biased, softmax, top, largest_score, topk, lane, candidates[warp], c);
            chosen = c.expert;
            cx = c.x;
          }
        }
      } else {
        bool near;
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = kept ? v[j] : -INFINITY;
        chosen = choose_many(v, biased, unit, topk, lane, near);
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
        weight = chosen >= 0 ? weight * (a.router.scale * reciprocal(u)) : 0.0f;
      } else if (chosen >= 0) {
        weight = a.router.scale * (softmax ? exp2_fast((cx - top) * kLog2e) * largest_score : sigmoid(cx));
      }
    }
    if (lane < topk) {
      ids_out[token * topk] = chosen;
      weights_out[token * topk] = weight;
    }
    token = after;
  }
}

template <typename Elem>
cudaError_t launch_as(RouteArgs a, cudaStream_t st) {
  OverlapLaunch overlap;
  return with_per(a.router.num_experts, [&](auto per) {
    constexpr int kPer = decltype(per)::value;
    const int size = a.router.num_experts / a.router.groups, lanes = size / kPer;
    a.group_lanes = size % kPer == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    a.vec = Row<Elem, kPer>::vec_ok(a.logits, a.ld, a.router.num_experts);
    auto* kernel = a.router.topk > kFewTopk ? route_kernel<Elem, kPer, false, false>
                   : a.bias != nullptr ? route_kernel<Elem, kPer, true, true> : route_kernel<Elem, kPer, true, false>;
    // as many blocks as fit at once, of equal shares, and a warp for each of their tokens where there are few
    const int64_t blocks = std::min<int64_t>(a.tokens, 152 * kBlocksPerSm), most = cdiv(a.tokens, blocks);
    return launch_kernel(kernel, dim3((unsigned)blocks), dim3(32 * (unsigned)std::min<int64_t>(most, kWarps)), 0, st, true, a);
  });
}

}  // namespace route

}  // namespace ftmoe
