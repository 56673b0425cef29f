// Work on many tensors in one launch: the list travels in the kernel's parameters, each tensor cut
// into units of kPass or kPasses * kPass elements; a block finds its unit's tensor by bisection.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace ftmoe {

namespace many {

constexpr int kThreads = 256;
constexpr int64_t kPass = 8 * kThreads;  // elements that a block takes together, 8 a thread
constexpr int kPasses = 4;               // of a large list's units

// Passes of a unit for `total` elements: long units where they fill the GPU's 152 SMs four times over, else
// one pass, for as many blocks as there can be.
inline int passes_for(int64_t total) { return total >= 152 * 4 * kPasses * kPass ? kPasses : 1; }

// kMax tensors of a launch; first[i]: units before tensor i, first[count] all of them
template <typename Entry, int kMax>
struct Table {
  int32_t count;
  int32_t first[kMax + 1];
  Entry entry[kMax];
  // tensor of a unit
  __device__ __forceinline__ int find(int unit) const {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= unit) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// The launches for a list of tensors of size(i) elements, f(from, to, tensors that are not empty, passes)
// each: `most` tensors and 2^42 elements (2^30 units) at most.
template <typename Size, typename F>
inline cudaError_t for_launches(int count, int most, Size size, F f) {
  for (int from = 0; from < count;) {
    int to = from, taken = 0;
    int64_t total = 0;
    while (to < count && taken < most) {
      const int64_t n = size(to);
      if (taken > 0 && total + n > ((int64_t)1 << 42)) break;
      total += n;
      taken += n > 0;
      ++to;
    }
    if (taken > 0) {
      const cudaError_t e = f(from, to, taken, passes_for(total));
      if (e != cudaSuccess) return e;
    }
    from = to;
  }
  return cudaSuccess;
}

}  // namespace many

}  // namespace ftmoe
