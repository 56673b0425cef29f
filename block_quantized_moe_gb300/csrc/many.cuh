// Work on many tensors in one launch: the list travels in the kernel's parameters, each tensor cut
// into units of kUnit elements; a block finds its unit's tensor by bisection.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace ftmoe {

namespace many {

constexpr int kThreads = 256;
constexpr int kPasses = 4;                      // of 8 elements a thread
constexpr int64_t kUnit = 8 * kThreads * kPasses;

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

}  // namespace many

}  // namespace ftmoe
