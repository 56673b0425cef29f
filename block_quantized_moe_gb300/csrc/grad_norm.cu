// Global norm of many gradients, and the factor that scales and clips them.
//
// Every gradient is read once (memory bounds it) in units of 8,192 elements that the blocks of a
// grid take in turn; a second launch adds the blocks' sums in order. A thread squares and sums the eight
// elements that it reads together in fp32; those sums are added as pairs of fp32 numbers, whose errors are
// carried along (two-sum: D. E. Knuth, The Art of Computer Programming, vol. 2, 4.2.2), and a block's
// pair becomes one fp64 number. (fp64 sums throughout would hold the GPU's few fp64 units for a third of the time:
// an addition by 1,024 threads takes 0.3 us.) Sums of eight that are large or small for fp32 (an
// element beyond 2^38, gradients so small that their squares would be subnormal, NaN) are taken in fp64.
// (One launch for small lists, a cluster of eight blocks whose sums meet in shared memory, was no faster:
// 4.4 us for 1,000 elements and 7.1 for 262,144, where the two launches take 4.1.)
// Measured on GB300: 939 M bf16 elements 268 us, 103% of the measured copy rate; 268 M fp32 ones 154 us, 103%.
#include <algorithm>

#include "common.cuh"
#include "elem16.cuh"
#include "many.cuh"

namespace ftmoe {

namespace grad_norm {

using many::kPasses;
using many::kThreads;
using many::kPass;

struct Entry {
  int64_t n;
  const void* grad;
  int32_t vec;
};

constexpr int kFew = 64, kMany = 1024;  // gradients of a launch
// Blocks of a launch, one part each: as many as are resident (a block more a SM runs in a second wave: 939 M bf16
// elements 314 us instead of 269).
constexpr int kGrid = 152 * 6;  // at most
template <typename G>
constexpr int grid_of() {
  return 152 * (sizeof(typename G::T) == 4 ? 5 : 6);
}

// a sum and what its roundings left out
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float s = hi + v, of_v = s - hi;
    lo += (hi - (s - of_v)) + (v - of_v);
    hi = s;
  }
  __device__ __forceinline__ void add_of_warp() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, hi, o), rest = __shfl_xor_sync(0xffffffffu, lo, o);
      add(other);
      lo += rest;
    }
  }
};

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// the block's sums together, on its first thread. `far`: what was taken in fp64 (zero for almost every block)
__device__ __forceinline__ double block_sum(Sum near, double far, double* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool any = __syncthreads_or(far != 0.0);  // (NaN too)
  if (any) {
    far = warp_sum64(far);
    if (lane == 0) sh[warp] = far;
    __syncthreads();
    far = 0.0;
    if (threadIdx.x == 0) {
      for (int w = 0; w < warps; ++w) far += sh[w];
    }
    __syncthreads();
  }
  near.add_of_warp();
  float2* pairs = reinterpret_cast<float2*>(sh);
  if (lane == 0) pairs[warp] = make_float2(near.hi, near.lo);
  __syncthreads();
  if (warp == 0) {
    const float2 mine = lane < warps ? pairs[lane] : make_float2(0.0f, 0.0f);
    near.hi = mine.x, near.lo = mine.y;
    near.add_of_warp();
  }
  return far + ((double)near.hi + (double)near.lo);
}

// Squares of what a thread reads of a unit, added to `total`.
template <typename G, int kMax>
__device__ __forceinline__ void add_unit(const many::Table<Entry, kMax>& table, int unit, Sum& near, double& far) {
  const int which = table.find(unit);
  const Entry t = table.entry[which];
  const int64_t start = (int64_t)(unit - table.first[which]) * (kPasses * kPass);
  Raw8<G> raw[kPasses];
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int64_t at = start + pass * kPass + (int64_t)threadIdx.x * 8, left = t.n - at;
    raw[pass] = raw_load8<G>(static_cast<const typename G::T*>(t.grad) + at, t.vec != 0, left >= 8 ? 8 : left > 0 ? (int)left : 0);
  }
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    float g[8];
    raw_get8<G>(raw[pass], g);
    float s = 0.0f, most = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s = fmaf(g[i], g[i], s);
      most = fmaxf(most, fabsf(g[i]));
    }
    if ((s >= 0x1p-100f && s <= 0x1p78f) || (s == 0.0f && most == 0.0f)) {
      near.add(s);  // (2^39 of these are below fp32's largest)
    } else {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) far += (double)g[i] * (double)g[i];
    }
  }
}

template <typename G, int kMax>
__global__ void __launch_bounds__(kThreads) sums_kernel(const __grid_constant__ many::Table<Entry, kMax> table,
                                                        double* __restrict__ parts) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sh[32];
  Sum near;
  double far = 0.0;
  for (int unit = blockIdx.x; unit < table.first[table.count]; unit += gridDim.x) add_unit<G, kMax>(table, unit, near, far);
  const double total = block_sum(near, far, sh);
  if (threadIdx.x == 0) parts[blockIdx.x] = total;
}

__device__ __forceinline__ void write_result(double total, float scale, float max_norm, float* result) {
  const double norm = (double)scale * sqrt(total);
  const float norm32 = (float)norm;
  result[0] = norm32;
  const double clip = (double)max_norm / (norm + 1e-6);
  result[1] = fabsf(norm32) < INFINITY ? (float)((double)scale * (clip < 1.0 ? clip : 1.0)) : __int_as_float(0x7fc00000);
}

constexpr int kFinish = 128;
__global__ void __launch_bounds__(kFinish) finish_kernel(const double* __restrict__ parts, int n, float scale, float max_norm,
                                                         float* __restrict__ result) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sh[kFinish / 32];
  double total = 0.0;
  for (int i = threadIdx.x; i < n; i += kFinish) total += parts[i];
  total = warp_sum64(total);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    total = 0.0;
    for (int w = 0; w < kFinish / 32; ++w) total += sh[w];
    write_result(total, scale, max_norm, result);
  }
}

template <typename G, int kMax>
cudaError_t launch_some(const ftmoe_grad_list& list, int from, int to, double* parts, int& blocks, cudaStream_t st) {
  many::Table<Entry, kMax> table = {};
  int units = 0;
  for (int i = from; i < to; ++i) {
    const ftmoe_grad& t = list.grads[i];
    if (t.n == 0) continue;
    table.entry[table.count] = {t.n, t.grad, (uintptr_t)t.grad % 16 == 0};
    table.first[table.count++] = units;
    units += (int)cdiv(t.n, kPasses * kPass);
  }
  table.first[table.count] = units;
  blocks = std::min(units, grid_of<G>());
  return launch_kernel(sums_kernel<G, kMax>, dim3(blocks), dim3(kThreads), 0, st, true, table, parts);
}

template <typename F>
cudaError_t for_launches(const ftmoe_grad_list& list, F f) {
  return many::for_launches(list.count, kMany, [&](int i) { return list.grads[i].n; },
                            [&](int from, int to, int taken, int) { return f(from, to, taken); });
}

}  // namespace grad_norm

size_t grad_norm_workspace(const ftmoe_grad_list& list) {
  int launches = 0;
  grad_norm::for_launches(list, [&](int, int, int) { ++launches; return cudaSuccess; });
  return (size_t)(launches > 0 ? launches : 1) * grad_norm::kGrid * sizeof(double);
}

cudaError_t launch_grad_norm(const ftmoe_grad_list& list, float scale, float max_norm, double* parts, float* result,
                             cudaStream_t st) {
  using namespace grad_norm;
  OverlapLaunch overlap;
  int n = 0;
  const cudaError_t e = for_launches(list, [&](int from, int to, int taken) {
    int blocks = 0;
    const cudaError_t e = with_elem(list.dtype, [&](auto g) {
      using G = decltype(g);
      return taken <= kFew ? launch_some<G, kFew>(list, from, to, parts + n, blocks, st)
                           : launch_some<G, kMany>(list, from, to, parts + n, blocks, st);
    });
    n += blocks;
    return e;
  });
  if (e != cudaSuccess) return e;
  return launch_kernel(finish_kernel, dim3(1), dim3(kFinish), 0, st, true, (const double*)parts, n, scale, max_norm, result);
}

}  // namespace ftmoe
