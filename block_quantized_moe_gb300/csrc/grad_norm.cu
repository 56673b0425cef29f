// Global norm of many gradients, and the factor that scales and clips them.
//
// Every gradient is read once (memory bounds it) in units of 8,192 elements that the blocks of a
// fixed grid take in turn; a second launch adds the blocks' sums in order. Squares are summed in
// fp32 over the eight elements that a thread reads together, and, where that sum is neither large nor
// small, over the unit; anything else (an element beyond 2^50 or so, gradients so small that their squares
// would be subnormal, NaN) goes through fp64. Unit sums are added in fp64.
#include "common.cuh"
#include "elem16.cuh"
#include "many.cuh"

namespace ftmoe {

namespace grad_norm {

using many::kPasses;
using many::kThreads;
using many::kUnit;

struct Entry {
  int64_t n;
  const void* grad;
  int32_t vec;
};

constexpr int kFew = 64, kMany = 1024;  // gradients of a launch
constexpr int kGrid = 152 * 8;          // blocks of a launch, one part each

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// the block's sum, on thread 0
__device__ __forceinline__ double block_sum64(double v, double* sh) {
  v = warp_sum64(v);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0) {
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) v += sh[w];
  }
  return v;
}

template <typename G, int kMax>
__global__ void __launch_bounds__(kThreads) sums_kernel(const __grid_constant__ many::Table<Entry, kMax> table,
                                                        double* __restrict__ parts) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sh[kThreads / 32];
  double total = 0.0;
  for (int unit = blockIdx.x; unit < table.first[table.count]; unit += gridDim.x) {
    const int which = table.find(unit);
    const Entry& t = table.entry[which];
    const int64_t start = (int64_t)(unit - table.first[which]) * kUnit;
    const bool vec = t.vec != 0;
    float sum = 0.0f;
    Raw8<G> raw[kPasses];
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int64_t at = start + (int64_t)(pass * kThreads + threadIdx.x) * 8, left = t.n - at;
      raw[pass] = raw_load8<G>(static_cast<const typename G::T*>(t.grad) + at, vec, left >= 8 ? 8 : left > 0 ? (int)left : 0);
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
      if ((s >= 0x1p-100f && s <= 0x1p100f) || (s == 0.0f && most == 0.0f)) {
        sum += s;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) total += (double)g[i] * (double)g[i];
      }
    }
    total += (double)sum;
  }
  total = block_sum64(total, sh);
  if (threadIdx.x == 0) parts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) finish_kernel(const double* __restrict__ parts, int n, float scale, float max_norm,
                                                      float* __restrict__ result) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sh[32];
  double total = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) total += parts[i];
  total = block_sum64(total, sh);
  if (threadIdx.x == 0) {
    const double norm = (double)scale * sqrt(total);
    const float norm32 = (float)norm;
    result[0] = norm32;
    const double clip = (double)max_norm / (norm + 1e-6);
    result[1] = fabsf(norm32) < INFINITY ? (float)((double)scale * (clip < 1.0 ? clip : 1.0)) : __int_as_float(0x7fc00000);
  }
}

template <typename G, int kMax>
cudaError_t launch_some(const ftmoe_grad_list& list, int from, int to, double* parts, cudaStream_t st) {
  many::Table<Entry, kMax> table = {};
  int units = 0;
  for (int i = from; i < to; ++i) {
    const ftmoe_grad& t = list.grads[i];
    if (t.n == 0) continue;
    table.entry[table.count] = {t.n, t.grad, (uintptr_t)t.grad % 16 == 0};
    table.first[table.count++] = units;
    units += (int)cdiv(t.n, kUnit);
  }
  table.first[table.count] = units;
  return launch_kernel(sums_kernel<G, kMax>, dim3(kGrid), dim3(kThreads), 0, st, true, table, parts);
}

// The launches of a list: [from, to) of each to f, until there are no more
template <typename F>
cudaError_t for_launches(const ftmoe_grad_list& list, F f) {
  for (int from = 0; from < list.count;) {
    int to = from, taken = 0;
    int64_t units = 0;
    while (to < list.count && taken < kMany) {
      const int64_t n = list.grads[to].n, more = cdiv(n, kUnit);
      if (taken > 0 && units + more > ((int64_t)1 << 30)) break;
      units += more;
      taken += n > 0;
      ++to;
    }
    if (taken > 0) {
      const cudaError_t e = f(from, to, taken);
      if (e != cudaSuccess) return e;
    }
    from = to;
  }
  return cudaSuccess;
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
    const cudaError_t e = with_elem(list.dtype, [&](auto g) {
      using G = decltype(g);
      return taken <= kFew ? launch_some<G, kFew>(list, from, to, parts + n, st) : launch_some<G, kMany>(list, from, to, parts + n, st);
    });
    n += kGrid;
    return e;
  });
  if (e != cudaSuccess) return e;
  return launch_kernel(finish_kernel, dim3(1), dim3(1024), 0, st, true, (const double*)parts, n, scale, max_norm, result);
}

}  // namespace ftmoe
