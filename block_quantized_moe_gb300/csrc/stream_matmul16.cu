// The product grouped by expert for a handful of rows (decoding): out[r, i] = sum_j a[r, j] w[e, i, j]
// with about one row per expert. Every weight is used for a few rows, so reading it is most of what
// there is: 2 n k bytes per expert that has rows.
//
// A warp takes one weight row i: its lanes hold up to 2,048 of the row's elements in registers,
// eight 16-byte loads in flight each, and multiply them with up to four rows of a (from L2, then
// L1) before the next piece; fp32 sums, one butterfly per output. More than four rows of an expert
// take another pass over its weights, and every row costs issue slots and reads of a (one expert,
// 2048 x 4096: one row 7.1 us, four 17.2, eight 31.5), which bounds where this kernel is used. Eight warps of a CTA take eight
// consecutive i. All SMs stream, whatever the number of experts: the tensor-core kernel's units
// of 256 weight rows leave most of the SMs idle here (two rows over two experts, 1536 x 2048: 12
// units). Measured there: 5.0 us, of which about 3 are launch and the offsets' round trip; one row,
// 4096 x 7168: 19 us (3 TB/s).
#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"

namespace ftmoe {

namespace stream16 {

constexpr int kWarps = 8, kPieces = 8, kRows = 4;

__device__ __forceinline__ uint4 ld_weights(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <typename Elem>
__device__ __forceinline__ float dot8(uint4 x, uint4 y, float acc) {
  const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc = fmaf(Elem::get((uint16_t)(a[i] & 0xffffu)), Elem::get((uint16_t)(b[i] & 0xffffu)), acc);
    acc = fmaf(Elem::get((uint16_t)(a[i] >> 16)), Elem::get((uint16_t)(b[i] >> 16)), acc);
  }
  return acc;
}

struct Params {
  const uint16_t* a;
  int64_t ld_a;
  const int32_t* offsets;
  int64_t rows;
  const uint16_t* w;
  int64_t ld, expert_stride;
  int n, k, E;
  void* out;
  int64_t ld_out;
  int out_dtype;
};

template <typename Elem>
__global__ void __launch_bounds__(32 * kWarps) stream_matmul16_kernel(Params p) {
  __shared__ int s_e[32 * kWarps], s_lo[32 * kWarps], s_m[32 * kWarps], s_count[kWarps + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = (p.n + kWarps - 1) / kWarps;
  pdl_wait();
  pdl_trigger();
  // 256 experts at a time: those that have rows, in order
  for (int base = 0; base < p.E; base += 32 * kWarps) {
    const int e = base + threadIdx.x;
    int lo = 0, m = 0;
    if (e < p.E) {
      // (both cut to [0, rows], so that no difference of them leaves 32 bits)
      const int most = (int)p.rows;
      lo = max(0, min(__ldg(p.offsets + e), most));
      m = max(0, min(__ldg(p.offsets + e + 1), most)) - lo;
    }
    const uint32_t have = __ballot_sync(0xffffffffu, m > 0);
    __syncthreads();  // the previous pass has read the list
    if (lane == 0) s_count[warp] = __popc(have);
    __syncthreads();
    int at = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) at += s_count[i];
      total += s_count[i];
    }
    if (m > 0) {
      at += __popc(have & ((1u << lane) - 1u));
      s_e[at] = e;
      s_lo[at] = lo;
      s_m[at] = m;
    }
    __syncthreads();
    for (int64_t u = blockIdx.x; u < (int64_t)total * blocks; u += gridDim.x) {
      const int idx = (int)(u / blocks), i = (int)(u - (int64_t)idx * blocks) * kWarps + warp;
      if (i >= p.n) continue;
      const uint16_t* wr = p.w + (int64_t)s_e[idx] * p.expert_stride + (int64_t)i * p.ld;
      const int first = s_lo[idx], count = s_m[idx];
      for (int r0 = 0; r0 < count; r0 += kRows) {
        const uint16_t* ar = p.a + (int64_t)(first + r0) * p.ld_a;
        const int live = min(kRows, count - r0);
        float acc[kRows] = {};
        for (int k0 = lane * 8; k0 < p.k; k0 += kPieces * 256) {
          uint4 wv[kPieces];
#pragma unroll
          for (int j = 0; j < kPieces; ++j)
            wv[j] = k0 + j * 256 < p.k ? ld_weights(wr + k0 + j * 256) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (r >= live) break;
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
              if (k0 + j * 256 < p.k)
                acc[r] = dot8<Elem>(wv[j], *reinterpret_cast<const uint4*>(ar + r * p.ld_a + k0 + j * 256), acc[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (r >= live) break;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
          if (lane == 0) {
            const int64_t at_out = (int64_t)(first + r0 + r) * p.ld_out + i;
            if (p.out_dtype == FTMOE_OUT_FP32)
              static_cast<float*>(p.out)[at_out] = acc[r];
            else
              static_cast<uint16_t*>(p.out)[at_out] = p.out_dtype == FTMOE_OUT_BF16 ? OutBf16::cvt(acc[r]) : OutF16::cvt(acc[r]);
          }
        }
      }
    }
  }
}

}  // namespace stream16

bool stream_matmul16_ok(const Matmul16Args& a) {
  const ftmoe_matrix_bank& w = a.w;
  return !a.wgrad && !a.input_grad && w.k % 8 == 0 && elem_vec_ok(a.a, a.ld_a, 2) && elem_vec_ok(w.w, w.ld, 2) &&
         (w.num_experts == 1 || w.expert_stride % 8 == 0);
}

cudaError_t launch_stream_matmul16(const Matmul16Args& a, cudaStream_t st) {
  using namespace stream16;
  const ftmoe_matrix_bank& w = a.w;
  Params p;
  p.a = static_cast<const uint16_t*>(a.a);
  p.ld_a = a.ld_a;
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.w = static_cast<const uint16_t*>(w.w);
  p.ld = w.ld;
  p.expert_stride = w.expert_stride;
  p.n = (int)w.n;
  p.k = (int)w.k;
  p.E = w.num_experts;
  p.out = a.out;
  p.ld_out = a.ld_out;
  p.out_dtype = a.out_dtype;
  const int64_t units = (a.rows < p.E ? a.rows : p.E) * cdiv(w.n, kWarps), cap = (int64_t)sm_count_once() * 4;
  const int grid = (int)(units < cap ? units : cap);
  const OverlapLaunch overlap;
  return launch_kernel(a.dtype == FTMOE_OUT_BF16 ? stream_matmul16_kernel<ElemBf16> : stream_matmul16_kernel<ElemF16>,
                       dim3(grid), dim3(32 * kWarps), 0, st, true, p);
}

}  // namespace ftmoe
