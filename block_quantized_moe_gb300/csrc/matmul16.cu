// Products grouped by expert in 16 bits, the general kernel: any sizes, strides and alignment.
//
// The three directions are one contraction over rows of an expert's segment [lo, hi):
//   product       out[r, i]    = sum_j a[r, j] w[e, i, j]
//   input grad    out[r, j]    = sum_i a[r, i] w[e, i, j]
//   weight grad   dw[e, i, j] (+)= sum_r dy[r, i] x[r, j]
// each written as D[i, j] = sum_l A[i, l] B[l, j] with element strides. A block takes 64 x 64
// outputs, a thread 4 x 4 of them in fp32 registers, the contraction in steps of 16 through
// shared memory. It runs where the tensor cores cannot: TMA wants 16-byte bases and row
// strides. fp32 FMAs and the strided loads bound it: 145 us for the weight gradient of 333 rows
// over 8 experts, 1536 x 2048 (14 TFLOP/s; the tensor cores take 24 us).
#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"

namespace ftmoe {

namespace mm16 {

constexpr int kT = 64, kStep = 16, kPer = 4;

struct Params {
  const void* a;
  const void* b;
  const uint8_t* bs;   // scale bytes of b where it holds MXFP8 codes
  void* d;
  const int32_t* offsets;
  int64_t rows;
  int64_t ai, al, bl, bj, di;    // element strides (D's columns are contiguous)
  int64_t be, de;                // per expert
  int64_t m, n, l;               // D is m x n per expert; m or l is the row count for the ragged one
  int64_t bs_ld;                 // scale bytes per row of b
  int32_t E, ragged_m, accumulate;
};

__device__ __forceinline__ void segment(const Params& p, int e, int64_t& lo, int64_t& hi) {
  lo = p.offsets[e];
  hi = p.offsets[e + 1];
  lo = lo < 0 ? 0 : lo;
  hi = hi > p.rows ? p.rows : hi;
  if (hi < lo) hi = lo;
}

template <typename In, typename Out, bool kSaved>
__global__ void __launch_bounds__(256) general_kernel(Params p) {
  __shared__ float sa[kStep][kT + 1], sb[kStep][kT + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t nj = (p.n + kT - 1) / kT;
  int64_t done = 0;  // units of the experts before e
  int64_t unit = blockIdx.x;
  for (int e = 0; e < p.E; ++e) {
    int64_t lo, hi;
    segment(p, e, lo, hi);
    const int64_t m = p.ragged_m ? hi - lo : p.m, len = p.ragged_m ? p.l : hi - lo;
    // (nothing to add keeps the old values as they are, zeros of either sign and NaN among them)
    const int64_t units = p.accumulate && len == 0 ? 0 : ((m + kT - 1) / kT) * nj;
    for (; unit < done + units; unit += gridDim.x) {
      const int64_t local = unit - done;
      const int64_t i0 = local / nj * kT, j0 = local % nj * kT;
      const int64_t arow = p.ragged_m ? lo * p.ai : lo * p.al;
      const typename In::T* a = static_cast<const typename In::T*>(p.a) + arow;
      const int64_t brow = p.ragged_m ? (int64_t)e * p.be : lo * p.bl;
      float acc[kPer][kPer] = {};
      for (int64_t l0 = 0; l0 < len; l0 += kStep) {
#pragma unroll
        for (int v = 0; v < kT * kStep / 256; ++v) {
          const int t = threadIdx.x + 256 * v;
          // consecutive threads along the operand's contiguous axis
          const int ai = p.al == 1 ? t / kStep : t % kT, al = p.al == 1 ? t % kStep : t / kT;
          sa[al][ai] = i0 + ai < m && l0 + al < len ? In::get(a[(i0 + ai) * p.ai + (l0 + al) * p.al]) : 0.0f;
          const int bj = p.bl == 1 ? t / kStep : t % kT, bl = p.bl == 1 ? t % kStep : t / kT;
          float b = 0.0f;
          if (j0 + bj < p.n && l0 + bl < len) {
            const int64_t at = brow + (l0 + bl) * p.bl + (j0 + bj) * p.bj;
            if constexpr (kSaved) {
              const uint8_t s = p.bs[(lo + l0 + bl) * p.bs_ld + (j0 + bj) / kMxBlock];
              b = In::get(In::put(e4m3_to_f(static_cast<const uint8_t*>(p.b)[at]) * e8m0_to_f(s)));
            } else {
              b = In::get(static_cast<const typename In::T*>(p.b)[at]);
            }
          }
          sb[bl][bj] = b;
        }
        __syncthreads();
#pragma unroll
        for (int l = 0; l < kStep; ++l) {
          float av[kPer], bv[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) av[i] = sa[l][ty + 16 * i], bv[i] = sb[l][tx + 16 * i];
#pragma unroll
          for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int j = 0; j < kPer; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
        }
        __syncthreads();
      }
      const int64_t drow = p.ragged_m ? lo * p.di : (int64_t)e * p.de;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int64_t r = i0 + ty + 16 * i, c = j0 + tx + 16 * j;
          if (r < m && c < p.n) {
            typename Out::T* o = static_cast<typename Out::T*>(p.d) + drow + r * p.di + c;
            *o = Out::put(p.accumulate ? Out::get(*o) + acc[i][j] : acc[i][j]);
          }
        }
    }
    done += units;
  }
}

static cudaError_t run(const Params& p, int32_t in_dtype, int32_t out_dtype, bool saved, int64_t units,
                       cudaStream_t st) {
  const int64_t cap = (int64_t)sm_count() * 8;
  const int grid = (int)(units < 1 ? 1 : (units < cap ? units : cap));
  return with_elem(out_dtype, [&](auto out) {
    using Out = decltype(out);
    auto go = [&](auto kernel) { return launch_kernel(kernel, dim3(grid), dim3(256), 0, st, false, p); };
    if (in_dtype == FTMOE_OUT_BF16)
      return saved ? go(general_kernel<ElemBf16, Out, true>) : go(general_kernel<ElemBf16, Out, false>);
    return saved ? go(general_kernel<ElemF16, Out, true>) : go(general_kernel<ElemF16, Out, false>);
  });
}

}  // namespace mm16

cudaError_t launch_matmul16_general(const Matmul16Args& a, cudaStream_t st) {
  mm16::Params p = {};
  const ftmoe_matrix_bank& w = a.w;
  p.offsets = a.offsets;
  p.rows = a.rows;
  p.E = w.num_experts;
  if (a.wgrad) {
    p.a = a.a;          // dy^T: i over n, l over rows
    p.ai = 1;
    p.al = a.ld_a;
    p.b = a.x;
    p.bs = a.x_scales;
    p.bs_ld = w.k / kMxBlock;
    p.bl = a.ld_x;
    p.bj = 1;
    p.d = w.w;
    p.di = w.ld;
    p.de = w.expert_stride;
    p.m = w.n;
    p.n = w.k;
    p.accumulate = a.accumulate;
    return mm16::run(p, a.dtype, w.dtype, a.x_scales != nullptr, (int64_t)w.num_experts * cdiv(p.m, 64) * cdiv(p.n, 64),
                     st);
  }
  p.a = a.a;
  p.ai = a.ld_a;
  p.al = 1;
  p.b = w.w;
  p.be = w.expert_stride;
  p.bl = a.input_grad ? w.ld : 1;
  p.bj = a.input_grad ? 1 : w.ld;
  p.d = a.out;
  p.di = a.ld_out;
  p.n = a.input_grad ? w.k : w.n;
  p.l = a.input_grad ? w.n : w.k;
  p.ragged_m = 1;
  return mm16::run(p, a.dtype, a.out_dtype, false, (cdiv(a.rows, 64) + w.num_experts) * cdiv(p.n, 64), st);
}

// The streaming kernel where its rows, times units of 256 weight rows, are at most a quarter of the
// SMs (38), and an expert has at most the four rows that one pass over its weights takes, on average. It
// fills the GPU whatever the number of units, but its time grows with every row; the tensor-core
// kernel's is that of one unit until the units are more than half of the CTA pairs. Measured on GB300,
// one launch after another (streaming, tensor cores, us):
//   1 expert, 1536 x 2048:  1 row 4.0, 10.8;  2 rows 5.7, 10.9;  4 rows 9.2, 11.1;  5 rows 11.3, 11.1
//   1 expert, 2048 x 4096:  1 row 7.1, 18.5;  4 rows 17.2, 18.6;  8 rows 31.5, 18.9
//   1 expert, 4096 x 7168:  1 row 19.6, 30.0;  2 rows 31.0, 30.0;  4 rows 53.1, 30.0;  16 rows 198, 30.5
//   rows spread over 8 experts, 512 x 7168:  4 rows 11.7, 29.5;  8 rows 18.7, 30.2;  16 rows 30.0, 30.2
//   over 8 experts, 1536 x 2048:  5 rows 9.8, 12.1;  8 rows 15.0, 13.4;  16 rows 23.8, 13.5
//   over 2 experts, 1536 x 2048:  5 rows 8.4, 11.4;  12 rows 14.3, 11.4
// (16 rows that all go to one of 8 experts, 512 x 7168, take 102 where the tensor cores would take 26:
// the host does not know where they go.)
static bool prefer_stream(const Matmul16Args& a) {
  return a.rows <= 16 && a.rows <= 4 * (int64_t)a.w.num_experts && a.rows * cdiv(a.w.n, 256) <= sm_count_once() / 4 &&
         stream_matmul16_ok(a);
}

cudaError_t launch_matmul16(const Matmul16Args& a, cudaStream_t st) {
  if (prefer_stream(a)) return launch_stream_matmul16(a, st);
  int unsupported = 0;
  const cudaError_t e = launch_tc_matmul16(a, st, &unsupported);
  return unsupported ? launch_matmul16_general(a, st) : e;
}

}  // namespace ftmoe
