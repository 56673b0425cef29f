// SiLU-and-mul that keeps its gate/up rows in 8 bits, and its backward pass from them.
//
// Forward, per row: h = silu(g) * u with silu(g) = g * s, s = 1 / (1 + exp(-g)); g and u are
// kept as e4m3 codes with an fp32 scale per 128 or a power of two per 32. The fp32 scale is amax times
// fp32's 1 / 448, which is what torch's CUDA kernels make of a division by that constant, so that the
// codes are those of rows kept by plain torch operations. The quantizers of the forward divide: their
// scale differs in the last bit for about half of the groups, and a code on a midpoint may then go the
// other way. The scale travels with its codes, and both leave the same error (2.571% of the norm, for
// normal values).
// Backward, with the kept g and u, the gradient dh of the unweighted h and the routing weight w:
//   d h / d u = g s,   d h / d g = u s (1 + g (1 - s))
//   dgu = w dh (d h / d g | d h / d u),   hw = w h,   dweight = sum_i dh_i h_i
// Both passes are elementwise but for the group maxima and dweight. The forward moves 8 bytes per
// intermediate column (4 read, 2 + 2 written) and 1/16 to 1/32 of scales, the backward 10 (2 codes
// and 2 of dh read, 4 + 2 written): memory bounds them, closely followed by the issue rate (about
// 310 and 340 instructions per warp and 8 columns a lane). Reading the bf16 gate/up rows again instead
// would move as many bytes (2 less written, 2 more read a column) and hold twice the memory between the
// passes. Measured on GB300, both passes of 24,576 rows of 2,048 columns, bf16: FP8 156 us (5.8 TB/s, 86%
// of the measured copy rate), MXFP8 156 us (FP8 280 us before packed fp32 pairs, the sigmoid below and
// the loads ahead).
#include <type_traits>

#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"

namespace ftmoe {

namespace act_train {

__device__ __forceinline__ int64_t valid_rows(int64_t rows, const int32_t* rows_dev) {
  if (rows_dev == nullptr) return rows;
  const int64_t d = *rows_dev;
  return d < 0 ? 0 : (d < rows ? d : rows);
}

using Pair = F32Pair;

// The sigmoids 1 / (1 + exp(-x)) of two values x = g + r, r a residual far below g's rounding.
// exp(-x) = 2^t (1 + ln2 (T - t)) with T = -x log2(e) and t its fp32 rounding: the difference T - t,
// from the residual of the product, log2(e)'s low part and r, keeps the exponential to a few units
// in the last place however large |g| is (the rounding of t alone would cost |g| of them). The
// factor is applied as a factor, so that an infinite 2^t stays infinite; it is near 1 unless t has left
// fp32's range, where T - t is infinite or NaN: cut at 2 it leaves a 2^t of zero zero (x above 2.36e38
// has the sigmoid 1, like all x above 17). 1 + e is scaled by 2^-24
// before the reciprocal, which would flush to zero from 2^126 on, and its result again. (Where
// exp(-x) passes fp32's range, x < -88.7, the sigmoid is 0; its value there is below 1e-38.)
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f, kDown = 0x1p-24f;
template <bool kResidual>
__device__ __forceinline__ Pair sigmoid(Pair g, Pair r) {
  const Pair l(-kLog2e), t = g * l, minus(-1.0f);
  Pair rest = fma2(g, Pair(-kLog2eLow), fma2(g, l, t * minus));
  if constexpr (kResidual) rest = fma2(r, l, rest);
  float t_lo, t_hi;
  t.get(t_lo, t_hi);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t_lo));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(t_hi));
  float f_lo, f_hi;
  fma2(rest, Pair(kLn2), Pair(1.0f)).get(f_lo, f_hi);
  const Pair e = Pair(t_lo, t_hi) * Pair(fminf(f_lo, 2.0f), fminf(f_hi, 2.0f));
  float y_lo, y_hi;
  fma2(e, Pair(kDown), Pair(kDown)).get(y_lo, y_hi);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y_lo));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(y_hi));
  return Pair(y_lo, y_hi) * Pair(kDown);
}

// Codes of 8 values that share a maximum with the lanes around them: 16 lanes (FP8's group of
// 128) or 4 (MXFP8's 32). Every lane of the warp calls it. sc: the group's fp32 scale, or the
// E8M0 byte.
template <bool kMx>
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float& sc, uint8_t& byte) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
  for (int o = kMx ? 2 : 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float q[8];
  if constexpr (kMx) {
    // floor(log2 m) off the exponent field; a zero or subnormal maximum takes the smallest scale
    const int ef = (int)((__float_as_uint(m) >> 23) & 0xff);
    const int shared = ef == 0 || ef < 8 ? -127 : ef - 127 - 8;
    byte = (uint8_t)(shared + 127);
    const float f = __uint_as_float((uint32_t)(127 - shared) << 23);  // 2^-shared, exact
#pragma unroll
    for (int i = 0; i < 8; i += 2) (Pair(v[i], v[i + 1]) * Pair(f)).get(q[i], q[i + 1]);
  } else {
    sc = m * (1.0f / kE4M3Max);
    if (!(m > 0.0f)) return make_uint2(0u, 0u);
    if (sc >= 0x1p-100f && sc <= 0x1p100f) {
      // v / sc as IEEE division rounds it, by one reciprocal and Markstein's correction (see
      // SharedDivisor). The residual is taken with the sign that leaves a zero quotient its own:
      // q0 sc - v is +0 for v = -0, and q0 - (+0) y stays -0.
      const Pair y(__fdiv_rn(1.0f, sc)), ny(-__fdiv_rn(1.0f, sc)), d(sc), minus(-1.0f);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const Pair x(v[i], v[i + 1]), q0 = x * y;
        fma2(fma2(q0, d, x * minus), ny, q0).get(q[i], q[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = div_rn(v[i], sc);
    }
  }
  return make_uint2((uint32_t)f2_to_e4m3x2(q[0], q[1]) | ((uint32_t)f2_to_e4m3x2(q[2], q[3]) << 16),
                    (uint32_t)f2_to_e4m3x2(q[4], q[5]) | ((uint32_t)f2_to_e4m3x2(q[6], q[7]) << 16));
}

__device__ __forceinline__ void store_codes(uint8_t* q, uint2 c, bool vec, int n) {
  if (vec && n >= 8) {
    *reinterpret_cast<uint2*>(q) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// The walk of a thread over its (row, pass of 8 columns) pairs: kTpr threads per row, 256 / kTpr
// rows per CTA at a time, CTAs over the rows in a grid stride. Each kernel loads the next pair's
// operands before it works on the current one: at these kernels' arithmetic per byte the loads of
// one pair per thread do not cover the memory's latency.
template <int kTpr>
struct Walk {
  static constexpr int kRows = 256 / kTpr;
  int64_t row, limit, step;
  int inter, c0, n;  // first column of this thread's eight, and how many of them exist (0: nothing to do)
  __device__ __forceinline__ Walk(int64_t limit_, int64_t inter_)
      : row((int64_t)blockIdx.x * kRows + threadIdx.x / kTpr), limit(limit_), step((int64_t)gridDim.x * kRows),
        inter((int)inter_), c0((int)(threadIdx.x % kTpr) * 8) {
    count();
  }
  __device__ __forceinline__ void count() {
    const int left = row < limit ? inter - c0 : 0;
    n = left >= 8 ? 8 : left > 0 ? left : 0;
  }
  // whether the CTA has anything left: the same for all of its threads
  __device__ __forceinline__ bool any() const { return row - threadIdx.x / kTpr < limit; }
  __device__ __forceinline__ bool last_pass() const { return c0 - (int)(threadIdx.x % kTpr) * 8 + kTpr * 8 >= inter; }
  __device__ __forceinline__ void next() {
    if (last_pass()) {
      row += step;
      c0 = (int)(threadIdx.x % kTpr) * 8;
    } else {
      c0 += kTpr * 8;
    }
    count();
  }
};

template <typename In, typename Out, bool kMx, int kTpr>
__global__ void __launch_bounds__(256, 4) silu_save_kernel(
    const typename In::T* __restrict__ gu, int64_t rows, int64_t inter, int64_t ld_gu,
    const int32_t* __restrict__ rows_dev, typename Out::T* __restrict__ h, int64_t ld_h, uint8_t* __restrict__ q,
    void* __restrict__ scales, bool vec_gu, bool vec_h, bool vec_q) {
  const int nb = (int)(kMx ? inter / kMxBlock : (inter + kGroup - 1) / kGroup);
  pdl_wait();
  pdl_trigger();
  Walk<kTpr> at(valid_rows(rows, rows_dev), inter);
  auto load = [&](Raw8<In>& g, Raw8<In>& u) {
    const typename In::T* gr = gu + at.row * ld_gu + at.c0;
    g = raw_load8<In>(gr, vec_gu, at.n);
    u = raw_load8<In>(gr + inter, vec_gu, at.n);
  };
  Raw8<In> g_next, u_next;
  load(g_next, u_next);
  while (at.any()) {  // (the same for the whole CTA, so every shuffle sees all lanes)
    float g[8], u[8], a[8];
    raw_get8<In>(g_next, g);
    raw_get8<In>(u_next, u);
    const int64_t row = at.row;
    const int c0 = at.c0, n = at.n;
    at.next();
    load(g_next, u_next);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const Pair x(g[i], g[i + 1]);
      (x * sigmoid<false>(x, x) * Pair(u[i], u[i + 1])).get(a[i], a[i + 1]);
    }
    float sg, su;
    uint8_t bg, bu;
    const uint2 cg = quantize8<kMx>(g, sg, bg), cu = quantize8<kMx>(u, su, bu);
    if (n > 0) {
      elem_store8<Out>(h + row * ld_h + c0, vec_h, n, a);
      uint8_t* qr = q + row * 2 * inter + c0;
      store_codes(qr, cg, vec_q, n);
      store_codes(qr + inter, cu, vec_q, n);
      if constexpr (kMx) {
        if ((threadIdx.x & 3) == 0) {
          uint8_t* s = static_cast<uint8_t*>(scales) + row * 2 * nb + c0 / kMxBlock;
          s[0] = bg;
          s[nb] = bu;
        }
      } else if ((threadIdx.x & 15) == 0) {
        float* s = static_cast<float*>(scales) + row * 2 * nb + c0 / kGroup;
        s[0] = sg;
        s[nb] = su;
      }
    }
  }
}

// n (at most 8) codes at q, the rest zero
__device__ __forceinline__ uint2 load_codes(const uint8_t* q, bool vec, int n) {
  if (vec && n >= 8) return *reinterpret_cast<const uint2*>(q);
  uint32_t c[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) c[i >> 2] |= (uint32_t)q[i] << (8 * (i & 3));
  return make_uint2(c[0], c[1]);
}
__device__ __forceinline__ Pair code_pair(uint2 c, int i) {  // codes i and i + 1, i even
  const uint32_t w = i < 4 ? c.x : c.y;
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (8 * (i & 3))), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return Pair(f.x, f.y);
}

// dweights: a thread adds its even and its odd columns in ascending order, then both, a butterfly
// over the warp and the warps in order.
template <typename Elem, bool kMx, int kTpr>
__global__ void __launch_bounds__(256, 4) silu_backward_kernel(
    const uint8_t* __restrict__ q, const void* __restrict__ scales, int64_t rows, int64_t inter,
    const int32_t* __restrict__ rows_dev, const typename Elem::T* __restrict__ dh, int64_t ld_dh,
    const float* __restrict__ row_weights, typename Elem::T* __restrict__ dgu, int64_t ld_dgu,
    typename Elem::T* __restrict__ hw, int64_t ld_hw, float* __restrict__ dweights, bool vec_q, bool vec_dh,
    bool vec_dgu, bool vec_hw) {
  constexpr int kWarps = kTpr / 32;
  __shared__ float part[2][8];
  const int sub = threadIdx.x / kTpr, tid = threadIdx.x % kTpr, lane = threadIdx.x & 31;
  const int nb = (int)(kMx ? inter / kMxBlock : (inter + kGroup - 1) / kGroup);
  pdl_wait();
  pdl_trigger();
  Walk<kTpr> at(valid_rows(rows, rows_dev), inter);
  struct Operands {
    uint2 g, u;
    Raw8<Elem> d;
    float sg, su, w;
  };
  auto load = [&](Operands& o) {
    const uint8_t* qr = q + at.row * 2 * inter + at.c0;
    o.g = load_codes(qr, vec_q, at.n);
    o.u = load_codes(qr + inter, vec_q, at.n);
    o.d = raw_load8<Elem>(dh + at.row * ld_dh + at.c0, vec_dh, at.n);
    o.sg = o.su = 0.0f;
    o.w = 1.0f;
    if (at.n > 0) {
      if constexpr (kMx) {
        const uint8_t* s = static_cast<const uint8_t*>(scales) + at.row * 2 * nb + at.c0 / kMxBlock;
        o.sg = e8m0_to_f(s[0]);
        o.su = e8m0_to_f(s[nb]);
      } else {
        const float* s = static_cast<const float*>(scales) + at.row * 2 * nb + at.c0 / kGroup;
        o.sg = s[0];
        o.su = s[nb];
      }
      if (row_weights != nullptr) o.w = row_weights[at.row];
    }
  };
  const Pair one(1.0f), minus(-1.0f);
  Pair dot2(0.0f);  // columns of even and of odd index
  int phase = 0;
  Operands next;
  load(next);
  while (at.any()) {
    const Operands o = next;
    const int64_t row = at.row;
    const int c0 = at.c0, n = at.n;
    const bool last = at.last_pass(), live = row < at.limit;
    at.next();
    load(next);
    float dg[8], du[8], hv[8], d[8];
    raw_get8<Elem>(o.d, d);
    const Pair w2(o.w), sg2(o.sg), su2(o.su);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const Pair gc = code_pair(o.g, i), g2 = gc * sg2, u2 = code_pair(o.u, i) * su2, d2(d[i], d[i + 1]);
      // (the rounding error of code * scale, exact by FMA; a power of two makes none)
      const Pair s = sigmoid<!kMx>(g2, fma2(gc, sg2, g2 * minus));
      const Pair silu = g2 * s, h = silu * u2, wd = w2 * d2;
      dot2 = fma2(d2, h, dot2);
      (wd * u2 * fma2(silu, fma2(s, minus, one), s)).get(dg[i], dg[i + 1]);
      (wd * silu).get(du[i], du[i + 1]);
      (w2 * h).get(hv[i], hv[i + 1]);
    }
    if (n > 0) {
      elem_store8<Elem>(dgu + row * ld_dgu + c0, vec_dgu, n, dg);
      elem_store8<Elem>(dgu + row * ld_dgu + inter + c0, vec_dgu, n, du);
      if (hw != nullptr) elem_store8<Elem>(hw + row * ld_hw + c0, vec_hw, n, hv);
    }
    if (last && dweights != nullptr) {  // (uniform over the CTA)
      float dot, odd;
      dot2.get(dot, odd);
      dot += odd;
      dot2 = Pair(0.0f);
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
      if constexpr (kWarps == 1) {
        if (live && lane == 0) dweights[row] = dot;
      } else {
        // two buffers in turn: a warp may begin the next row's sum while another still reads this one
        if (lane == 0) part[phase][threadIdx.x >> 5] = dot;
        __syncthreads();
        if (live && tid == 0) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < kWarps; ++i) sum += part[phase][sub * kWarps + i];
          dweights[row] = sum;
        }
        phase ^= 1;
      }
    }
  }
}

// Four CTAs per SM (64 registers a thread), each walking its share of the rows.
static int grid_for(int64_t rows, int tpr) {
  const int64_t blocks = cdiv(rows, 256 / tpr), cap = (int64_t)sm_count_once() * 4;
  return (int)(blocks < cap ? blocks : cap);
}

// as many threads per row as it has runs of 8 columns, so that a thread makes few passes
template <typename F>
static cudaError_t with_threads_per_row(int64_t inter, F f) {
  if (inter <= 256) return f(std::integral_constant<int, 32>{});
  if (inter <= 1024) return f(std::integral_constant<int, 128>{});
  return f(std::integral_constant<int, 256>{});
}

}  // namespace act_train

cudaError_t launch_silu_save(const SiluSaveArgs& a, cudaStream_t st) {
  using namespace act_train;
  return with_elem(a.gu_dtype, [&](auto in) {
    return with_elem(a.h_dtype, [&](auto out) {
      return with_threads_per_row(a.inter, [&](auto t) {
        using In = decltype(in);
        using Out = decltype(out);
        constexpr int kTpr = decltype(t)::value;
        // the up half begins at column inter: it has to keep the vectors' alignment
        const bool vg = elem_vec_ok(a.gu, a.ld_gu, sizeof(typename In::T)) && a.inter % 8 == 0;
        const bool vh = elem_vec_ok(a.h, a.ld_h, sizeof(typename Out::T));
        const bool vq = (uintptr_t)a.q % 8 == 0 && a.inter % 8 == 0;
        auto k = a.mx ? silu_save_kernel<In, Out, true, kTpr> : silu_save_kernel<In, Out, false, kTpr>;
        const OverlapLaunch overlap;
        return launch_kernel(k, dim3(grid_for(a.rows, kTpr)), dim3(256), 0, st, true,
                             static_cast<const typename In::T*>(a.gu), a.rows, a.inter, a.ld_gu, a.rows_dev,
                             static_cast<typename Out::T*>(a.h), a.ld_h, a.q, a.scales, vg, vh, vq);
      });
    });
  });
}

cudaError_t launch_silu_backward(const SiluBackwardArgs& a, cudaStream_t st) {
  using namespace act_train;
  return with_elem(a.dtype, [&](auto elem) {
    using E = decltype(elem);
    using T = typename E::T;
    const bool vq = (uintptr_t)a.q % 8 == 0 && a.inter % 8 == 0;
    const bool vd = elem_vec_ok(a.dh, a.ld_dh, sizeof(T));
    const bool vgu = elem_vec_ok(a.dgu, a.ld_dgu, sizeof(T)) && a.inter % 8 == 0;
    const bool vhw = a.hw == nullptr || elem_vec_ok(a.hw, a.ld_hw, sizeof(T));
    return with_threads_per_row(a.inter, [&](auto t) {
      constexpr int kTpr = decltype(t)::value;
      auto k = a.mx ? silu_backward_kernel<E, true, kTpr> : silu_backward_kernel<E, false, kTpr>;
      const OverlapLaunch overlap;
      return launch_kernel(k, dim3(grid_for(a.rows, kTpr)), dim3(256), 0, st, true, a.q, a.scales, a.rows, a.inter,
                           a.rows_dev, static_cast<const T*>(a.dh), a.ld_dh, a.row_weights, static_cast<T*>(a.dgu),
                           a.ld_dgu, static_cast<T*>(a.hw), a.ld_hw, a.dweights, vq, vd, vgu, vhw);
    });
  });
}

}  // namespace ftmoe
