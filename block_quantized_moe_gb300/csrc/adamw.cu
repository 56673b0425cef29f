// An AdamW step over many tensors in one launch, moments in fp32 or in 8 bits.
//
//   g = grad_scale grad,  m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
//   p = p - (lr decay p + lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps))
// Elementwise: 24 bytes an element and the gradient with fp32 moments, 12 1/8 and the gradient with
// 8-bit ones (p 8, codes 4, scales 1/8), and 2 for a 16-bit copy. Memory bounds it.
//
// 8-bit moments: per 32 elements a power of two, codes e4m3 (m) and e5m2 (v), stochastically
// rounded. With beta2 = 0.999 v moves by a thousandth of itself a step, far below half of e5m2's step: rounded
// to nearest it would never move. A code is cut from the bits of an fp32 number: the value times the power that
// puts the format's least normal on fp32's least normal has the code in its upper bits, subnormal ones
// included, so that adding random bits below them and shifting is the rounding. v's code is at least 1
// where v > 0: a zero under a moment that is not zero would divide it by eps.
// The random bits: a hash per chunk of eight elements, multiplied out by eight odd constants (the halves of each
// 64-bit product combined); 16 bits for m, 16 for v. Constants: fractional parts of square roots of primes.
// The products and sums of m and v are rounded one by one (no fused multiply-add), which any fp32
// program can repeat bit for bit; the codes depend on it.
#include "common.cuh"
#include "elem16.cuh"
#include "many.cuh"

namespace ftmoe {

namespace adamw {

using many::kPasses;
using many::kThreads;
using many::kUnit;

struct Entry {
  int64_t n;
  void* param;
  const void* grad;
  void* m;
  void* v;
  uint8_t* m_scales;
  uint8_t* v_scales;
  void* copy;
  int32_t index;  // place in the caller's list
  int32_t vec;    // every array takes vectors of eight elements
};

// tensors of a launch: kernel parameters up to 4 KB, and up to 32 KB for long lists
constexpr int kFew = 48, kMany = 400;

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}
template <int kJ>
__device__ __forceinline__ uint32_t spread(uint32_t base) {
  constexpr uint32_t kOdd[8] = {0x3C6EF373u, 0xA54FF53Bu, 0x510E527Fu, 0x9B05688Du,
                                0x1F83D9ABu, 0x5BE0CD19u, 0xCBBB9D5Du, 0x629A292Bu};
  const uint64_t h = (uint64_t)base * kOdd[kJ];
  return (uint32_t)h ^ (uint32_t)(h >> 32);
}
__device__ __forceinline__ void noise8(uint32_t base, uint32_t (&h)[8]) {
  h[0] = spread<0>(base), h[1] = spread<1>(base), h[2] = spread<2>(base), h[3] = spread<3>(base);
  h[4] = spread<4>(base), h[5] = spread<5>(base), h[6] = spread<6>(base), h[7] = spread<7>(base);
}

// E8M0 byte of a group with this largest magnitude (the bits of it): the least power for which it is
// at most 1.75 * 2^kTop
template <int kTop>
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  const int power = (int)((bits + 0x1FFFFFu) >> 23) - 127 - kTop;
  return (uint32_t)(max(power, -127) + 127);
}
// 2^(127 - b)
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return byte >= 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return a | (b << 8) | (c << 16) | (d << 24);
}

// eight bytes at p, or the first n of them
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, bool vec, int n) {
  if (vec && n >= 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, bool vec, int n, uint2 c) {
  if (vec && n >= 8) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}

// the values of eight codes
template <__nv_fp8_interpretation_t kFormat>
__device__ __forceinline__ void decode8(uint2 c, float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = (i < 2 ? c.x : c.y) >> (16 * (i & 1));
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), kFormat)));
    v[2 * i] = __fmul_rn(f.x, scale);
    v[2 * i + 1] = __fmul_rn(f.y, scale);
  }
}

__device__ __forceinline__ float square_root(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <typename P, typename G, bool k8, int kMax>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ many::Table<Entry, kMax> table,
                                                         const AdamwConstants c, const int copy_dtype) {
  pdl_wait();
  pdl_trigger();
  const int which = table.find(blockIdx.x);
  const Entry& t = table.entry[which];
  const int64_t start = (int64_t)((int)blockIdx.x - table.first[which]) * kUnit;

  const float grad_scale = c.grad_scale != nullptr ? *c.grad_scale : 1.0f;
  if (!(fabsf(grad_scale) < INFINITY)) return;  // no step
  const float lr = c.lr_dev != nullptr ? *c.lr_dev : c.lr;
  float correction1 = c.correction1, correction2 = c.correction2;
  int64_t step = c.step;
  if (c.step_dev != nullptr) {
    step = max(*c.step_dev, (int64_t)1);
    correction1 = -1.0f / expm1f((float)step * c.ln_beta1);
    correction2 = rsqrtf(-expm1f((float)step * c.ln_beta2));
  }
  const float decay = lr * c.weight_decay, rate = lr * correction1;
  uint32_t key = 0;
  if constexpr (k8) {
    key = mix(mix(mix(c.seed) + (uint32_t)step) + (uint32_t)t.index);
    key = mix(key + (uint32_t)((uint64_t)(start >> 3) >> 32));
  }

#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int64_t at = start + (int64_t)(pass * kThreads + threadIdx.x) * 8;
    const int64_t left = t.n - at;
    // (lanes past the end stay for the exchange between the four lanes of a group)
    if (__all_sync(0xffffffffu, left <= 0)) break;
    const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
    const bool vec = t.vec != 0;
    float p[8], g[8], m[8], v[8];
    raw_get8<P>(raw_load8<P>(static_cast<const typename P::T*>(t.param) + at, vec, n), p);
    raw_get8<G>(raw_load8<G>(static_cast<const typename G::T*>(t.grad) + at, vec, n), g);
    if constexpr (k8) {
      const uint2 mc = load_codes(static_cast<const uint8_t*>(t.m) + at, vec, n);
      const uint2 vc = load_codes(static_cast<const uint8_t*>(t.v) + at, vec, n);
      const float ms = n > 0 ? e8m0_to_f(t.m_scales[at >> 5]) : 0.0f, vs = n > 0 ? e8m0_to_f(t.v_scales[at >> 5]) : 0.0f;
      decode8<__NV_E4M3>(mc, ms, m);
      decode8<__NV_E5M2>(vc, vs, v);
    } else {
      raw_get8<ElemF32>(raw_load8<ElemF32>(static_cast<const float*>(t.m) + at, vec, n), m);
      raw_get8<ElemF32>(raw_load8<ElemF32>(static_cast<const float*>(t.v) + at, vec, n), v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = __fmul_rn(g[i], grad_scale);
      m[i] = __fadd_rn(__fmul_rn(m[i], c.beta1), __fmul_rn(g[i], c.rest1));
      v[i] = __fadd_rn(__fmul_rn(v[i], c.beta2), __fmul_rn(__fmul_rn(g[i], g[i]), c.rest2));
      const float d = fmaf(square_root(v[i]), correction2, c.eps);
      p[i] -= fmaf(rate, m[i] * reciprocal(d), p[i] * decay);
    }
    elem_store8<P>(static_cast<typename P::T*>(t.param) + at, vec, n, p);
    if (copy_dtype == FTMOE_OUT_BF16) elem_store8<ElemBf16>(static_cast<uint16_t*>(t.copy) + at, vec, n, p);
    else if (copy_dtype == FTMOE_OUT_FP16) elem_store8<ElemF16>(static_cast<uint16_t*>(t.copy) + at, vec, n, p);
    if constexpr (k8) {
      uint32_t m_top = 0u, v_top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m_top = i < n ? max(m_top, __float_as_uint(m[i]) & 0x7fffffffu) : m_top;
        v_top = i < n ? max(v_top, __float_as_uint(v[i]) & 0x7fffffffu) : v_top;
      }
      const uint32_t mb = scale_byte<8>(group_max(m_top)), vb = scale_byte<15>(group_max(v_top));
      const float mf = inverse_scale(mb), vf = inverse_scale(vb);
      uint32_t h[8], mq[8], vq[8];
      noise8(mix(key + (uint32_t)(at >> 3)), h);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t sign = (__float_as_uint(m[i]) >> 24) & 0x80u;
        const uint32_t mbits = __float_as_uint(__fmul_rn(__fmul_rn(fabsf(m[i]), mf), 0x1p-120f));
        const uint32_t vbits = __float_as_uint(__fmul_rn(__fmul_rn(v[i], vf), 0x1p-112f)) & 0x7fffffffu;
        mq[i] = min((mbits + ((h[i] & 0xffffu) << 4)) >> 20, 0x7fu) | sign;
        vq[i] = min((vbits + ((h[i] >> 16) << 5)) >> 21, 0x7cu);
        if (v[i] > 0.0f) vq[i] = max(vq[i], 1u);
      }
      store_codes(static_cast<uint8_t*>(t.m) + at, vec, n, make_uint2(pack4(mq[0], mq[1], mq[2], mq[3]), pack4(mq[4], mq[5], mq[6], mq[7])));
      store_codes(static_cast<uint8_t*>(t.v) + at, vec, n, make_uint2(pack4(vq[0], vq[1], vq[2], vq[3]), pack4(vq[4], vq[5], vq[6], vq[7])));
      if ((threadIdx.x & 3) == 0 && n > 0) {
        t.m_scales[at >> 5] = (uint8_t)mb;
        t.v_scales[at >> 5] = (uint8_t)vb;
      }
    } else {
      elem_store8<ElemF32>(static_cast<float*>(t.m) + at, vec, n, m);
      elem_store8<ElemF32>(static_cast<float*>(t.v) + at, vec, n, v);
    }
  }
}

template <typename P, typename G, bool k8, int kMax>
cudaError_t launch_some(const ftmoe_adamw_list& list, int from, int to, const AdamwConstants& c, cudaStream_t st) {
  many::Table<Entry, kMax> table = {};
  int units = 0;
  for (int i = from; i < to; ++i) {
    const ftmoe_adamw_tensor& t = list.tensors[i];
    if (t.n == 0) continue;
    Entry& e = table.entry[table.count];
    e = {t.n, t.param, t.grad, t.m, t.v, static_cast<uint8_t*>(t.m_scales), static_cast<uint8_t*>(t.v_scales), t.copy, i, 0};
    const uintptr_t all16 = (uintptr_t)t.param | (uintptr_t)t.grad | (uintptr_t)t.copy | (k8 ? 0 : (uintptr_t)t.m | (uintptr_t)t.v);
    const uintptr_t all8 = (uintptr_t)t.m | (uintptr_t)t.v;
    e.vec = all16 % 16 == 0 && all8 % 8 == 0;
    table.first[table.count++] = units;
    units += (int)cdiv(t.n, kUnit);
  }
  table.first[table.count] = units;
  if (units == 0) return cudaSuccess;
  return launch_kernel(adamw_kernel<P, G, k8, kMax>, dim3((unsigned)units), dim3(kThreads), 0, st, true, table, c,
                       (int)list.copy_dtype);
}

// A launch takes kMany tensors (kFew where that is all of them) and 2^30 units at most.
template <typename P, typename G, bool k8>
cudaError_t launch_all(const ftmoe_adamw_list& list, const AdamwConstants& c, cudaStream_t st) {
  for (int from = 0; from < list.count;) {
    int to = from, taken = 0;
    int64_t units = 0;
    while (to < list.count && taken < kMany) {
      const int64_t n = list.tensors[to].n, more = cdiv(n, kUnit);
      if (taken > 0 && units + more > ((int64_t)1 << 30)) break;
      units += more;
      taken += n > 0;
      ++to;
    }
    const cudaError_t e = taken <= kFew ? launch_some<P, G, k8, kFew>(list, from, to, c, st)
                                        : launch_some<P, G, k8, kMany>(list, from, to, c, st);
    if (e != cudaSuccess) return e;
    from = to;
  }
  return cudaSuccess;
}

}  // namespace adamw

cudaError_t launch_adamw(const ftmoe_adamw_list& list, const AdamwConstants& c, cudaStream_t st) {
  using namespace adamw;
  OverlapLaunch overlap;
  return with_elem(list.param_dtype, [&](auto p) {
    return with_elem(list.grad_dtype, [&](auto g) {
      using P = decltype(p);
      using G = decltype(g);
      return list.moments == FTMOE_MOMENTS_8BIT ? launch_all<P, G, true>(list, c, st) : launch_all<P, G, false>(list, c, st);
    });
  });
}

}  // namespace ftmoe
