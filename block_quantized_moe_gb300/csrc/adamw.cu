// An AdamW step over many tensors in one launch, moments in fp32 or in 8 bits.
//
//   g = grad_scale grad,  m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
//   p = p - (lr decay p + lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps))
// Elementwise: 24 bytes an element and the gradient with fp32 moments, 12 1/8 and the gradient with
// 8-bit ones (p 8, codes 4, scales 1/8), and 2 for a 16-bit copy. Memory bounds it. Measured on GB300,
// 939 M fp32 parameters with bf16 gradients and copies: 3.84 ms with fp32 moments (101% of the measured
// copy rate), 2.28 ms with 8-bit ones (98%; 52 instructions an element, 56% of the issue slots). The same in
// bf16 parameters without copies: 3.00 ms (102%), and 1.65 ms with 8-bit moments (85%: 10 bytes an element
// under the same instructions).
//
// 8-bit moments: per 32 elements a power of two, codes e4m3 (m) and e5m2 (v), stochastically rounded.
// With beta2 = 0.999 v moves by a thousandth of itself a step, far below half of e5m2's step: rounded
// to nearest it would never move. The value times the power that puts the format's least normal on
// fp32's least normal has the code's digits in the upper bits of the fp32 number, subnormal ones
// included, so that adding random bits below them and cutting those off is the rounding; the rest
// converts exactly. v's code is at least 1 where v > 0: a zero under a moment that is not zero would
// divide it by eps.
// The random bits: a hash per chunk of eight elements, multiplied out by eight odd constants (the
// halves of each 64-bit product combined); 16 bits for m, 16 for v. Constants: fractional parts of
// square roots of primes, made odd.
// The products and sums of m and v are rounded one by one (no fused multiply-add), which any fp32
// program can repeat bit for bit; the codes depend on it.
#include "common.cuh"
#include "elem16.cuh"
#include "many.cuh"

namespace ftmoe {

namespace adamw {

using many::kPasses;
using many::kThreads;
using many::kPass;

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

// tensors of a launch: kernel parameters of 4 KB, and of 31 KB for long lists
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

// the largest of the four lanes of a group
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
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
__device__ __forceinline__ void decode8(uint2 c, float scale, F32Pair (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = (i < 2 ? c.x : c.y) >> (16 * (i & 1));
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), kFormat)));
    v[i] = F32Pair(f.x, f.y) * F32Pair(scale);
  }
}

__device__ __forceinline__ float square_root(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// (of a number from eps to 2^126)
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// what a step needs of its constants
struct Step {
  float grad_scale, beta1, beta2, rest1, rest2, eps;
  float decay;       // lr * weight decay
  float rate;        // lr / (1 - beta1^t)
  float correction;  // 1 / sqrt(1 - beta2^t)
  float one;         // 1, which the compiler does not know: x * one + y is a sum that it cannot fuse with the product x
};

// the step on eight elements
__device__ __forceinline__ void update8(const Step& s, float (&p)[8], const float (&grad)[8], F32Pair (&m)[4], F32Pair (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F32Pair g = F32Pair(grad[2 * i], grad[2 * i + 1]) * F32Pair(s.grad_scale);
    m[i] = fma2(m[i] * F32Pair(s.beta1), F32Pair(s.one), g * F32Pair(s.rest1));
    v[i] = fma2(v[i] * F32Pair(s.beta2), F32Pair(s.one), g * g * F32Pair(s.rest2));
    float a, b;
    v[i].get(a, b);
    fma2(F32Pair(square_root(a), square_root(b)), F32Pair(s.correction), F32Pair(s.eps)).get(a, b);
    const F32Pair old(p[2 * i], p[2 * i + 1]);
    const F32Pair less = fma2(m[i] * F32Pair(reciprocal(a), reciprocal(b)), F32Pair(s.rate), old * F32Pair(s.decay));
    fma2(less, F32Pair(-1.0f), old).get(p[2 * i], p[2 * i + 1]);
  }
}

// Codes of eight elements' moments; the four lanes of a group call together. base: the chunk's hash.
__device__ __forceinline__ void encode8(const F32Pair (&m)[4], const F32Pair (&v)[4], uint32_t base, uint2& mc, uint2& vc,
                                        uint32_t& m_byte, uint32_t& v_byte) {
  float m_top = 0.0f, v_top = 0.0f;
  F32Pair zero(0.0f);  // NaN where an element is not finite
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    zero = fma2(m[i], F32Pair(0.0f), fma2(v[i], F32Pair(0.0f), zero));
    m[i].get(a, b);
    m_top = fmaxf(fmaxf(m_top, fabsf(a)), fabsf(b));
    v[i].get(a, b);
    v_top = fmaxf(fmaxf(v_top, a), b);
  }
  m_byte = scale_byte<8>(__float_as_uint(group_max(m_top)));
  v_byte = scale_byte<15>(__float_as_uint(group_max(v_top)));
  const F32Pair mf(inverse_scale(m_byte)), vf(inverse_scale(v_byte));
  uint32_t h[8];
  noise8(base, h);
  uint32_t mq[4], vq[4];  // two codes each
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b, va, vb;
    (m[i] * mf * F32Pair(0x1p-120f)).get(a, b);
    a = __uint_as_float((__float_as_uint(a) + ((h[2 * i] & 0xffffu) << 4)) & 0xfff00000u);
    b = __uint_as_float((__float_as_uint(b) + ((h[2 * i + 1] & 0xffffu) << 4)) & 0xfff00000u);
    (F32Pair(a, b) * F32Pair(0x1p120f)).get(a, b);
    mq[i] = f2_to_e4m3x2(a, b);
    (v[i] * vf * F32Pair(0x1p-112f)).get(a, b);
    v[i].get(va, vb);
    uint32_t x = (__float_as_uint(a) + ((h[2 * i] >> 16) << 5)) & 0xffe00000u;
    uint32_t y = (__float_as_uint(b) + ((h[2 * i + 1] >> 16) << 5)) & 0xffe00000u;
    if (va > 0.0f) x = max(x, 0x00200000u);
    if (vb > 0.0f) y = max(y, 0x00200000u);
    (F32Pair(__uint_as_float(x), __uint_as_float(y)) * F32Pair(0x1p112f)).get(a, b);
    vq[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
  }
  mc = make_uint2(mq[0] | (mq[1] << 16), mq[2] | (mq[3] << 16));
  vc = make_uint2(vq[0] | (vq[1] << 16), vq[2] | (vq[3] << 16));
  float a, b;
  zero.get(a, b);
  if (!(a + b == 0.0f)) {  // (random bits make any number of a NaN)
    mc = make_uint2(0u, 0u);
    vc = make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[2], y[2];
      m[i].get(x[0], x[1]);
      v[i].get(y[0], y[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t sign = (__float_as_uint(x[j]) >> 24) & 0x80u;
        uint32_t mb = (mq[i] >> (8 * j)) & 0xffu, vb = (vq[i] >> (8 * j)) & 0xffu;
        if (!(fabsf(x[j]) < INFINITY)) mb = sign | (x[j] != x[j] ? 0x7fu : 0x7eu);
        if (!(y[j] < INFINITY)) vb = y[j] != y[j] ? 0x7fu : 0x7bu;
        (i < 2 ? mc.x : mc.y) |= mb << (16 * (i & 1) + 8 * j);
        (i < 2 ? vc.x : vc.y) |= vb << (16 * (i & 1) + 8 * j);
      }
    }
  }
}

// eight elements as they lie in memory
template <typename P, typename G, bool k8>
struct Chunk {
  Raw8<P> p;
  Raw8<G> g;
  Raw8<ElemF32> m, v;
  __device__ __forceinline__ void load(const Entry& t, int64_t at, bool vec, int n) {
    p = raw_load8<P>(static_cast<const typename P::T*>(t.param) + at, vec, n);
    g = raw_load8<G>(static_cast<const typename G::T*>(t.grad) + at, vec, n);
    m = raw_load8<ElemF32>(static_cast<const float*>(t.m) + at, vec, n);
    v = raw_load8<ElemF32>(static_cast<const float*>(t.v) + at, vec, n);
  }
  __device__ __forceinline__ void moments(F32Pair (&a)[4], F32Pair (&b)[4]) const {
    float x[8];
    raw_get8<ElemF32>(m, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = F32Pair(x[2 * i], x[2 * i + 1]);
    raw_get8<ElemF32>(v, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = F32Pair(x[2 * i], x[2 * i + 1]);
  }
};
template <typename P, typename G>
struct Chunk<P, G, true> {
  Raw8<P> p;
  Raw8<G> g;
  uint2 m, v;
  uint8_t m_byte, v_byte;
  __device__ __forceinline__ void load(const Entry& t, int64_t at, bool vec, int n) {
    p = raw_load8<P>(static_cast<const typename P::T*>(t.param) + at, vec, n);
    g = raw_load8<G>(static_cast<const typename G::T*>(t.grad) + at, vec, n);
    m = load_codes(static_cast<const uint8_t*>(t.m) + at, vec, n);
    v = load_codes(static_cast<const uint8_t*>(t.v) + at, vec, n);
    m_byte = n > 0 ? t.m_scales[at >> 5] : (uint8_t)0;
    v_byte = n > 0 ? t.v_scales[at >> 5] : (uint8_t)0;
  }
  __device__ __forceinline__ void moments(F32Pair (&a)[4], F32Pair (&b)[4]) const {
    decode8<__NV_E4M3>(m, e8m0_to_f(m_byte), a);
    decode8<__NV_E5M2>(v, e8m0_to_f(v_byte), b);
  }
};

template <typename P, typename G, bool k8>
__device__ __forceinline__ void step8(const Step& s, const Entry& t, const Chunk<P, G, k8>& c, int64_t at, bool vec, int n,
                                      uint32_t key, int copy_dtype) {
  float p[8], g[8];
  F32Pair m[4], v[4];
  raw_get8<P>(c.p, p);
  raw_get8<G>(c.g, g);
  c.moments(m, v);
  update8(s, p, g, m, v);
  elem_store8<P>(static_cast<typename P::T*>(t.param) + at, vec, n, p);
  if constexpr (sizeof(typename P::T) == 2) {  // the copy is of the parameter as it is kept
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = P::get(P::put(p[i]));
  }
  if (copy_dtype == FTMOE_OUT_BF16) elem_store8<ElemBf16>(static_cast<uint16_t*>(t.copy) + at, vec, n, p);
  else if (copy_dtype == FTMOE_OUT_FP16) elem_store8<ElemF16>(static_cast<uint16_t*>(t.copy) + at, vec, n, p);
  if constexpr (k8) {
    uint2 mc, vc;
    uint32_t m_byte, v_byte;
    encode8(m, v, mix(key + (uint32_t)(at >> 3)), mc, vc, m_byte, v_byte);
    store_codes(static_cast<uint8_t*>(t.m) + at, vec, n, mc);
    store_codes(static_cast<uint8_t*>(t.v) + at, vec, n, vc);
    if ((threadIdx.x & 3) == 0 && n > 0) {
      t.m_scales[at >> 5] = (uint8_t)m_byte;
      t.v_scales[at >> 5] = (uint8_t)v_byte;
    }
  } else {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i].get(x[2 * i], x[2 * i + 1]);
    elem_store8<ElemF32>(static_cast<float*>(t.m) + at, vec, n, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i].get(x[2 * i], x[2 * i + 1]);
    elem_store8<ElemF32>(static_cast<float*>(t.v) + at, vec, n, x);
  }
}

template <typename P, typename G, bool k8, int kMax>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ many::Table<Entry, kMax> table,
                                                         const AdamwConstants c, const int copy_dtype, const int passes) {
  pdl_wait();
  pdl_trigger();
  const int which = table.find(blockIdx.x);
  const Entry t = table.entry[which];
  const int64_t start = (int64_t)((int)blockIdx.x - table.first[which]) * (passes * kPass);

  Step s = {c.grad_scale != nullptr ? *c.grad_scale : 1.0f, c.beta1, c.beta2, c.rest1, c.rest2, c.eps};
  if (!(fabsf(s.grad_scale) < INFINITY)) return;  // no step
  const float lr = c.lr_dev != nullptr ? *c.lr_dev : c.lr;
  float correction1 = c.correction1;
  s.correction = c.correction2;
  int64_t step = c.step;
  if (c.step_dev != nullptr) {
    step = max(*c.step_dev, (int64_t)1);
    correction1 = -1.0f / expm1f((float)step * c.ln_beta1);
    s.correction = rsqrtf(-expm1f((float)step * c.ln_beta2));
  }
  s.decay = lr * c.weight_decay;
  s.rate = lr * correction1;
  s.one = c.one;
  uint32_t key = 0;
  if constexpr (k8) {
    key = mix(mix(mix(c.seed) + (uint32_t)step) + (uint32_t)t.index);
    key = mix(key + (uint32_t)((uint64_t)(start >> 3) >> 32));
  }

  const int64_t first = start + (int64_t)threadIdx.x * 8;
  if constexpr (k8) {
    if (passes == kPasses && t.vec && start + kPasses * kPass <= t.n) {
      // whole vectors: the next chunk is on its way while this one is worked on (with fp32 moments a chunk
      // is up to 32 registers, and enough warps fit to do without: unrolled like this they lose 6%)
      Chunk<P, G, true> now, next;
      now.load(t, first, true, 8);
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        const int64_t at = first + pass * kPass;
        if (pass + 1 < kPasses) next.load(t, at + kPass, true, 8);
        step8<P, G, true>(s, t, now, at, true, 8, key, copy_dtype);
        now = next;
      }
      return;
    }
  }
#pragma unroll 1
  for (int pass = 0; pass < passes; ++pass) {
    const int64_t at = first + pass * kPass, left = t.n - at;
    // (lanes past the end stay for the exchange between the four lanes of a group; their elements are zeros)
    if (__all_sync(0xffffffffu, left <= 0)) break;
    const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
    Chunk<P, G, k8> now;
    now.load(t, at, t.vec != 0, n);
    step8<P, G, k8>(s, t, now, at, t.vec != 0, n, key, copy_dtype);
  }
}

template <typename P, typename G, bool k8, int kMax>
cudaError_t launch_some(const ftmoe_adamw_list& list, int from, int to, int passes, const AdamwConstants& c, cudaStream_t st) {
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
    units += (int)cdiv(t.n, passes * kPass);
  }
  table.first[table.count] = units;
  return launch_kernel(adamw_kernel<P, G, k8, kMax>, dim3((unsigned)units), dim3(kThreads), 0, st, true, table, c,
                       (int)list.copy_dtype, passes);
}

// A launch takes kMany tensors (kFew where that is all of them) and 2^30 units at most.
template <typename P, typename G, bool k8>
cudaError_t launch_all(const ftmoe_adamw_list& list, const AdamwConstants& c, cudaStream_t st) {
  return many::for_launches(list.count, kMany, [&](int i) { return list.tensors[i].n; },
                            [&](int from, int to, int taken, int passes) {
                              return taken <= kFew ? launch_some<P, G, k8, kFew>(list, from, to, passes, c, st)
                                                   : launch_some<P, G, k8, kMany>(list, from, to, passes, c, st);
                            });
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
