// Element access by ftmoe_out_dtype for the training kernels: eight consecutive elements of a
// bf16, fp16 or fp32 row as fp32 values, in one or two vector accesses where the caller has
// checked the alignment, else one by one up to a given count.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace ftmoe {

struct ElemBf16 {
  using T = uint16_t;
  static __device__ __forceinline__ float get(uint16_t b) { return bf16_bits_to_f(b); }
  static __device__ __forceinline__ uint16_t put(float v) { return OutBf16::cvt(v); }
};
struct ElemF16 {
  using T = uint16_t;
  static __device__ __forceinline__ float get(uint16_t b) { return __half2float(__ushort_as_half(b)); }
  static __device__ __forceinline__ uint16_t put(float v) { return OutF16::cvt(v); }
};
struct ElemF32 {
  using T = float;
  static __device__ __forceinline__ float get(float b) { return b; }
  static __device__ __forceinline__ float put(float v) { return v; }
};

// eight elements as they lie in memory
template <typename Elem>
struct Raw8 {
  uint4 w[sizeof(typename Elem::T) / 2];
};

// n (at most 8) elements at p, the rest zero
template <typename Elem>
__device__ __forceinline__ Raw8<Elem> raw_load8(const typename Elem::T* p, bool vec, int n) {
  Raw8<Elem> r;
  constexpr int kV = sizeof(typename Elem::T) / 2;
  if (vec && n >= 8) {
#pragma unroll
    for (int i = 0; i < kV; ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if constexpr (kV == 1) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? __float_as_uint(p[i]) : 0u;
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}

template <typename Elem>
__device__ __forceinline__ void raw_get8(const Raw8<Elem>& r, float (&v)[8]) {
  if constexpr (sizeof(typename Elem::T) == 2) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = Elem::get((uint16_t)(w[i] & 0xffffu));
      v[2 * i + 1] = Elem::get((uint16_t)(w[i] >> 16));
    }
  } else {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
}

// two values rounded to 16 bits, lo in the low half
template <typename Elem>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r = 0;
  if constexpr (std::is_same<Elem, ElemBf16>::value)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else if constexpr (std::is_same<Elem, ElemF16>::value)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// the first n (at most 8) of v, each rounded once
template <typename Elem>
__device__ __forceinline__ void elem_store8(typename Elem::T* p, bool vec, int n, const float (&v)[8]) {
  if (vec && n >= 8) {
    if constexpr (sizeof(typename Elem::T) == 2) {
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack2<Elem>(v[0], v[1]), pack2<Elem>(v[2], v[3]), pack2<Elem>(v[4], v[5]), pack2<Elem>(v[6], v[7]));
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = Elem::put(v[i]);
  }
}

// Pairs of fp32 values in one instruction (Blackwell's packed fp32 pipe): for kernels that run at
// the issue rate it halves their products and sums.
struct F32Pair {
  unsigned long long v;
  __device__ __forceinline__ F32Pair() {}
  __device__ __forceinline__ F32Pair(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ explicit F32Pair(float both) : F32Pair(both, both) {}
  __device__ __forceinline__ void get(float& lo, float& hi) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
};
__device__ __forceinline__ F32Pair operator*(F32Pair a, F32Pair b) {
  F32Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F32Pair fma2(F32Pair a, F32Pair b, F32Pair c) {
  F32Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// whether rows of `elem_bytes`-byte elements at base with stride ld may take 8-element vectors
// (16-byte accesses)
inline bool elem_vec_ok(const void* base, int64_t ld, int elem_bytes) {
  return (uintptr_t)base % 16 == 0 && (ld * elem_bytes) % 16 == 0;
}

// dtype -> element type, for host dispatch: f(ElemBf16{}) and so on
template <typename F>
inline cudaError_t with_elem(int32_t dtype, F f) {
  if (dtype == FTMOE_OUT_BF16) return f(ElemBf16{});
  if (dtype == FTMOE_OUT_FP16) return f(ElemF16{});
  return f(ElemF32{});
}

// 2^(b - 127) of an E8M0 scale byte (b = 0 gives the subnormal 2^-127; 255 is the format's NaN)
__device__ __forceinline__ float e8m0_to_f(uint8_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : (uint32_t)b << 23);
}

}  // namespace ftmoe
