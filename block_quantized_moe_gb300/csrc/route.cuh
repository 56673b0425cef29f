// What routing and its gradient share: a token's logits by lanes of a warp, softmax statistics.
#pragma once

#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "elem16.cuh"
#include "internal.h"

namespace ftmoe {

namespace route {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// NaN and -inf take no part (-inf); +inf counts as the largest finite number
__device__ __forceinline__ float taken(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Scores for the order alone, by the hardware's exponential and reciprocal. exp(-x) is off by the
// argument's rounding (|x| 2^-23.6 of it) and 4 half steps of the exponential: s by s (1 - s) of that, at
// most 0.3 * 2^-24 + 2^-24, and by 3 * 2^-24 s of the sum's rounding and the reciprocal: under 2^-21.5.
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sigmoid_fast(float x) { return reciprocal(1.0f + exp2_fast(x * -kLog2e)); }

// a lane's logits as they lie in memory (-inf past the last expert), in pieces of up to 16 bytes
template <typename Elem, int kPer>
struct Row {
  using T = typename Elem::T;
  static constexpr int kBytes = kPer * (int)sizeof(T), kPiece = kBytes < 16 ? kBytes : 16;  // (the piece of one 16-bit logit: 2)
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  static constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : std::is_same<Elem, ElemBf16>::value ? 0xff80ff80u : 0xfc00fc00u;
  uint32_t raw[kWords];
  __device__ __forceinline__ Row() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) raw[i] = kNone;
  }
  // whether rows at base, ld elements apart, can be read in pieces
  static bool vec_ok(const void* base, int64_t ld, int E) {
    return (uintptr_t)base % kPiece == 0 && ld * (int64_t)sizeof(T) % kPiece == 0 && E * (int)sizeof(T) % kPiece == 0;
  }
  __device__ __forceinline__ void load(const T* row, int lane, int E, bool vec) {
    const int e0 = lane * kPer;
    if (vec) {
#pragma unroll
      for (int c = 0; c < kBytes / kPiece; ++c) {
        const T* from = row + e0 + c * (kPiece / (int)sizeof(T));
        if (e0 + c * (kPiece / (int)sizeof(T)) < E) {
          if constexpr (kPiece == 16) {
            const uint4 q = *reinterpret_cast<const uint4*>(from);
            raw[4 * c] = q.x, raw[4 * c + 1] = q.y, raw[4 * c + 2] = q.z, raw[4 * c + 3] = q.w;
          } else if constexpr (kPiece == 8) {
            const uint2 q = *reinterpret_cast<const uint2*>(from);
            raw[0] = q.x, raw[1] = q.y;
          } else if constexpr (kPiece == 4) {
            raw[0] = *reinterpret_cast<const uint32_t*>(from);
          } else {
            raw[0] = *reinterpret_cast<const uint16_t*>(from);
          }
        }
      }
    } else {
      const uint32_t* words = reinterpret_cast<const uint32_t*>(row);
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (e0 + j < E) raw[j] = words[e0 + j];
      } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (e0 + j < E) raw[j / 2] = (raw[j / 2] & (j % 2 ? 0x0000ffffu : 0xffff0000u)) | (uint32_t)row[e0 + j] << (16 * (j % 2));
      }
    }
  }
  __device__ __forceinline__ void get(float (&x)[kPer]) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if constexpr (sizeof(T) == 4) x[j] = __uint_as_float(raw[j]);
      else x[j] = Elem::get((uint16_t)(raw[j / 2] >> (16 * (j % 2))));
    }
  }
  // the logits as they take part: see taken(). (A token of finite numbers is left as it is: a product
  // and a vote in place of two comparisons a logit, which run at half the rate.)
  __device__ __forceinline__ void get_taken(float (&x)[kPer]) const {
    get(x);
    float zero = 0.0f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) zero = fmaf(x[j], 0.0f, zero);
    if (__any_sync(kFull, !(zero == 0.0f))) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[j] = taken(x[j]);
    }
  }
};

// largest logit of the row and the sum of exp(x - max) (softmax scores)
template <int kPer>
__device__ __forceinline__ void softmax_stats(const float (&x)[kPer], float& top, float& sum) {
  float m = x[0];
#pragma unroll
  for (int j = 1; j < kPer; ++j) m = fmaxf(m, x[j]);
  top = warp_top(m);
  float s = 0.0f;
  if (top > -INFINITY) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) s += exp2_fast((x[j] - top) * kLog2e);
  }
  sum = warp_sum(s);
}

// experts per lane: the smallest power of two that covers them
template <typename F>
inline cudaError_t with_per(int32_t E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace route

}  // namespace ftmoe
