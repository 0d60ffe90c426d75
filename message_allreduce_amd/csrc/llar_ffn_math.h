// llar_ffn_math.h -- element types, activations and their derivatives of the
// feed-forward kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "llar_ffn.h"

namespace llar_ffn {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct F32 {
  typedef float T;
  static constexpr int kind = 0;
  static __device__ __forceinline__ float to(float v) { return v; }
  static __device__ __forceinline__ float from(float v) { return v; }
};
struct F16 {
  typedef _Float16 T;
  static constexpr int kind = 1;
  static __device__ __forceinline__ float to(_Float16 v) { return (float)v; }
  static __device__ __forceinline__ _Float16 from(float v) { return (_Float16)v; }
};
struct BF16 {
  typedef __bf16 T;
  static constexpr int kind = 2;
  static __device__ __forceinline__ float to(__bf16 v) {
    return __builtin_bit_cast(float, (uint32_t)__builtin_bit_cast(uint16_t, v) << 16);
  }
  static __device__ __forceinline__ __bf16 from(float v) { return (__bf16)v; }
};

// n neighbouring values moved to or from memory: one access at the element's
// alignment (which the memory pipeline takes for any width), or at a row's end
// the `cnt` that exist one by one.
template <class E, int n>
struct Vals {
  float v[n];
};

template <class E, int n>
struct Wide {
  typedef typename E::T vec __attribute__((ext_vector_type(n)));
  typedef vec loose __attribute__((aligned(2)));
};

template <class E, int n>
__device__ __forceinline__ Vals<E, n> load_vals(const typename E::T* p, int cnt) {
  Vals<E, n> r;
  if (cnt >= n) {
    const typename Wide<E, n>::vec q = *(const typename Wide<E, n>::loose*)p;
#pragma unroll
    for (int i = 0; i < n; i++) r.v[i] = E::to(q[i]);
  } else {
#pragma unroll
    for (int i = 0; i < n; i++) r.v[i] = i < cnt ? E::to(p[i]) : 0.f;
  }
  return r;
}

template <class E, int n>
__device__ __forceinline__ void store_vals(typename E::T* p, const float* v, int cnt) {
  if (cnt >= n) {
    typename Wide<E, n>::vec q;
#pragma unroll
    for (int i = 0; i < n; i++) q[i] = E::from(v[i]);
    *(typename Wide<E, n>::loose*)p = q;
  } else {
#pragma unroll
    for (int i = 0; i < n; i++)
      if (i < cnt) p[i] = E::from(v[i]);
  }
}

// ---- activations ---------------------------------------------------------------------
// For 16-bit results the hardware's exponential and reciprocal do: the product's
// and the constant's rounding make the exponential off by up to |x| 2^-23.6, the
// instruction adds 2^-23, so below 2^-17 of it over binary32's range, against the
// result's own 2^-9 or 2^-12.  binary32 takes the library's.
template <class E>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (E::kind == 0) return expf(x);
  return __builtin_amdgcn_exp2f(x * 1.44269504f);
}
template <class E>
__device__ __forceinline__ float inverse(float x) {
  if constexpr (E::kind == 0) return 1.f / x;
  return __builtin_amdgcn_rcpf(x);
}
template <class E>
__device__ __forceinline__ float sigmoid(float t) {
  return inverse<E>(1.f + exp_of<E>(-t));
}

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// z s for a factor s that reaches 0 at z = -inf faster than z grows: the limit
// there is 0, where the plain product would be a NaN.
__device__ __forceinline__ float fading(float z, float s) { return s == 0.f ? 0.f : z * s; }

// Phi(z) and e = exp(-z^2 / 2), which the density shares.  For t = |z|,
// Phi(-t) exp(t^2 / 2) is a smooth function of s = 1 / (1 + 0.36 t): a minimax
// polynomial of degree 9 in s (fitted for this file over t = 0 .. 40) is within
// 9e-8 of it, relatively, so the tail keeps its digits.
template <class E>
__device__ __forceinline__ float normal(float z, float& e) {
  const float zz = z * z;
  const float rest = zz < 1e4f ? fmaf(z, z, -zz) : 0.f;  // what the square's rounding lost
  e = exp_of<E>(-0.5f * zz);
  e = fmaf(-0.5f * rest, e, e);
  const float s = inverse<E>(fmaf(0.36f, fabsf(z), 1.f));
  float p = -0.0302381665f;
  p = fmaf(p, s, 0.139508024f);
  p = fmaf(p, s, -0.223599017f);
  p = fmaf(p, s, 0.107368767f);
  p = fmaf(p, s, -0.000386219239f);
  p = fmaf(p, s, 0.0960373282f);
  p = fmaf(p, s, 0.124009758f);
  p = fmaf(p, s, 0.143681884f);
  p = fmaf(p, s, 0.14361766f);
  const float tail = e * (p * s);
  return z > 0.f ? 1.f - tail : tail;
}

// tanh(t) = 2 s(2t) - 1, so the tanh form of GELU is z s(2 w) with
// w = sqrt(2/pi) (z + 0.044715 z^3): no cancellation for negative z.
template <int act, class E>
__device__ __forceinline__ float act_one(float z) {
  if constexpr (act == kActRelu) return z < 0.f ? 0.f : z;  // keeps a NaN
  if constexpr (act == kActGelu) {
    float e;
    return fading(z, normal<E>(z, e));
  }
  if constexpr (act == kActGeluTanh) return fading(z, sigmoid<E>(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z)));
  if constexpr (act == kActSilu) return fading(z, sigmoid<E>(z));
  return z;
}

// The value and the derivative together: they share the exponential.
template <int act, class E>
__device__ __forceinline__ void act_two(float z, float& value, float& slope) {
  value = z;
  slope = 1.f;
  if constexpr (act == kActRelu) {
    value = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
  } else if constexpr (act == kActGelu) {
    float e;
    const float p = normal<E>(z, e);
    value = fading(z, p);
    slope = p + fading(z, kInvSqrt2Pi * e);
  } else if constexpr (act == kActGeluTanh) {
    const float s = sigmoid<E>(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
    value = fading(z, s);
    // s (1 - s) is 0 long before the square would overflow
    const float d = s * (1.f - s);
    slope = d == 0.f ? s : s + z * d * 2.f * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
  } else if constexpr (act == kActSilu) {
    const float s = sigmoid<E>(z);
    value = fading(z, s);
    slope = s + fading(z, s * (1.f - s));
  }
}

// Calls f with the activation as a constant.
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case kActRelu: return f(std::integral_constant<int, kActRelu>());
    case kActGelu: return f(std::integral_constant<int, kActGelu>());
    case kActGeluTanh: return f(std::integral_constant<int, kActGeluTanh>());
    case kActSilu: return f(std::integral_constant<int, kActSilu>());
    default: return f(std::integral_constant<int, kActNone>());
  }
}
template <class E, int n>
__device__ __forceinline__ void act_values(float (&y)[n], int act) {
  with_act(act, [&](auto c) {
#pragma unroll
    for (int i = 0; i < n; i++) y[i] = act_one<decltype(c)::value, E>(y[i]);
  });
}

}  // namespace llar_ffn
