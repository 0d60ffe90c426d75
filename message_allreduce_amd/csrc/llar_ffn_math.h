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

// n values held in registers moved to or from memory: one wide access where
// the caller says the address allows it, else element by element up to `cnt`.
template <class E, int n>
struct Vals {
  float v[n];
};

template <class E, int n>
__device__ __forceinline__ Vals<E, n> load_vals(const typename E::T* p, int cnt, bool vec) {
  typedef typename E::T T;
  typedef T Vec __attribute__((ext_vector_type(n)));
  Vals<E, n> r;
  if (vec && cnt >= n) {
    Vec q = *(const Vec*)p;
#pragma unroll
    for (int i = 0; i < n; i++) r.v[i] = E::to(q[i]);
  } else {
#pragma unroll
    for (int i = 0; i < n; i++) r.v[i] = i < cnt ? E::to(p[i]) : 0.f;
  }
  return r;
}

template <class E, int n>
__device__ __forceinline__ void store_vals(typename E::T* p, const float* v, int cnt, bool vec) {
  typedef typename E::T T;
  typedef T Vec __attribute__((ext_vector_type(n)));
  if (vec && cnt >= n) {
    Vec q;
#pragma unroll
    for (int i = 0; i < n; i++) q[i] = E::from(v[i]);
    *(Vec*)p = q;
  } else {
#pragma unroll
    for (int i = 0; i < n; i++)
      if (i < cnt) p[i] = E::from(v[i]);
  }
}

// tanh(t) = 2 s(2t) - 1, so the tanh form of GELU is z s(2 w) with
// w = sqrt(2/pi) (z + 0.044715 z^3): no cancellation for negative z.
__device__ __forceinline__ float sigmoid(float t) { return 1.f / (1.f + expf(-t)); }

constexpr float kSqrt2OverPi = 0.7978845608028654f;
constexpr float kGeluCubic = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// z s for a factor s that reaches 0 at z = -inf faster than z grows: the limit
// there is 0, where the plain product would be a NaN.
__device__ __forceinline__ float fading(float z, float s) { return s == 0.f ? 0.f : z * s; }

template <int act>
__device__ __forceinline__ float act_one(float z) {
  if constexpr (act == kActRelu) return z < 0.f ? 0.f : z;  // keeps a NaN
  if constexpr (act == kActGelu) return fading(z, 0.5f * erfcf(-z * kSqrtHalf));
  if constexpr (act == kActGeluTanh) return fading(z, sigmoid(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z)));
  if constexpr (act == kActSilu) return fading(z, sigmoid(z));
  return z;
}

// The value and the derivative together: they share the exponential.
template <int act>
__device__ __forceinline__ void act_two(float z, float& value, float& slope) {
  value = z;
  slope = 1.f;
  if constexpr (act == kActRelu) {
    value = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
  } else if constexpr (act == kActGelu) {
    const float p = 0.5f * erfcf(-z * kSqrtHalf);
    value = fading(z, p);
    slope = p + fading(z, kInvSqrt2Pi * expf(-0.5f * z * z));
  } else if constexpr (act == kActGeluTanh) {
    const float s = sigmoid(2.f * kSqrt2OverPi * (z + kGeluCubic * z * z * z));
    value = fading(z, s);
    // s (1 - s) is 0 long before the square would overflow
    const float d = s * (1.f - s);
    slope = d == 0.f ? s : s + z * d * 2.f * kSqrt2OverPi * (1.f + 3.f * kGeluCubic * z * z);
  } else if constexpr (act == kActSilu) {
    const float s = sigmoid(z);
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
template <int n>
__device__ __forceinline__ void act_values(float (&y)[n], int act) {
  with_act(act, [&](auto c) {
#pragma unroll
    for (int i = 0; i < n; i++) y[i] = act_one<decltype(c)::value>(y[i]);
  });
}

}  // namespace llar_ffn
