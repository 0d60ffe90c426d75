// llar_chunk.h -- 16-row products whose weights go from memory straight to the
// matrix units' operand registers, for any type of operand: what the 8-bit and the
// experts' kernels for few tokens share.
//
// A chunk is a lane's 16 bytes of a fragment: 16 rows of 64 bytes, lane l holds
// bytes 16 (l / 16) .. + 15 of row l % 16.  That is a whole matrix instruction's
// operand for 8- and 16-bit numbers and four of them for binary32, whose own
// instruction keeps infinities where they are; the order of k within 64 bytes is
// the same for both operands and so does not matter.
#pragma once
#include "llar_gemm.h"

namespace llar_ffn {

typedef u32x4 __attribute__((aligned(1))) any_u32x4;

template <class E>
struct Chunk {
  static constexpr int ES = sizeof(typename E::X), CE = 16 / ES;
  u32x4 v;
  __device__ __forceinline__ void zero() { v = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void load(const char* p) { v = *(const any_u32x4*)p; }
  // `left` elements of a row of K exist from here on, none if it is not positive.
  // The row's last chunk is read as its last 16 bytes (fetch), and moved down (settle).
  __device__ __forceinline__ void fetch(const char* p, int64_t left, int K) {
    if (K >= CE) {
      load(p - (left >= CE ? 0 : (CE - left) * ES));
      return;
    }
    union {
      u32x4 v;
      uint64_t d[2];
    } u;
    u.v = u32x4{0u, 0u, 0u, 0u};
#pragma clang loop unroll(disable)
    for (int i = 0; i < (int)left * ES; i++) {
      const uint64_t byte = ((const uint8_t*)p)[i];
      if (i < 8)
        u.d[0] |= byte << 8 * i;
      else
        u.d[1] |= byte << 8 * (i - 8);
    }
    v = u.v;
  }
  __device__ __forceinline__ void settle(int64_t left, int K) {
    if (left >= CE || K < CE) return;
    union {
      u32x4 v;
      uint64_t d[2];
    } u;
    u.v = v;
    const int bits = left <= 0 ? 128 : (CE - (int)left) * ES * 8;
    if (bits >= 64) {
      u.d[0] = bits < 128 ? u.d[1] >> (bits - 64) : 0;
      u.d[1] = 0;
    } else {
      u.d[0] = u.d[0] >> bits | u.d[1] << (64 - bits);
      u.d[1] >>= bits;
    }
    v = u.v;
  }
  __device__ __forceinline__ void load(const char* p, int64_t left, int K) {
    fetch(p, left, K);
    settle(left, K);
  }
  // rows in LDS are aligned, and zeros follow them up to a whole step
  __device__ __forceinline__ void load(const lds_char* p) { v = *(const LLAR_LDS u32x4*)p; }
  __device__ __forceinline__ void load(const lds_char* p, int64_t, int) { load(p); }
};

template <class E>
__device__ __forceinline__ f32x4 mma_chunk(const Chunk<E>& a, const Chunk<E>& b, f32x4 c) {
  if constexpr (E::kParts) {
#pragma unroll
    for (int i = 0; i < 4; i++)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[i]), __uint_as_float(b.v[i]), c, 0, 0, 0);
    return c;
  } else {
    return mma<E>(Frag<E>{__builtin_bit_cast(s16x8, a.v)}, Frag<E>{__builtin_bit_cast(s16x8, b.v)}, c);
  }
}

// A sum's bits, of an integer for 8-bit operands, added to another's.
template <class E>
__device__ __forceinline__ float add_sums(float a, float b) {
  if constexpr (E::kInt8) return __int_as_float(__float_as_int(a) + __float_as_int(b));
  return a + b;
}

// P planes of 16 weight rows times NB blocks of 16 rows of x, over the steps
// i0, i0 + stride, ... below i1 of k: a step is 64 G bytes of a row, G chunks a
// lane.  w and x point at the lane's first chunk of step 0 (16 G q bytes into the
// row); a row of x that is not live counts as zeros and is not read.  U steps'
// loads are in flight.  x may lie in LDS.  acc[p][b], lane (r, q): row 16 b + r of x, weight rows 4 q
// .. 4 q + 3 of plane p.
template <class E, int P, int NB, int G, int U, class X>
__device__ __forceinline__ void multiply_steps(f32x4 (&acc)[P][NB], const char* const (&w)[P], X* const (&x)[NB],
                                               const bool (&live)[NB], int K, int i0, int i1, int stride) {
  typedef Chunk<E> C;
  constexpr int kStep = 4 * C::CE * G;  // elements
  const int q = (threadIdx.x & 63) >> 4;
  const int full = min(i1, K / kStep);
  int i = i0;
#pragma clang loop unroll(disable)
  for (; i + (U - 1) * stride < full; i += U * stride) {
    C wv[U][P][G], xv[U][NB][G];
#pragma unroll
    for (int s = 0; s < U; s++)
#pragma unroll
      for (int p = 0; p < P; p++)
#pragma unroll
        for (int g = 0; g < G; g++) wv[s][p][g].load(w[p] + (int64_t)(i + s * stride) * (64 * G) + g * 16);
#pragma unroll
    for (int s = 0; s < U; s++)
#pragma unroll
      for (int b = 0; b < NB; b++)
#pragma unroll
        for (int g = 0; g < G; g++) {
          xv[s][b][g].zero();
          if (live[b]) xv[s][b][g].load(x[b] + (int64_t)(i + s * stride) * (64 * G) + g * 16);
        }
#pragma unroll
    for (int s = 0; s < U; s++)
#pragma unroll
      for (int g = 0; g < G; g++)
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
          for (int b = 0; b < NB; b++) acc[p][b] = mma_chunk<E>(wv[s][p][g], xv[s][b][g], acc[p][b]);
  }
#pragma clang loop unroll(disable)
  for (; i < i1; i += stride) {
    C wv[P][G], xv[NB][G];
#pragma unroll
    for (int g = 0; g < G; g++) {
      const int64_t left = K - (int64_t)i * kStep - (q * G + g) * C::CE;
#pragma unroll
      for (int p = 0; p < P; p++) wv[p][g].load(w[p] + (int64_t)i * (64 * G) + g * 16, left, K);
#pragma unroll
      for (int b = 0; b < NB; b++) {
        xv[b][g].zero();
        if (live[b]) xv[b][g].load(x[b] + (int64_t)i * (64 * G) + g * 16, left, K);
      }
    }
#pragma unroll
    for (int g = 0; g < G; g++)
#pragma unroll
      for (int p = 0; p < P; p++)
#pragma unroll
        for (int b = 0; b < NB; b++) acc[p][b] = mma_chunk<E>(wv[p][g], xv[b][g], acc[p][b]);
  }
}

template <class E, int P, int NB>
__device__ __forceinline__ void clear(f32x4 (&acc)[P][NB]) {
#pragma unroll
  for (int p = 0; p < P; p++)
#pragma unroll
    for (int b = 0; b < NB; b++) acc[p][b] = f32x4{0.f, 0.f, 0.f, 0.f};  // an integer's zeros too
}

// ---- rows of whole numbers -----------------------------------------------------------
// q = x / scale rounded to the nearest, ties to even, where scale is the row's
// largest magnitude / 127.  The product with the reciprocal can be off by one next
// to a half; the remainder x - q scale is exact in binary32 (it is a multiple of
// half of scale's last bit and at most about half of scale), and decides: a lane
// with a remainder of half of scale or more among its eight looks at each of them.
struct Quantizer {
  float scale, inv, unit, half, lift;
  bool plain;
  // top: the largest magnitude's bits, a NaN above infinity
  __device__ __forceinline__ explicit Quantizer(uint32_t top) {
    const float t = __uint_as_float(top);
    scale = top >= 0x7f800000u ? __builtin_nanf("") : t / 127.f;
    // tiny rows are lifted, so that the reciprocal exists
    plain = scale >= 0x1p-90f;
    lift = plain ? 1.f : 0x1p60f;
    unit = scale * lift;
    inv = unit > 0.f ? 1.f / unit : 0.f;  // a row of zeros, or with a NaN: zeros
    half = 0.5f * unit;
  }
  __device__ __forceinline__ int one(float x) const {
    if (!(inv > 0.f)) return 0;
    x *= lift;
    float r = rintf(x * inv);
    const float d = fmaf(-r, unit, x), m = fabsf(d);
    const bool odd = (int)r & 1;
    if (m > half || (m == half && odd)) r += d > 0.f ? 1.f : -1.f;
    return (int)fminf(fmaxf(r, -127.f), 127.f);  // a tiny row's scale is not exact enough
  }
  // eight bytes
  __device__ __forceinline__ uint2 eight(const float (&x)[8]) const {
    // 1.5 x 2^23 + n has n in its low bits, rounded by the addition
    constexpr float kShift = 12582912.f;
    float y[8], worst = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      y[i] = fmaf(x[i], inv, kShift);
      worst = fmaxf(worst, fabsf(fmaf(-(y[i] - kShift), unit, x[i])));
    }
    if (!plain || worst >= half) {
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = __int_as_float(one(x[i]));
    }
    return make_uint2(pack4(y), pack4(y + 4));
  }
  // the low bytes of four words
  static __device__ __forceinline__ uint32_t pack4(const float* y) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(y[1]), __float_as_uint(y[0]), 0x0c0c0400);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(y[3]), __float_as_uint(y[2]), 0x04000c0c);
    return lo | hi;
  }
};
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
template <class E>
__device__ __forceinline__ uint32_t magnitude(const Vals<E, 8>& v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) top = max(top, magnitude(v.v[i]));
  return top;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

}  // namespace llar_ffn
