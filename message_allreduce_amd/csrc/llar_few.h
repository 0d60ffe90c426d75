// llar_few.h -- products with at most 16 rows of x: decoding.  Bound by reading
// the weights once, so they go from memory straight to the matrix units'
// operand registers; no LDS tile, no barrier until the waves' sums are joined.
#pragma once
#include "llar_gemm.h"

namespace llar_ffn {

// 8 consecutive k of one row as a fragment lane's share; `left` of them exist
// (8 or more: all), read at the element's alignment.
template <class E>
struct Eight {
  typedef typename E::T T;
  typedef u32x4 __attribute__((aligned(2))) loose;
  u32x4 v[sizeof(T) / 2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) v[i] = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) v[i] = ((const loose*)p)[i];
  }
  __device__ __forceinline__ void load(const T* p, int64_t left) {
    if (left >= 8) {
      load(p);
      return;
    }
    union {
      T t[8];
      u32x4 q[sizeof(T) / 2];
    } u;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) u.q[i] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < left) u.t[i] = p[i];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) v[i] = u.q[i];
  }
  __device__ __forceinline__ Frag<E> frag() const;
  __device__ __forceinline__ void values(float (&f)[8]) const {
    union {
      T t[8];
      u32x4 q[sizeof(T) / 2];
    } u;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) u.q[i] = v[i];
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] = E::to(u.t[i]);
  }
};
template <>
__device__ __forceinline__ Frag<F16> Eight<F16>::frag() const {
  return Frag<F16>{__builtin_bit_cast(s16x8, v[0])};
}
template <>
__device__ __forceinline__ Frag<BF16> Eight<BF16>::frag() const {
  return Frag<BF16>{__builtin_bit_cast(s16x8, v[0])};
}
template <>
__device__ __forceinline__ Frag<F32> Eight<F32>::frag() const {
  const f32x4 a = __builtin_bit_cast(f32x4, v[0]), b = __builtin_bit_cast(f32x4, v[1]);
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return split3(x);
}

// The waves' sums of kOut outputs ([m][n of the workgroup], planes apart) are
// joined in LDS and finished, one output a thread.
template <class E, bool kXRows, bool kWRows, bool kGated, int kWaves, int kN>
__device__ __forceinline__ void few_finish(const GemmArgs& a, const float* part, int n0, int split, int64_t k0,
                                           int64_t k1) {
  constexpr int P = kGated ? 2 : 1;
  __syncthreads();
  for (int i = threadIdx.x; i < a.M * kN; i += kWaves * 64) {
    const int m = i / kN, n = i % kN;
    if (n0 + n >= a.N) continue;
    float v[P];
#pragma unroll
    for (int p = 0; p < P; p++) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; w++) s += part[((w * P + p) * 16 + m) * kN + n];
      if constexpr (E::kind == 0) {
        if (not_finite(s)) s = sum_again<kXRows, kWRows>(a, 0, p, m, n0 + n, k0, k1);
      }
      v[p] = s;
    }
    if (a.splits > 1) {
#pragma unroll
      for (int p = 0; p < P; p++)
        a.partial[(((int64_t)split * P + p) * a.M + m) * a.npad + n0 + n] = v[p];
    } else {
      finish<E, kGated, 1>(a, 0, m, n0 + n, &v[0], &v[P - 1]);
    }
  }
}

// Weights contiguous along k.  A wave multiplies 16 weight rows (gated: 8 of
// each projection) by all rows of x; a row's four lanes read 128 consecutive
// bytes a step, and the workgroup's waves take the steps in turn.  16 waves of
// two steps in flight: 8192 x 3584 bf16 with cold weights 19.4 us at 16 rows (3.0
// TB/s) and 14.8 at 4; 8 waves of four steps took 20.1 and 16.
template <class E, bool kGated, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void k_few_k(GemmArgs a) {
  typedef typename E::T T;
  constexpr int kN = kGated ? 8 : 16;
  constexpr int G = sizeof(T) == 2 ? 2 : 1;  // fragments of a step
  constexpr int kStep = 32 * G;
  constexpr int U = 2;                       // steps in flight
  __shared__ float part[kWaves * 16 * 16];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kN;
  const int row = min(n0 + (kGated ? r & 7 : r), a.N - 1);
  const bool live = r < a.M;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int seg = 0; seg < a.segs; seg++) {
    const T* w = (const T*)a.w[kGated ? r >> 3 : seg] + row * a.wld + q * (8 * G);
    const T* x = (const T*)a.x[seg] + (live ? r : 0) * a.xld + q * (8 * G);
    const int full = a.K / kStep;
    int i = wave;
    for (; i + (U - 1) * kWaves < full; i += U * kWaves) {
      Eight<E> wv[U][G], xv[U][G];
#pragma unroll
      for (int s = 0; s < U; s++)
#pragma unroll
        for (int g = 0; g < G; g++) wv[s][g].load(w + (int64_t)(i + s * kWaves) * kStep + g * 8);
#pragma unroll
      for (int s = 0; s < U; s++)
#pragma unroll
        for (int g = 0; g < G; g++) {
          xv[s][g].zero();
          if (live) xv[s][g].load(x + (int64_t)(i + s * kWaves) * kStep + g * 8);
        }
#pragma unroll
      for (int s = 0; s < U; s++)
#pragma unroll
        for (int g = 0; g < G; g++) acc = mma<E>(wv[s][g].frag(), xv[s][g].frag(), acc);
    }
    for (; i * kStep < a.K; i += kWaves) {
      const int64_t k = (int64_t)i * kStep;
      Eight<E> wv[G], xv[G];
#pragma unroll
      for (int g = 0; g < G; g++) {
        const int64_t left = a.K - k - q * (8 * G) - g * 8;
        wv[g].load(w + k + g * 8, left);
        xv[g].zero();
        if (live) xv[g].load(x + k + g * 8, left);
      }
#pragma unroll
      for (int g = 0; g < G; g++) acc = mma<E>(wv[g].frag(), xv[g].frag(), acc);
    }
  }
  // lane: row r of x, weight rows 4 q + i
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int n = 4 * q + i;
    if constexpr (kGated)
      part[((wave * 2 + (n >> 3)) * 16 + r) * 8 + (n & 7)] = acc[i];
    else
      part[(wave * 16 + r) * 16 + n] = acc[i];
  }
  few_finish<E, false, false, kGated, kWaves, kN>(a, part, n0, 0, 0, (int64_t)a.K * a.segs);
}

// One or two rows of x and weights contiguous along k: a wave takes two weight
// rows (gated: one of each projection) over all of k, a step of 512 consecutive
// k at a time; no other wave is needed for its sums.  Whole lines a load: cold
// weights at one row, bf16, against the kernel above: gated 2 x 3584 x 8192 24.0
// against 25.5 us (4.9 TB/s), 8192 x 3584 13.5 against 14.1, 28672 x 8192 82
// against 85 (5.7 TB/s); two rows 14.0 against 14.2, four 19.1 against 14.8.
template <class E, bool kGated, int kRows>
__global__ __launch_bounds__(256) void k_few_dot(GemmArgs a) {
  typedef typename E::T T;
  constexpr int R = 2, kN = kGated ? 1 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kN;
  if (n0 >= a.N) return;
  float acc[R][kRows] = {};
  for (int seg = 0; seg < a.segs; seg++) {
    const T* w[R];
#pragma unroll
    for (int r = 0; r < R; r++)
      w[r] = (const T*)a.w[kGated ? r / kN : seg] + min(n0 + r % kN, (int64_t)a.N - 1) * a.wld;
    const T* x = (const T*)a.x[seg];
    auto step = [&](int64_t k, auto whole) {
      Eight<E> wv[R], xv[kRows];
      const int64_t left = a.K - k;
#pragma unroll
      for (int r = 0; r < R; r++) {
        if constexpr (decltype(whole)::value)
          wv[r].load(w[r] + k);
        else
          wv[r].load(w[r] + k, left);
      }
#pragma unroll
      for (int m = 0; m < kRows; m++) {
        xv[m].zero();
        if (m < a.M) {
          if constexpr (decltype(whole)::value)
            xv[m].load(x + m * a.xld + k);
          else
            xv[m].load(x + m * a.xld + k, left);
        }
      }
      float xf[kRows][8];
#pragma unroll
      for (int m = 0; m < kRows; m++) xv[m].values(xf[m]);
#pragma unroll
      for (int r = 0; r < R; r++) {
        float wf[8];
        wv[r].values(wf);
#pragma unroll
        for (int m = 0; m < kRows; m++)
#pragma unroll
          for (int e = 0; e < 8; e++) acc[r][m] = fmaf(wf[e], xf[m][e], acc[r][m]);
      }
    };
    int64_t k = lane * 8;
#pragma unroll 4
    for (; k + 512 <= a.K + lane * 8; k += 512) step(k, std::integral_constant<bool, true>());
    if (k < a.K) step(k, std::integral_constant<bool, false>());
  }
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int m = 0; m < kRows; m++)
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) acc[r][m] += __shfl_xor(acc[r][m], d);
  // every lane has every sum: lane n + kN m finishes output (m, n)
  const int n = lane % kN, mine = lane / kN;
  if (mine >= a.M || n0 + n >= a.N) return;
  float v[2] = {};
#pragma unroll
  for (int r = 0; r < R; r++)
#pragma unroll
    for (int m = 0; m < kRows; m++)
      if (r % kN == n && m == mine) v[r / kN] = acc[r][m];
  finish<E, kGated, 1>(a, 0, mine, (int)n0 + n, &v[0], &v[1]);
}

// Weights contiguous along n.  Lane (r, q) reads kC neighbouring columns of
// the 8 lines k = 8 q + t, which are 8 k of each of its columns: column j of
// every lane makes fragment j without leaving the lane's registers.  Eight waves
// and k split over up to 512 workgroups: cold weights bf16, 2 x 3584 x 8192 gated
// 34 us (3.4 TB/s), 8192 x 3584 20 us, 16 x 4096 x 4096 14 us, joins included;
// 16 waves on 256 workgroups took 42, 21 and 19.
template <class E, int kC>
struct Lines {
  typedef typename E::T T;
  T v[8][kC];
  __device__ __forceinline__ void load(const T* p, int64_t ld) {
    typedef T vec __attribute__((ext_vector_type(kC), aligned(sizeof(T))));
    typedef vec loose __attribute__((aligned(2)));
#pragma unroll
    for (int t = 0; t < 8; t++) {
      const vec l = *(const loose*)(p + t * ld);
#pragma unroll
      for (int j = 0; j < kC; j++) v[t][j] = l[j];
    }
  }
  __device__ __forceinline__ void load(const T* p, int64_t ld, int64_t lines, int cols) {
    if (lines >= 8 && cols >= kC) {
      load(p, ld);
      return;
    }
#pragma unroll
    for (int t = 0; t < 8; t++)
#pragma unroll
      for (int j = 0; j < kC; j++) v[t][j] = t < lines && j < cols ? p[t * ld + j] : (T)0.f;
  }
  __device__ __forceinline__ Frag<E> frag(int j) const {
    if constexpr (sizeof(T) == 2) {
      s16x8 f;
#pragma unroll
      for (int t = 0; t < 8; t++) f[t] = __builtin_bit_cast(short, v[t][j]);
      return Frag<E>{f};
    } else {
      const float x[8] = {v[0][j], v[1][j], v[2][j], v[3][j], v[4][j], v[5][j], v[6][j], v[7][j]};
      return split3(x);
    }
  }
};

template <class E, bool kGated, int kC, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void k_few_n(GemmArgs a) {
  typedef typename E::T T;
  constexpr int P = kGated ? 2 : 1;
  constexpr int kN = 16 * kC;
  __shared__ float part[kWaves * P * 16 * kN];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tn = (a.N + kN - 1) / kN;
  const int n0 = (int)(blockIdx.x % tn) * kN, split = blockIdx.x / tn;
  const int col = n0 + r * kC, cols = a.N - col;
  const bool live = r < a.M;
  // 32 lines of k a step; the splits take runs of steps, the waves steps in turn
  const int steps = (a.K + 31) / 32, all = steps * a.segs;
  const int s0 = (int)((int64_t)all * split / a.splits), s1 = (int)((int64_t)all * (split + 1) / a.splits);
  f32x4 acc[P][kC];
#pragma unroll
  for (int p = 0; p < P; p++)
#pragma unroll
    for (int j = 0; j < kC; j++) acc[p][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = s0 + wave; s < s1; s += kWaves) {
    const int seg = s >= steps ? 1 : 0;
    const int64_t k = (int64_t)(s - seg * steps) * 32 + q * 8;
    Eight<E> xv;
    xv.zero();
    if (live && k < a.K) xv.load((const T*)a.x[seg] + r * a.xld + k, a.K - k);
    const Frag<E> xf = xv.frag();
#pragma unroll
    for (int p = 0; p < P; p++) {
      Lines<E, kC> l;
      l.load((const T*)a.w[kGated ? p : seg] + k * a.wld + col, a.wld, a.K - k, cols);
#pragma unroll
      for (int j = 0; j < kC; j++) acc[p][j] = mma<E>(l.frag(j), xf, acc[p][j]);
    }
  }
#pragma unroll
  for (int p = 0; p < P; p++)
#pragma unroll
    for (int j = 0; j < kC; j++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        part[((wave * P + p) * 16 + r) * kN + (4 * q + i) * kC + j] = acc[p][j][i];
  auto k_of = [&](int s) { return (int64_t)(s / steps) * a.K + min((s % steps) * 32, a.K); };
  few_finish<E, false, true, kGated, kWaves, kN>(a, part, n0, split, a.K ? k_of(s0) : 0, a.K ? k_of(s1) : 0);
}

}  // namespace llar_ffn
