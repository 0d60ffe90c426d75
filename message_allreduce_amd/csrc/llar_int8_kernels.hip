// llar_int8_kernels.hip -- rows of whole numbers, their products for few tokens and
// the join of a split one.  The tiled product is llar_gemm.h's.
#include "llar_chunk.h"
#include "llar_int8.h"

namespace llar_ffn {

// ---- quantisation ----------------------------------------------------------------------
// NT threads a row (a wave, or a workgroup), eight neighbours at a time; up to
// kKeep such pieces a thread stay in registers between the maximum and the
// rounding, longer rows are read twice.
constexpr int kKeep = 4;

template <class E, int NT>
__device__ __forceinline__ uint32_t row_max(uint32_t top, uint32_t* shared) {
  top = wave_max<64>(top);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; i++) top = max(top, shared[i]);
  }
  return top;
}

template <class E, int NT, bool kStrided>
__global__ __launch_bounds__(256) void k_quantize(QuantArgs a) {
  typedef typename E::T T;
  __shared__ uint32_t shared[4];
  const int t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * (256 / NT) + threadIdx.x / NT;
  if (row >= a.M) return;  // NT == 256: whole workgroups
  const T* x = (const T*)a.x + row * a.xld;
  auto fetch = [&](int col) {
    if constexpr (!kStrided) {
      return load_vals<E, 8>(x + col, a.K - col);
    } else {
      Vals<E, 8> v;
#pragma unroll
      for (int i = 0; i < 8; i++) v.v[i] = col + i < a.K ? E::to(x[(col + i) * a.xcs]) : 0.f;
      return v;
    }
  };
  Vals<E, 8> kept[kKeep];
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < kKeep; p++) {
    const int col = (p * NT + t) * 8;
    if (col < a.K) {
      kept[p] = fetch(col);
#pragma unroll
      for (int i = 0; i < 8; i++) top = max(top, magnitude(kept[p].v[i]));
    }
  }
  for (int col = (kKeep * NT + t) * 8; col < a.K; col += NT * 8) {
    const Vals<E, 8> v = fetch(col);
#pragma unroll
    for (int i = 0; i < 8; i++) top = max(top, magnitude(v.v[i]));
  }
  const Quantizer quantize(row_max<E, NT>(top, shared));
  if (t == 0) a.scale[row] = quantize.scale;
  int8_t* q = a.q + row * a.qld;
  auto put = [&](int col, const Vals<E, 8>& v) {
    int n[8];
#pragma unroll
    for (int i = 0; i < 8; i++) n[i] = quantize(v.v[i]);
    if (col + 8 <= a.qpad) {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      typedef u32x2 __attribute__((aligned(1))) any_u32x2;
      *(any_u32x2*)(q + col) = u32x2{pack4(n[0], n[1], n[2], n[3]), pack4(n[4], n[5], n[6], n[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (col + i < a.qpad) q[col + i] = (int8_t)n[i];
    }
  };
#pragma unroll
  for (int p = 0; p < kKeep; p++) {
    const int col = (p * NT + t) * 8;
    if (col < a.K) put(col, kept[p]);
  }
  for (int col = (kKeep * NT + t) * 8; col < a.K; col += NT * 8) put(col, fetch(col));
  // whole pieces end at a multiple of 8; the rest of the padding
  for (int col = (a.K + 7) / 8 * 8 + t; col < a.qpad; col += NT) q[col] = 0;
}

template <class E, bool kStrided>
hipError_t quantize(const QuantArgs& a, hipStream_t s) {
  // a wave a row where its registers hold the row
  const bool wave = a.K <= 64 * 8 * kKeep;
  const int64_t groups = wave ? (a.M + 3) / 4 : a.M;
  if (groups == 0) return hipSuccess;
  if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
  if (wave)
    k_quantize<E, 64, kStrided><<<dim3((uint32_t)groups), dim3(256), 0, s>>>(a);
  else
    k_quantize<E, 256, kStrided><<<dim3((uint32_t)groups), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_quantize(int kind, const QuantArgs& a, hipStream_t s) {
  if (a.xcs == 1)
    return kind == 0 ? quantize<F32, false>(a, s) : kind == 1 ? quantize<F16, false>(a, s) : quantize<BF16, false>(a, s);
  return kind == 0 ? quantize<F32, true>(a, s) : kind == 1 ? quantize<F16, true>(a, s) : quantize<BF16, true>(a, s);
}

// ---- aligned copies ----------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_pack8(Pack8Args a) {
  int i = 0;
  while (i + 1 < a.count && blockIdx.x >= a.first[i + 1]) i++;
  const int64_t groups = a.dld / 16;
  const int64_t id = (blockIdx.x - a.first[i]) * 256 + threadIdx.x;
  const int64_t line = id / groups;
  const int64_t at = (id - line * groups) * 16;
  if (line >= a.lines[i]) return;
  Chunk<Int8<F32>> c;
  c.load((const char*)a.src[i] + line * a.ld[i] + at, a.width - at);
  *(u32x4*)(a.dst[i] + line * a.dld + at) = c.v;
}
hipError_t launch_pack8(const Pack8Args& a, hipStream_t s) {
  const int64_t groups = a.first[a.count];
  if (groups == 0) return hipSuccess;
  if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
  k_pack8<<<dim3((uint32_t)groups), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

// ---- few rows ------------------------------------------------------------------------
// 16 weight rows (gated: 8 of each projection) a workgroup, its waves take the
// steps of k in turn.
template <class Out, bool kGated, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void k_few_int8(GemmArgs a) {
  typedef Int8<Out> E;
  constexpr int kN = kGated ? 8 : 16, G = 2;
  __shared__ int part[kWaves][16][16];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kN;
  const int row = min(n0 + (kGated ? r & 7 : r), a.N - 1);
  const char* w[1] = {(const char*)a.w[kGated ? r >> 3 : 0] + row * a.wld + q * (16 * G)};
  const bool live[1] = {r < a.M};
  const char* x[1] = {(const char*)a.x[0] + (live[0] ? r : 0) * a.xld + q * (16 * G)};
  f32x4 acc[1][1];
  clear<E>(acc);
  constexpr int kStep = 64 * G;
  multiply_steps<E, 1, 1, G, 2>(acc, w, x, live, a.K, wave, (a.K + kStep - 1) / kStep, kWaves);
#pragma unroll
  for (int i = 0; i < 4; i++) part[wave][r][4 * q + i] = __float_as_int(acc[0][0][i]);
  __syncthreads();
  for (int i = threadIdx.x; i < a.M * kN; i += kWaves * 64) {
    const int m = i / kN, n = i % kN;
    if (n0 + n >= a.N) continue;
    constexpr int P = kGated ? 2 : 1;
    float v[P];
#pragma unroll
    for (int p = 0; p < P; p++) {
      int sum = 0;
#pragma unroll
      for (int k = 0; k < kWaves; k++) sum += part[k][m][p * kN + n];
      v[p] = scaled(sum, a.xscale[m], a.wscale[p][n0 + n]);
    }
    finish<E, kGated, 1>(a, 0, m, n0 + n, &v[0], &v[P - 1]);
  }
}

template <class Out, bool kGated>
hipError_t few_int8(const GemmArgs& a, hipStream_t s) {
  constexpr int kN = kGated ? 8 : 16, kWaves = 16;
  const int64_t groups = ((int64_t)a.N + kN - 1) / kN;
  if (groups == 0 || a.M == 0) return hipSuccess;
  if (!launchable(groups, kWaves * 64)) return hipErrorInvalidConfiguration;
  k_few_int8<Out, kGated, kWaves><<<dim3((uint32_t)groups), dim3(kWaves * 64), 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_few_int8(int kind, bool gated, const GemmArgs& a, hipStream_t s) {
  if (kind == 0) return gated ? few_int8<F32, true>(a, s) : few_int8<F32, false>(a, s);
  if (kind == 1) return gated ? few_int8<F16, true>(a, s) : few_int8<F16, false>(a, s);
  return gated ? few_int8<BF16, true>(a, s) : few_int8<BF16, false>(a, s);
}

// ---- join ----------------------------------------------------------------------------
template <class Out, bool kGated>
__global__ __launch_bounds__(256) void k_join_int8(GemmArgs a) {
  constexpr int P = kGated ? 2 : 1;
  const int groups = (a.N + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = id / groups;
  const int col = (int)(id - m * groups) * 4;
  if (m >= a.M) return;
  float v[2][4] = {};
#pragma unroll
  for (int p = 0; p < P; p++) {
    const int* src = (const int*)a.partial + ((int64_t)p * a.M + m) * a.npad + col;
    const int64_t step = (int64_t)P * a.M * a.npad;
    i32x4 sum = {0, 0, 0, 0};
    for (int i = 0; i < a.splits; i++) sum += *(const i32x4*)(src + i * step);
#pragma unroll
    for (int e = 0; e < 4; e++) v[p][e] = col + e < a.N ? scaled(sum[e], a.xscale[m], a.wscale[p][col + e]) : 0.f;
  }
  finish<Int8<Out>, kGated, 4>(a, 0, (int)m, col, v[0], v[1]);
}

template <class Out>
hipError_t join_int8(bool gated, const GemmArgs& a, hipStream_t s) {
  const int64_t groups = ((int64_t)a.M * ((a.N + 3) / 4) + 255) / 256;
  if (groups == 0) return hipSuccess;
  if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
  if (gated)
    k_join_int8<Out, true><<<dim3((uint32_t)groups), dim3(256), 0, s>>>(a);
  else
    k_join_int8<Out, false><<<dim3((uint32_t)groups), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_join_int8(int kind, bool gated, const GemmArgs& a, hipStream_t s) {
  return kind == 0 ? join_int8<F32>(gated, a, s) : kind == 1 ? join_int8<F16>(gated, a, s) : join_int8<BF16>(gated, a, s);
}

#define LLAR_DECL(E) hipError_t launch_gemm_int8_##E(const GemmPlan&, const GemmArgs&, hipStream_t);
LLAR_DECL(F32) LLAR_DECL(F16) LLAR_DECL(BF16)

hipError_t launch_gemm_int8(const GemmPlan& p, const GemmArgs& a, hipStream_t s) {
  return p.kind == 0 ? launch_gemm_int8_F32(p, a, s) : p.kind == 1 ? launch_gemm_int8_F16(p, a, s) : launch_gemm_int8_BF16(p, a, s);
}

}  // namespace llar_ffn
