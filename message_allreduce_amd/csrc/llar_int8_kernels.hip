// llar_int8_kernels.hip -- rows of whole numbers, their products for few tokens and
// the join of a split one.  The tiled product is llar_gemm.h's.
#include <algorithm>

#include "llar_chunk.h"
#include "llar_int8.h"

namespace llar_ffn {

// ---- aligned copies --------------------------------------------------------------------
__device__ __forceinline__ void pack8_piece(const Pack8Args& a, int64_t group, int threads) {
  int i = 0;
  while (i + 1 < a.count && group >= a.first[i + 1]) i++;
  const int64_t pieces = a.dld / 16;
  const int64_t id = (group - a.first[i]) * threads + threadIdx.x;
  const int64_t line = id / pieces;
  const int64_t at = (id - line * pieces) * 16;
  if (line >= a.lines[i]) return;
  Chunk<Int8<F32>> c;
  c.load((const char*)a.src[i] + line * a.ld[i] + at, a.width - at, a.width);
  *(u32x4*)(a.dst[i] + line * a.dld + at) = c.v;
}
__global__ __launch_bounds__(kPack8Threads) void k_pack8(Pack8Args a) { pack8_piece(a, blockIdx.x, kPack8Threads); }
hipError_t launch_pack8(const Pack8Args& a, hipStream_t s) {
  const int64_t groups = a.first[a.count];
  if (groups == 0) return hipSuccess;
  if (!launchable(groups, kPack8Threads)) return hipErrorInvalidConfiguration;
  k_pack8<<<dim3((uint32_t)groups), dim3(kPack8Threads), 0, s>>>(a);
  return hipGetLastError();
}

// ---- quantisation ----------------------------------------------------------------------
// NT threads a row, eight neighbours at a time; up to kKeep such pieces a thread
// stay in registers between the maximum and the rounding, longer rows are read
// twice.  The copies that the product behind it needs go into the same launch.
// 4096 x 8192 bf16 22 us (4.6 TB/s), 16 x 8192 3 to 4.  Columns apart (a transposed
// view) are read one by one, through the caches: 166 us; a workgroup that walks 32 rows
// abreast took 182, and 54 instead of 7 at 64 rows.
template <int NT>
constexpr int kQuantThreads = NT < 256 ? 256 : NT;

template <class E, int NT, int kKeep, bool kStrided>
__global__ __launch_bounds__(kQuantThreads<NT>) void k_quantize(QuantArgs a, Pack8Args copies) {
  typedef typename E::T T;
  constexpr int kThreads = kQuantThreads<NT>, kRows = kThreads / NT;
  __shared__ uint32_t shared[NT / 64];
  const int64_t groups = (a.M + kRows - 1) / kRows;
  if (blockIdx.x >= groups) {
    pack8_piece(copies, blockIdx.x - groups, kThreads);
    return;
  }
  const int t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
  if (row >= a.M) return;  // whole waves, and none of a row that waits for others
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
    if (col < a.K) kept[p] = fetch(col);
  }
#pragma unroll
  for (int p = 0; p < kKeep; p++)
    if ((p * NT + t) * 8 < a.K) top = max(top, magnitude(kept[p]));
  for (int col = (kKeep * NT + t) * 8; col < a.K; col += NT * 8) top = max(top, magnitude(fetch(col)));
  top = wave_max(top);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; i++) top = max(top, shared[i]);
  }
  const Quantizer quantizer(top);
  if (t == 0) a.scale[row] = quantizer.scale;
  int8_t* q = a.q + row * a.qld;
  auto put = [&](int col, const Vals<E, 8>& v) {
    const uint2 n = quantizer.eight(v.v);
    if (col + 8 <= a.qpad) {
      typedef u32x2 __attribute__((aligned(1))) any_u32x2;
      *(any_u32x2*)(q + col) = u32x2{n.x, n.y};
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (col + i < a.qpad) q[col + i] = (int8_t)((i < 4 ? n.x : n.y) >> 8 * (i & 3));
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
hipError_t quantize(const QuantArgs& a, Pack8Args copies, hipStream_t s) {
  auto launch = [&](auto kernel, int threads, int rows) {
    if (copies.count) copies.first[0] = 0;
    for (int i = 0; i < copies.count; i++)
      copies.first[i + 1] = copies.first[i] + (copies.lines[i] * (copies.dld / 16) + threads - 1) / threads;
    const int64_t copying = copies.count ? copies.first[copies.count] : 0;
    if (!launchable(copying + 1, threads)) return hipErrorInvalidConfiguration;
    if (copying == 0 && a.M == 0) return hipSuccess;
    // more rows than fit below 2^32 threads (2^26 of up to 2048 columns) take further launches
    const int64_t most = ((1ll << 32) - 1) / threads;
    QuantArgs part = a;
    part.M = std::min(a.M, (most - copying) * rows);
    for (int64_t row = 0;;) {
      const int64_t groups = (part.M + rows - 1) / rows + (row == 0 ? copying : 0);
      kernel<<<dim3((uint32_t)groups), dim3(threads), 0, s>>>(part, copies);
      const hipError_t e = hipGetLastError();
      row += part.M;
      if (e != hipSuccess || row == a.M) return e;
      part.x = (const typename E::T*)a.x + row * a.xld;
      part.q = a.q + row * a.qld;
      part.scale = a.scale + row;
      part.M = std::min(a.M - row, most * rows);
    }
  };
  // Many rows: as few threads as hold the row in their registers.  Few: one piece a
  // thread, for the latency.
  if (a.M >= 1024) {
    if (a.K <= 2048) return launch(k_quantize<E, 64, 4, kStrided>, 256, 4);
    if (a.K <= 8192) return launch(k_quantize<E, 256, 4, kStrided>, 256, 1);
    return launch(k_quantize<E, 1024, 2, kStrided>, 1024, 1);
  }
  if (a.K <= 512) return launch(k_quantize<E, 64, 1, kStrided>, 256, 4);
  if (a.K <= 2048) return launch(k_quantize<E, 256, 1, kStrided>, 256, 1);
  return launch(k_quantize<E, 1024, 2, kStrided>, 1024, 1);
}
hipError_t launch_quantize(int kind, const QuantArgs& a, const Pack8Args& copies, hipStream_t s) {
  if (a.xcs == 1)
    return kind == 0   ? quantize<F32, false>(a, copies, s)
           : kind == 1 ? quantize<F16, false>(a, copies, s)
                       : quantize<BF16, false>(a, copies, s);
  return kind == 0   ? quantize<F32, true>(a, copies, s)
         : kind == 1 ? quantize<F16, true>(a, copies, s)
                     : quantize<BF16, true>(a, copies, s);
}

// ---- few rows ------------------------------------------------------------------------
// 16 P weight rows (gated: half of them of each projection) a workgroup times up to 16
// NB rows of x, its waves take the steps of k in turn.
template <class Out, bool kGated, int P, int NB, int kWaves>
__global__ __launch_bounds__(kWaves * 64) void k_few_int8(GemmArgs a) {
  typedef Int8<Out> E;
  constexpr int kN = kGated ? 8 * P : 16 * P, G = 2;
  __shared__ int part[P][kWaves][16][16];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kN;
  // weight row i of the workgroup: gated, the first half of one projection
  const char* w[P];
#pragma unroll
  for (int p = 0; p < P; p++) {
    const int i = 16 * p + r;
    w[p] = (const char*)a.w[kGated ? i / kN : 0] + min(n0 + i % kN, a.N - 1) * a.wld + q * (16 * G);
  }
  bool live[NB];
  const char* x[NB];
#pragma unroll
  for (int b = 0; b < NB; b++) {
    live[b] = 16 * b + r < a.M;
    x[b] = (const char*)a.x[0] + (live[b] ? 16 * b + r : 0) * a.xld + q * (16 * G);
  }
  f32x4 acc[P][NB];
  clear<E>(acc);
  constexpr int kStep = 64 * G;
  multiply_steps<E, P, NB, G, 2>(acc, w, x, live, a.K, wave, (a.K + kStep - 1) / kStep, kWaves);
#pragma unroll
  for (int b = 0; b < NB; b++) {
    if (b > 0) __syncthreads();
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
      for (int i = 0; i < 4; i++) part[p][wave][r][4 * q + i] = __float_as_int(acc[p][b][i]);
    __syncthreads();
    for (int i = threadIdx.x; i < min(a.M - 16 * b, 16) * kN; i += kWaves * 64) {
      const int row = i / kN, n = i % kN, m = 16 * b + row;
      if (n0 + n >= a.N) continue;
      constexpr int kPlanes = kGated ? 2 : 1;
      float v[kPlanes];
#pragma unroll
      for (int p = 0; p < kPlanes; p++) {
        const int c = p * kN + n;
        int sum = 0;
#pragma unroll
        for (int k = 0; k < kWaves; k++) sum += part[c / 16][k][row][c % 16];
        v[p] = scaled(sum, a.xscale[m], a.wscale[p][n0 + n]);
      }
      finish<E, kGated, 1>(a, 0, m, n0 + n, &v[0], &v[kPlanes - 1]);
    }
  }
}

// The same for one or two rows of values, quantised by every workgroup for itself
// (a call with weights that are not in the caches, bf16, 3584 -> 8192: one row 7.8 us, two
// 9.4; four rows would take 13.2, against 11.3 with the quantisation before it):
// the rows' loads go first, half of the weights' follow (all of them up to k = 4096),
// and the maximum and the rounding take place while those are on their way.
template <class Out, bool kGated, int kRows, int kWaves>
__global__ __launch_bounds__(kWaves * 64, 8) void k_few_int8_values(GemmArgs a) {
  typedef Int8<Out> E;
  constexpr int kN = kGated ? 8 : 16, G = 2, kStep = 64 * G, kSteps = kFewValuesK / (kStep * kWaves);
  constexpr int kEarly = kSteps / 2;  // all of them would not leave the registers for a second workgroup
  static_assert(kFewValuesK == kWaves * 64 * 8 && kFewValuesK % (kStep * kWaves) == 0, "a piece a thread");
  __shared__ int part[kWaves][16][16];
  __shared__ __attribute__((aligned(16))) int8_t rows[kRows][kFewValuesK];
  __shared__ uint32_t tops[kRows][kWaves];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kN;
  const int col = threadIdx.x * 8;
  Vals<Out, 8> v[kRows];
#pragma unroll
  for (int m = 0; m < kRows; m++) {
    v[m] = {};
    if (col < a.K) v[m] = load_vals<Out, 8>((const typename Out::T*)a.x[0] + m * a.xld + col, a.K - col);
  }
  const int row = min(n0 + (kGated ? r & 7 : r), a.N - 1);
  const char* w = (const char*)a.w[kGated ? r >> 3 : 0] + row * a.wld + q * (16 * G);
  Chunk<E> wv[kSteps][G];
  auto fetch = [&](int s) {
    const int k = (wave + s * kWaves) * kStep;
#pragma unroll
    for (int g = 0; g < G; g++)
      if (k < a.K) wv[s][g].fetch(w + k + g * 16, a.K - k - (q * G + g) * 16, a.K);
  };
#pragma unroll
  for (int s = 0; s < kEarly; s++) fetch(s);
#pragma unroll
  for (int m = 0; m < kRows; m++) {
    const uint32_t top = wave_max(magnitude(v[m]));
    if (lane == 0) tops[m][wave] = top;
  }
  __syncthreads();
  float scale[kRows];
#pragma unroll
  for (int m = 0; m < kRows; m++) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kWaves; i++) top = max(top, tops[m][i]);
    const Quantizer quantizer(top);
    scale[m] = quantizer.scale;
    if (col < (a.K + kStep - 1) / kStep * kStep) *(uint2*)&rows[m][col] = quantizer.eight(v[m].v);
  }
  __syncthreads();
#pragma unroll
  for (int s = kEarly; s < kSteps; s++) fetch(s);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < kSteps; s++)
#pragma unroll
    for (int g = 0; g < G; g++) {
      const int k = (wave + s * kWaves) * kStep;
      if (k >= a.K) continue;
      Chunk<E> xv;
      xv.zero();
      if (r < kRows) xv.v = *(const u32x4*)&rows[r][k + (q * G + g) * 16];
      if (k + kStep > a.K) wv[s][g].settle(a.K - k - (q * G + g) * 16, a.K);
      acc = mma_chunk<E>(wv[s][g], xv, acc);
    }
  if (r < kRows) {
#pragma unroll
    for (int i = 0; i < 4; i++) part[wave][r][4 * q + i] = __float_as_int(acc[i]);
  }
  __syncthreads();
  if (threadIdx.x >= kRows * kN) return;
  const int m = threadIdx.x / kN, n = threadIdx.x % kN;
  if (n0 + n >= a.N) return;
  constexpr int P = kGated ? 2 : 1;
  float xs = scale[0];
#pragma unroll
  for (int i = 1; i < kRows; i++) xs = m == i ? scale[i] : xs;
  float y[P];
#pragma unroll
  for (int p = 0; p < P; p++) {
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kWaves; k++) sum += part[k][m][p * kN + n];
    y[p] = scaled(sum, xs, a.wscale[p][n0 + n]);
  }
  finish<E, kGated, 1>(a, 0, m, n0 + n, &y[0], &y[P - 1]);
}

template <class Out, bool kGated>
hipError_t few_int8(bool values, const GemmArgs& a, hipStream_t s) {
  // x is read again by every workgroup, half as often where each takes twice the
  // columns: for as long as those still give nearly every CU one workgroup and none two
  // (16 rows, 3584 -> 8192: 8.8 us; 5 rows, 8192 -> 28672: 50.8 us, narrow 41.5).
  const int64_t pairs = few_pairs(a.N, kGated);
  const bool wide = !values && a.M > 4 && pairs >= 192 && pairs <= 256;
  constexpr int kWaves = 16;
  const int cols = (kGated ? 8 : 16) * (wide || a.M > 16 ? 2 : 1);
  const int64_t groups = ((int64_t)a.N + cols - 1) / cols;
  if (groups == 0 || a.M == 0) return hipSuccess;
  if (!launchable(groups, kWaves * 64)) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)groups), block(kWaves * 64);
  if (a.M > 16)
    k_few_int8<Out, kGated, 2, 2, kWaves><<<grid, block, 0, s>>>(a);
  else if (wide)
    k_few_int8<Out, kGated, 2, 1, kWaves><<<grid, block, 0, s>>>(a);
  else if (!values)
    k_few_int8<Out, kGated, 1, 1, kWaves><<<grid, block, 0, s>>>(a);
  else if (a.M == 1)
    k_few_int8_values<Out, kGated, 1, kWaves><<<grid, block, 0, s>>>(a);
  else
    k_few_int8_values<Out, kGated, 2, kWaves><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_few_int8(int kind, bool gated, bool values, const GemmArgs& a, hipStream_t s) {
  if (kind == 0) return gated ? few_int8<F32, true>(values, a, s) : few_int8<F32, false>(values, a, s);
  if (kind == 1) return gated ? few_int8<F16, true>(values, a, s) : few_int8<F16, false>(values, a, s);
  return gated ? few_int8<BF16, true>(values, a, s) : few_int8<BF16, false>(values, a, s);
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
