// llar_ffn_kernels.hip -- the feed-forward operators' kernels beside the
// product itself: joining a product split over k, the gated block's and the
// activation's gradients, and the dispatch over instances.
#include "llar_few.h"

namespace llar_ffn {

#define LLAR_DECL(E, x, w) hipError_t launch_gemm_##E##_##x##w(const GemmPlan&, const GemmArgs&, hipStream_t);
LLAR_DECL(F32, 0, 0) LLAR_DECL(F32, 0, 1) LLAR_DECL(F32, 1, 0) LLAR_DECL(F32, 1, 1)
LLAR_DECL(F16, 0, 0) LLAR_DECL(F16, 0, 1) LLAR_DECL(F16, 1, 0) LLAR_DECL(F16, 1, 1)
LLAR_DECL(BF16, 0, 0) LLAR_DECL(BF16, 0, 1) LLAR_DECL(BF16, 1, 0) LLAR_DECL(BF16, 1, 1)

hipError_t launch_gemm(const GemmPlan& p, const GemmArgs& a, hipStream_t s) {
  typedef hipError_t (*Fn)(const GemmPlan&, const GemmArgs&, hipStream_t);
  static const Fn table[3][2][2] = {
      {{launch_gemm_F32_00, launch_gemm_F32_01}, {launch_gemm_F32_10, launch_gemm_F32_11}},
      {{launch_gemm_F16_00, launch_gemm_F16_01}, {launch_gemm_F16_10, launch_gemm_F16_11}},
      {{launch_gemm_BF16_00, launch_gemm_BF16_01}, {launch_gemm_BF16_10, launch_gemm_BF16_11}}};
  return table[p.kind][p.x_rows][p.w_rows](p, a, s);
}

#define LLAR_PAIR(E) \
  hipError_t launch_pair_##E##_0(int, int, PairArgs&, hipStream_t); \
  hipError_t launch_pair_##E##_1(int, int, PairArgs&, hipStream_t);
LLAR_PAIR(F32) LLAR_PAIR(F16) LLAR_PAIR(BF16)

hipError_t launch_pair(int kind, int tile, int groups, bool w_rows, PairArgs a, hipStream_t s) {
  typedef hipError_t (*Fn)(int, int, PairArgs&, hipStream_t);
  static const Fn table[3][2] = {{launch_pair_F32_0, launch_pair_F32_1},
                                 {launch_pair_F16_0, launch_pair_F16_1},
                                 {launch_pair_BF16_0, launch_pair_BF16_1}};
  return table[kind][w_rows](tile, groups, a, s);
}

// ---- few rows ------------------------------------------------------------------------
template <class E, bool kGated>
hipError_t few(bool w_rows, const GemmArgs& a, hipStream_t s) {
  if (a.N > kFewColumns) return hipErrorInvalidConfiguration;
  if (w_rows) {
    constexpr int kC = 4, kWaves = 8;
    const int64_t grid = ((int64_t)a.N + 16 * kC - 1) / (16 * kC) * a.splits;
    k_few_n<E, kGated, kC, kWaves><<<dim3((uint32_t)grid), dim3(kWaves * 64), 0, s>>>(a);
  } else if (a.M <= 2) {
    constexpr int kN = 4 * (kGated ? 1 : 2);  // columns of a workgroup's four waves
    const dim3 grid((uint32_t)(((int64_t)a.N + kN - 1) / kN));
    if (a.M == 1)
      k_few_dot<E, kGated, 1><<<grid, dim3(256), 0, s>>>(a);
    else
      k_few_dot<E, kGated, 2><<<grid, dim3(256), 0, s>>>(a);
  } else {
    constexpr int kN = kGated ? 8 : 16, kWaves = 16;
    k_few_k<E, kGated, kWaves><<<dim3((uint32_t)((a.N + kN - 1) / kN)), dim3(kWaves * 64), 0, s>>>(a);
  }
  return hipGetLastError();
}
hipError_t launch_few(int kind, bool w_rows, bool gated, const GemmArgs& a, hipStream_t s) {
  if (kind == 0) return gated ? few<F32, true>(w_rows, a, s) : few<F32, false>(w_rows, a, s);
  if (kind == 1) return gated ? few<F16, true>(w_rows, a, s) : few<F16, false>(w_rows, a, s);
  return gated ? few<BF16, true>(w_rows, a, s) : few<BF16, false>(w_rows, a, s);
}

// ---- aligned copies ------------------------------------------------------------------
// Operands that are not whole 16-byte chunks, with zeros up to a whole one: all
// of a call's in one launch, eight elements a thread.  Bound by memory: 168 MB of
// odd rows in 36 us (4.7 TB/s), 19 MB in 8.
template <class E>
__global__ __launch_bounds__(256) void k_repack(RepackArgs a) {
  typedef typename E::T T;
  typedef T vec __attribute__((ext_vector_type(8)));
  typedef vec loose __attribute__((aligned(2)));
  int i = 0;
  while (i + 1 < a.count && blockIdx.x >= a.first[i + 1]) i++;
  const int64_t groups = a.dld[i] / 8;
  const int64_t id = (blockIdx.x - a.first[i]) * 256 + threadIdx.x;
  const int64_t line = id / groups;
  const int64_t at = (id - line * groups) * 8;
  if (line >= a.lines[i]) return;
  const T* src = (const T*)a.src[i] + line * a.ld[i] + at;
  vec v;
  if (at + 8 <= a.width[i]) {
    v = *(const loose*)src;
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = at + e < a.width[i] ? src[e] : (T)0.f;
  }
  *(vec*)((T*)a.dst[i] + line * a.dld[i] + at) = v;
}
hipError_t launch_repack(int kind, const RepackArgs& a, hipStream_t s) {
  const dim3 grid((uint32_t)a.first[a.count]), block(256);
  if (a.first[a.count] == 0) return hipSuccess;
  if (!launchable(a.first[a.count], 256)) return hipErrorInvalidConfiguration;
  if (kind == 0)
    k_repack<F32><<<grid, block, 0, s>>>(a);
  else if (kind == 1)
    k_repack<F16><<<grid, block, 0, s>>>(a);
  else
    k_repack<BF16><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}

// ---- join: out = epilogue(sum over splits, in order) -------------------------------
// Four columns a thread.  Bound by memory: two planes of 4096 x 2048 in 15 us (4.9
// TB/s), of 64 x 3584 in 4.
template <class E, bool kGated>
__global__ __launch_bounds__(256) void k_join(GemmArgs a) {
  const int groups = (a.N + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id / groups;
  const int col = (int)(id - row * groups) * 4;
  const int b = (int)(row / a.M), m = (int)(row - (int64_t)b * a.M);
  if (b >= a.batch) return;
  const int planes = kGated ? 2 : a.batch;
  float v[2][4] = {};
#pragma unroll
  for (int p = 0; p < (kGated ? 2 : 1); p++) {
    const float* src = a.partial + ((int64_t)(kGated ? p : b) * a.M + m) * a.npad + col;
    const int64_t step = (int64_t)planes * a.M * a.npad;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < a.splits; i++) {
      const f32x4 t = *(const f32x4*)(src + i * step);
#pragma unroll
      for (int e = 0; e < 4; e++) s[e] += t[e];
    }
#pragma unroll
    for (int e = 0; e < 4; e++) v[p][e] = s[e];
  }
  finish<E, kGated, 4>(a, b, m, col, v[0], v[1]);
}

template <class E>
hipError_t join(bool gated, const GemmArgs& a, hipStream_t s) {
  const int64_t n = (int64_t)a.batch * a.M * ((a.N + 3) / 4), groups = (n + 255) / 256;
  if (n == 0) return hipSuccess;
  if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)groups);
  if (gated)
    k_join<E, true><<<grid, dim3(256), 0, s>>>(a);
  else
    k_join<E, false><<<grid, dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_join(int kind, bool gated, const GemmArgs& a, hipStream_t s) {
  return kind == 0 ? join<F32>(gated, a, s) : kind == 1 ? join<F16>(gated, a, s) : join<BF16>(gated, a, s);
}

// Eight elements of a row of an incoming gradient; kAny: `cs` apart.
template <class E, bool kAny>
__device__ __forceinline__ Vals<E, 8> load_grad(const void* p, int64_t m, int64_t ld, int64_t cs, int col, int cnt) {
  const typename E::T* row = (const typename E::T*)p + m * ld;
  if constexpr (!kAny) return load_vals<E, 8>(row + col, cnt);
  Vals<E, 8> r;
#pragma unroll
  for (int i = 0; i < 8; i++) r.v[i] = i < cnt ? E::to(row[(col + i) * cs]) : 0.f;
  return r;
}
// The row and the first column of an element-wise pass's piece `id`; kAny: the
// rows first, neighbours in memory where the columns are not (a transposed view:
// 4096 x 8192 bf16 GELU slopes 56 us against 41 for contiguous rows, 43 for one
// value repeated; the gated block's 4096 x 3584 39 against 24).
template <bool kAny>
__device__ __forceinline__ int64_t piece_of(int64_t id, int M, int N, int& col) {
  const int groups = (N + 7) / 8;
  const int64_t m = kAny ? id % M : id / groups;
  col = (int)(kAny ? id / M : id - m * groups) * 8;
  return m;
}

// ---- the gated block's element-wise gradient: 3 reads, 2 writes --------------------
// Eight elements a thread, the exponential shared by value and slope.  Bound by
// memory: 4096 x 3584 bf16 moves 147 MB in 29 us (5.1 TB/s).
template <class E, bool kAny>
__global__ __launch_bounds__(256) void k_gate_grad(GateGradArgs a) {
  typedef typename E::T T;
  int col;
  const int64_t m = piece_of<kAny>((int64_t)blockIdx.x * 256 + threadIdx.x, a.M, a.N, col);
  if (m >= a.M || col >= a.N) return;
  const int cnt = a.N - col;
  const Vals<E, 8> dh = load_grad<E, kAny>(a.dh, m, a.dhld, a.dhcs, col, cnt);
  const Vals<E, 8> g = load_vals<E, 8>((const T*)a.g + m * a.gld + col, cnt);
  const Vals<E, 8> u = load_vals<E, 8>((const T*)a.u + m * a.uld + col, cnt);
  float dg[8], du[8];
  with_act(a.act, [&](auto c) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      float value, slope;
      act_two<decltype(c)::value, E>(g.v[i], value, slope);
      dg[i] = dh.v[i] * u.v[i] * slope;
      du[i] = dh.v[i] * value;
    }
  });
  // what is loaded beyond column N is 0, and so is its gradient
  store_vals<E, 8>((T*)a.dg + m * a.dld + col, dg, 8);
  store_vals<E, 8>((T*)a.du + m * a.dld + col, du, 8);
}

template <class E>
hipError_t gate_grad(const GateGradArgs& a, hipStream_t s) {
  const int64_t n = (int64_t)a.M * ((a.N + 7) / 8), groups = (n + 255) / 256;
  if (n == 0) return hipSuccess;
  if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)groups), block(256);
  if (a.dhcs == 1)
    k_gate_grad<E, false><<<grid, block, 0, s>>>(a);
  else
    k_gate_grad<E, true><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_gate_grad(int kind, const GateGradArgs& a, hipStream_t s) {
  return kind == 0 ? gate_grad<F32>(a, s) : kind == 1 ? gate_grad<F16>(a, s) : gate_grad<BF16>(a, s);
}

// ---- dz = dy act'(z), and column sums of dz ----------------------------------------
// Eight elements of a row; the sum's share is returned unrounded.
template <class E, bool kAny>
__device__ __forceinline__ Vals<E, 8> act_grad_piece(const ActGradArgs& a, int64_t m, int col) {
  typedef typename E::T T;
  const int cnt = a.N - col;
  Vals<E, 8> d = load_grad<E, kAny>(a.dy, m, a.dyld, a.dycs, col, cnt);
  if (a.z) {
    const Vals<E, 8> z = load_vals<E, 8>((const T*)a.z + m * a.zld + col, cnt);
    with_act(a.act, [&](auto c) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        float value, slope;
        act_two<decltype(c)::value, E>(z.v[i], value, slope);
        d.v[i] *= slope;
      }
    });
  }
  if (a.dz) store_vals<E, 8>((T*)a.dz + m * a.dzld + col, d.v, 8);  // zeros beyond column N
  return d;
}

// Without a bias gradient: a piece a thread (4096 x 4096 bf16, erf form of GELU: 101
// MB in 27 us, 3.7 TB/s; the arithmetic counts).
template <class E, bool kAny>
__global__ __launch_bounds__(256) void k_act_grad(ActGradArgs a) {
  int col;
  const int64_t m = piece_of<kAny>((int64_t)blockIdx.x * 256 + threadIdx.x, a.M, a.N, col);
  if (m < a.M && col < a.N) act_grad_piece<E, kAny>(a, m, col);
}

// With it: a workgroup takes 64 columns of one row chunk, 128 rows at a time
// (a line of memory a row).  One chunk: its sums are the bias gradient.  More:
// they go to part[chunk], and a second kernel adds the chunks in order, so the
// result does not depend on timing.  Bound by memory: 4096 x 8192 bf16 with the
// erf form of GELU moves 201 MB in 51 us (3.9 TB/s), 256 x 3008 takes 9 us.
constexpr int kSumCols = 64, kSumRows = 128, kSumThreads = kSumRows * kSumCols / 8;
template <class E, bool kAny>
__global__ __launch_bounds__(kSumThreads) void k_act_grad_sum(ActGradArgs a) {
  __shared__ float sums[kSumRows][kSumCols + 4];
  const int lane = threadIdx.x % (kSumCols / 8), r = threadIdx.x / (kSumCols / 8);
  const int col = blockIdx.x * kSumCols + lane * 8;
  const int64_t m0 = (int64_t)a.M * blockIdx.y / a.chunks, m1 = (int64_t)a.M * (blockIdx.y + 1) / a.chunks;
  float acc[8] = {};
  if (col < a.N) {
#pragma unroll 2
    for (int64_t m = m0 + r; m < m1; m += kSumRows) {
      const Vals<E, 8> d = act_grad_piece<E, kAny>(a, m, col);
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] += d.v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i++) sums[r][lane * 8 + i] = acc[i];
  // 16 threads a column, 8 rows each, then the 16
  __syncthreads();
  const int c = threadIdx.x % kSumCols, part = threadIdx.x / kSumCols;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumRows * kSumCols / kSumThreads; i++) s += sums[part + i * (kSumThreads / kSumCols)][c];
  __syncthreads();
  sums[part][c] = s;
  __syncthreads();
  const int out = blockIdx.x * kSumCols + c;
  if (part > 0 || out >= a.N) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumThreads / kSumCols; i++) s += sums[i][c];
  if (a.chunks == 1)
    ((typename E::T*)a.db)[out] = E::from(s);
  else
    a.part[(int64_t)blockIdx.y * a.N + out] = s;
}

template <class E>
__global__ __launch_bounds__(256) void k_bias_grad(ActGradArgs a) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.N) return;
  float s = 0.f;
#pragma unroll 8
  for (int i = 0; i < a.chunks; i++) s += a.part[(int64_t)i * a.N + c];
  ((typename E::T*)a.db)[c] = E::from(s);
}

template <class E, bool kAny>
hipError_t act_grad(const ActGradArgs& a, hipStream_t s) {
  if (a.N == 0) return hipSuccess;
  if (!a.db) {
    const int64_t groups = ((int64_t)a.M * ((a.N + 7) / 8) + 255) / 256;
    if (!launchable(groups, 256)) return hipErrorInvalidConfiguration;
    if (groups > 0) k_act_grad<E, kAny><<<dim3((uint32_t)groups), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  }
  const uint32_t cols = (uint32_t)((a.N + kSumCols - 1) / kSumCols);
  if (!launchable((int64_t)cols * a.chunks, kSumThreads)) return hipErrorInvalidConfiguration;
  k_act_grad_sum<E, kAny><<<dim3(cols, (uint32_t)a.chunks), dim3(kSumThreads), 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.chunks == 1) return e;
  k_bias_grad<E><<<dim3((uint32_t)((a.N + 255) / 256)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_act_grad(int kind, const ActGradArgs& a, hipStream_t s) {
  if (a.dycs == 1)
    return kind == 0 ? act_grad<F32, false>(a, s) : kind == 1 ? act_grad<F16, false>(a, s) : act_grad<BF16, false>(a, s);
  return kind == 0 ? act_grad<F32, true>(a, s) : kind == 1 ? act_grad<F16, true>(a, s) : act_grad<BF16, true>(a, s);
}

}  // namespace llar_ffn
