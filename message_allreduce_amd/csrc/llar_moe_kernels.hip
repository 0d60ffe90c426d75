// llar_moe_kernels.hip -- the router, and the experts of a few tokens in two kernels.
#include "llar_chunk.h"
#include "llar_moe.h"

namespace llar_ffn {

// ---- the router's logits --------------------------------------------------------------
// In binary64: the choice is that of the exact sums unless two are within its rounding,
// and equal rows of the router, summed in the same order, tie.  A workgroup takes 16
// tokens by 16 experts and a share of k, its waves 128 k at a time with all their loads
// in flight: lane (r, q) holds eight k of token r and of expert r, widened, and the
// matrix unit multiplies four k at a time (which four is the same for both).  k is
// shared between as many workgroups as the card holds: 1 token, 64 experts, k 4096 bf16
// 4.5 us, the loads' latency; 64 tokens, 256 experts, k 8192 11 us, of which the binary64
// products are 3.4.
typedef double f64x4 __attribute__((ext_vector_type(4)));

constexpr int kRouteWaves = 4, kRouteSteps = 4, kRouteK = kRouteWaves * kRouteSteps * 32;

// Eight neighbours as they lie in memory, zeros where they do not exist.
template <class E>
struct Row8 {
  typename Wide<E, 8>::vec v;
  __device__ __forceinline__ void load(const typename E::T* p, int64_t left) {
    if (left >= 8) {
      v = *(const typename Wide<E, 8>::loose*)p;
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = i < left ? p[i] : (typename E::T)0.f;
    }
  }
  __device__ __forceinline__ float at(int i) const { return E::to(v[i]); }
};

template <class E>
__global__ __launch_bounds__(kRouteWaves * 64) void k_route_logits(RouteArgs a) {
  typedef typename E::T T;
  __shared__ double part[kRouteWaves][16][16 + 1];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = (a.E + 15) / 16;
  const int split = (int)(blockIdx.x % a.splits), tile = (int)(blockIdx.x / a.splits);
  const int e0 = tile % groups * 16, t0 = tile / groups * 16;
  const T* x = (const T*)a.x + (int64_t)min(t0 + r, a.M - 1) * a.xld;
  const T* w = (const T*)a.w + (int64_t)min(e0 + r, a.E - 1) * a.wld;
  const int64_t stride = (int64_t)a.splits * kRouteK;
  Row8<E> xv[kRouteSteps], wv[kRouteSteps];
  auto fetch = [&](int64_t k0) {
#pragma unroll
    for (int s = 0; s < kRouteSteps; s++) {
      const int64_t k = k0 + s * 32 + q * 8;
      xv[s].load(x + k, a.K - k);
      wv[s].load(w + k, a.K - k);
    }
  };
  f64x4 acc = {0., 0., 0., 0.};
  int64_t k0 = (int64_t)split * kRouteK + wave * (kRouteSteps * 32);
  if (k0 < a.K) fetch(k0);
  for (; k0 < a.K; k0 += stride) {
    Row8<E> xn[kRouteSteps], wn[kRouteSteps];
#pragma unroll
    for (int s = 0; s < kRouteSteps; s++) {
      xn[s] = xv[s];
      wn[s] = wv[s];
    }
    if (k0 + stride < a.K) fetch(k0 + stride);
#pragma unroll
    for (int s = 0; s < kRouteSteps; s++)
#pragma unroll
      for (int e = 0; e < 8; e++)
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)wn[s].at(e), (double)xn[s].at(e), acc, 0, 0, 0);
  }
  // lane: token r, experts q + 4 i
#pragma unroll
  for (int i = 0; i < 4; i++) part[wave][r][q + 4 * i] = acc[i];
  __syncthreads();
  const int t = threadIdx.x / 16, e = threadIdx.x % 16;
  if (t0 + t >= a.M || e0 + e >= a.E) return;
  double s = 0.;
#pragma unroll
  for (int j = 0; j < kRouteWaves; j++) s += part[j][t][e];
  a.logits[((int64_t)split * a.M + t0 + t) * a.E + e0 + e] = s;
}

// ---- the choice ------------------------------------------------------------------------
// The largest of the wave's values, none of them a NaN.
__device__ __forceinline__ double wave_max(double v) {
  union {
    double d;
    int i[2];
  } u, o;
  u.d = v;
  auto step = [&](auto ctrl) {
#pragma unroll
    for (int h = 0; h < 2; h++) o.i[h] = __builtin_amdgcn_update_dpp(u.i[h], u.i[h], decltype(ctrl)::value, 0xf, 0xf, false);
    u.d = fmax(u.d, o.d);
  };
  step(std::integral_constant<int, 0x111>());  // lane - 1 of 16
  step(std::integral_constant<int, 0x112>());
  step(std::integral_constant<int, 0x114>());
  step(std::integral_constant<int, 0x118>());
  step(std::integral_constant<int, 0x142>());  // lane 15 of 16 to the next 16
  step(std::integral_constant<int, 0x143>());  // lane 31 to the upper 32
#pragma unroll
  for (int h = 0; h < 2; h++) u.i[h] = __builtin_amdgcn_readlane(u.i[h], 63);
  return u.d;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// A wave a token: lane l holds the logits of the experts l, l + 64, ...; the largest
// left is taken top_k times, the lowest number first among equals.  A NaN counts as
// below everything, so that the choices are distinct experts whatever the logits are.
template <int kPerLane>
__device__ __forceinline__ void route_choose(const RouteArgs& a, int64_t t, double (&v)[kPerLane]) {
  const int lane = threadIdx.x & 63;
  const double kNone = -__builtin_inf();
  uint32_t left = 0, nans = 0;  // bit i: expert lane + 64 i is not chosen yet; has a NaN
#pragma unroll
  for (int i = 0; i < kPerLane; i++) {
    if (lane + 64 * i < a.E) left |= 1u << i;
    if (v[i] != v[i]) nans |= 1u << i;
    if (lane + 64 * i >= a.E || v[i] != v[i]) v[i] = kNone;
  }
  left &= ~nans;
  const bool nan = __any(nans != 0);
  double mine = 0., top = 0.;  // lane j: the logit of choice j
  int chosen = 0;
  for (int j = 0; j < a.top_k; j++) {
    double best = kNone;
#pragma unroll
    for (int i = 0; i < kPerLane; i++)
      if (left >> i & 1) best = fmax(best, v[i]);
    best = wave_max(best);
    int e = -1;
#pragma unroll
    for (int i = kPerLane - 1; i >= 0; i--) {
      const uint64_t at = __ballot((left >> i & 1) && v[i] == best);
      if (at) e = 64 * i + __ffsll((unsigned long long)at) - 1;
    }
    if (e < 0) {  // only NaNs are left
#pragma unroll
      for (int i = kPerLane - 1; i >= 0; i--) {
        const uint64_t at = __ballot(nans >> i & 1);
        if (at) e = 64 * i + __ffsll((unsigned long long)at) - 1;
      }
    }
    if (e % 64 == lane) {
      left &= ~(1u << (e / 64));
      nans &= ~(1u << (e / 64));
    }
    if (j == 0) top = best;
    if (lane == j) {
      mine = best;
      chosen = e;
    }
  }
  const bool live = lane < a.top_k;
  // Below e^-600 sigmoids are exponentials to binary64's last digit; shares of their sum are
  // taken without the common factor, which would lead out of its range at e^-708.
  const bool shares = !a.sigmoid || (a.normalize && top < -600.);
  const double score = !live ? 0. : shares ? exp(mine - top) : 1. / (1. + exp(-mine));
  double sum = 1.;  // sigmoid scores stand by themselves unless they are normalised
  if (a.normalize) {
    sum = wave_sum(score);
  } else if (!a.sigmoid) {
    sum = 0.;
#pragma unroll
    for (int i = 0; i < kPerLane; i++)
      if (lane + 64 * i < a.E) sum += exp(v[i] - top);
    sum = wave_sum(sum);
  }
  if (live) {
    a.experts[t * a.top_k + lane] = chosen;
    a.weights[t * a.top_k + lane] = nan ? __builtin_nanf("") : (float)(score / sum);
  }
}

template <int kPerLane>
__global__ __launch_bounds__(64) void k_route_choose(RouteArgs a) {
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  double v[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; i++) v[i] = 0.;
  // the shares' sums in order, their loads a batch at a time
  constexpr int kBatch = kPerLane > 4 ? 1 : 8 / kPerLane;
  for (int s0 = 0; s0 < a.splits; s0 += kBatch) {
    double part[kBatch][kPerLane];
#pragma unroll
    for (int s = 0; s < kBatch; s++) {
      const double* l = a.logits + ((int64_t)min(s0 + s, a.splits - 1) * a.M + t) * a.E;
#pragma unroll
      for (int i = 0; i < kPerLane; i++) part[s][i] = l[min(lane + 64 * i, a.E - 1)];
    }
#pragma unroll
    for (int s = 0; s < kBatch; s++)
#pragma unroll
      for (int i = 0; i < kPerLane; i++)
        if (s0 + s < a.splits) v[i] += part[s][i];
  }
  route_choose<kPerLane>(a, t, v);
}

// Few tokens and a small router in one kernel: a workgroup a token, its waves kRows
// experts at a time.  Widening an element takes as long as four multiplications, so
// one CU is as fast as two kernels up to 2^17 elements (1 token bf16, 8 experts, k
// 4096: 4.4 us against 4.6 + 2.3; 64, k 1024: 6.3 against 4.6 + 3.1; 64, k 2048: 8.4
// against 4.6 + 3.3; 128, k 1024: 10.9 against 4.6 + 4.1).
template <class E, int kRows>
__global__ __launch_bounds__(1024) void k_route_token(RouteArgs a) {
  typedef typename E::T T;
  constexpr int kWaves = 16;
  __shared__ double logits[64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  const T* x = (const T*)a.x + t * a.xld;
  for (int e0 = wave * kRows; e0 < a.E; e0 += kWaves * kRows) {
    const T* w[kRows];
#pragma unroll
    for (int i = 0; i < kRows; i++) w[i] = (const T*)a.w + (int64_t)min(e0 + i, a.E - 1) * a.wld;
    double acc[kRows] = {};
#pragma unroll 2
    for (int k = lane * 8; k < a.K; k += 512) {
      Row8<E> xv, wv[kRows];
      xv.load(x + k, a.K - k);
#pragma unroll
      for (int i = 0; i < kRows; i++) wv[i].load(w[i] + k, a.K - k);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const double xe = xv.at(e);
#pragma unroll
        for (int i = 0; i < kRows; i++) acc[i] = fma((double)wv[i].at(e), xe, acc[i]);
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < kRows; i++) acc[i] += __shfl_xor(acc[i], d);
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kRows; i++)
        if (e0 + i < a.E) logits[e0 + i] = acc[i];
    }
  }
  __syncthreads();
  if (wave > 0) return;
  double v[1] = {logits[min(lane, a.E - 1)]};
  route_choose<1>(a, t, v);
}

bool route_small(int64_t m, int64_t experts, int64_t k) {
  return m <= kRouteSmallTokens && experts <= 64 && experts * k <= kRouteSmall;
}

int route_splits(int64_t m, int64_t experts, int64_t k) {
  // two workgroups a CU
  const int64_t tiles = (m + 15) / 16 * ((experts + 15) / 16), shares = (k + kRouteK - 1) / kRouteK;
  int64_t splits = 512 / (tiles > 0 ? tiles : 1);
  if (splits > shares) splits = shares;
  return splits < 1 ? 1 : (int)splits;
}

template <class E>
hipError_t route(const RouteArgs& a, hipStream_t s) {
  if (a.small) {
    const dim3 grid((uint32_t)a.M), block(1024);
    if (a.E <= 16)
      k_route_token<E, 1><<<grid, block, 0, s>>>(a);
    else
      k_route_token<E, 4><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
  }
  const int64_t groups = ((int64_t)a.M + 15) / 16 * ((a.E + 15) / 16) * a.splits;
  if (!launchable(groups, kRouteWaves * 64) || !launchable(a.M, 64)) return hipErrorInvalidConfiguration;
  k_route_logits<E><<<dim3((uint32_t)groups), dim3(kRouteWaves * 64), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((uint32_t)a.M), block(64);
  if (a.E <= 64)
    k_route_choose<1><<<grid, block, 0, s>>>(a);
  else if (a.E <= 256)
    k_route_choose<4><<<grid, block, 0, s>>>(a);
  else
    k_route_choose<kMoeExperts / 64><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_route(int kind, const RouteArgs& a, hipStream_t s) {
  return kind == 0 ? route<F32>(a, s) : kind == 1 ? route<F16>(a, s) : route<BF16>(a, s);
}

// ---- experts ----------------------------------------------------------------------------
// The expert of choice p, -1 if it is not one of these.
__device__ __forceinline__ int expert_at(const MoeArgs& a, int p) {
  const int words = a.id_bytes / 4;
  const uint32_t* id = (const uint32_t*)a.ids + (int64_t)p * words;
  const uint32_t low = id[0], high = id[words - 1];
  return low < (uint32_t)a.E && (words == 1 || high == 0) ? (int)low : -1;
}
// Which places of the lane's token's list name expert e, a bit each: the choices go
// over the lanes 64 at a time, their loads eight at a time, and what a ballot says of
// them is cut to the lane's token's part.
__device__ __forceinline__ uint32_t places_of(const MoeArgs& a, int e) {
  const int lane = threadIdx.x & 63, choices = a.T * a.top_k, first = lane * a.top_k;
  uint64_t mine = 0;
  for (int p0 = 0; p0 < choices; p0 += 512) {
    int id[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const int p = p0 + 64 * i + lane;
      id[i] = -1;
      if (p0 + 64 * i < choices) id[i] = expert_at(a, min(p, choices - 1));
      if (p >= choices) id[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
      if (p0 + 64 * i >= choices) break;
      const uint64_t named = __ballot(id[i] == e);
      const int off = first - p0 - 64 * i;
      mine |= off >= 64 ? 0 : off >= 0 ? named >> off : -off < a.top_k ? named << -off : 0;
    }
  }
  return lane < a.T ? (uint32_t)mine & (uint32_t)((1ull << a.top_k) - 1) : 0u;
}
// Lane i gets the value of the i-th of the lanes in `chose`.
__device__ __forceinline__ int gathered(uint64_t chose, int value) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (1ull << lane) - 1;
  const int to = chose >> lane & 1 ? __popcll(chose & below) : __popcll(chose) + __popcll(~chose & below);
  return __builtin_amdgcn_ds_permute(to * 4, value);
}
// A token and one of its places, as lanes hand them round.
__device__ __forceinline__ int member_of(int token, int place) { return token | place << 8; }

// Rows of whole numbers in LDS lie `moe_pitch` bytes apart: whole steps, and 16 more
// so that rows do not meet in the banks.
__host__ __device__ inline int moe_pitch(int k) { return (k + 127) / 128 * 128 + 16; }

// Quantises a row of k values into LDS, with zeros up to a whole step: NT threads, a
// wave or the whole workgroup (which then meets at barriers, and needs tops, a word a
// wave).
template <class V, int NT>
__device__ __forceinline__ void quantize_row(const typename V::T* x, int k, int pitch, lds_char* to, float* scale,
                                             uint32_t* tops) {
  const int t = threadIdx.x % NT;
  uint32_t top = 0;
  for (int col = t * 8; col < k; col += NT * 8) top = max(top, magnitude(load_vals<V, 8>(x + col, k - col)));
  top = wave_max(top);
  if constexpr (NT > 64) {
    if (t % 64 == 0) tops[t / 64] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; i++) top = max(top, tops[i]);
  }
  const Quantizer quantizer(top);
  if (t == 0) *scale = quantizer.scale;
  for (int col = t * 8; col < pitch; col += NT * 8) {
    uint2 n = make_uint2(0, 0);
    if (col < k) n = quantizer.eight(load_vals<V, 8>(x + col, k - col).v);
    *(LLAR_LDS u32x2*)(to + col) = u32x2{n.x, n.y};
  }
  if constexpr (NT > 64) __syncthreads();
}

// The inner rows as the second kernel's matrix operands: a 16-bit value, and as a second
// one what its rounding left, so that the result is rounded once (error in the 2-norm
// against binary64, bfloat16 0.0017 instead of 0.0024 with one number; binary16 0.00021
// instead of 0.00033).  binary16's rest is lifted by 2^11, because products of two small
// numbers are soon below its 2^-14 and have few digits there; bfloat16's has the range.
// Both kernels take 3 to 13 % more time for it, since every workgroup reads the inner rows
// (bfloat16 1 token 8 of 64 experts 4096 x 1024 44.4 -> 46.0 us, 64 tokens 311 -> 351;
// 2 of 8 8192 x 3584 85 -> 89 and 292 -> 325).
template <class E>
struct Inner {
  static constexpr bool kTwo = std::is_same_v<E, F16> || std::is_same_v<E, BF16>;
  static constexpr float kLift = std::is_same_v<E, F16> ? 2048.f : 1.f;
  static __device__ __forceinline__ void put(typename E::T* to, int64_t low, float v) {
    const typename E::T high = E::from(v);
    *to = high;
    if constexpr (kTwo) {
      const float rest = v - E::to(high);
      to[low] = E::from(fabsf(rest) < __builtin_inff() ? rest * kLift : 0.f);
    }
  }
  // Where the sum of the values is not finite, that of the rests says nothing.
  static __device__ __forceinline__ float sum(float high, float rest) {
    return fabsf(high) < __builtin_inff() ? fmaf(rest, 1.f / kLift, high) : high;
  }
};

// First kernel: h = act(x wg^T) (x wu^T) of every choice, in the I/O type (Inner), in
// binary32 where it is to be quantised.  A
// workgroup takes 16 inner columns (16 rows of each projection) of one expert for all
// the tokens that chose it, up to 64: its weights are read once.  Every wave finds
// those tokens by itself, a token a lane, without a word of shared memory.  Where the
// card would be half empty it takes eight inner columns (P = 1).  Bound by
// reading the weights: 1 token, 8 of 64 experts 4096 x 1024 bf16 28.5 us (4.7 TB/s, the
// launch included), 16 tokens 181 (5.2); 48 tokens, 8 experts 8192 x 3584 int8 95 (4.9).
//
// With fewer choices than experts the grid has a slot for each choice, and the
// slot of an expert's first choice does its work; else a slot for each expert.
template <class E, int P, int NB, int kWaves, bool kValues>
__device__ __forceinline__ void moe_up_rows(const MoeArgs& a, const char* const (&w)[P], int member, int count, int e,
                                            int n0, float (*part)[P][16][16], const lds_char* rows, int pitch,
                                            const float* xscale) {
  constexpr int G = NB <= 2 ? 2 : 1, U = 2, ES = sizeof(typename E::X), kStep = 64 * G / ES, kCols = 8 * P;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  typedef std::conditional_t<kValues, const lds_char, const char> Row;
  bool live[NB];
  Row* x[NB];
#pragma unroll
  for (int b = 0; b < NB; b++) {
    live[b] = 16 * b + r < count;
    const int t = __shfl(member, 16 * b + r) & 255;
    if constexpr (kValues)
      x[b] = rows + (live[b] ? t * pitch : 0) + q * (16 * G);
    else
      x[b] = (const char*)a.x + (live[b] ? t * a.xld * ES : 0) + q * (16 * G);
  }
  const char* at[P];
#pragma unroll
  for (int p = 0; p < P; p++) at[p] = w[p] + q * (16 * G);
  // the scales that a thread's results need, ahead of the operands
  float ws[2] = {1.f, 1.f}, xs[NB];
#pragma unroll
  for (int b = 0; b < NB; b++) xs[b] = 1.f;
  if constexpr (E::kInt8) {
    if (threadIdx.x < 16 * kCols) {
      const int64_t col = (int64_t)e * a.N + min(n0 + (int)threadIdx.x % kCols, a.N - 1);
#pragma unroll
      for (int p = 0; p < 2; p++) ws[p] = a.wscale[p][col];
#pragma unroll
      for (int b = 0; b < NB; b++) xs[b] = xscale[min(__shfl(member, 16 * b + (int)threadIdx.x / kCols) & 255, a.T - 1)];
    }
  }
  f32x4 acc[P][NB];
  clear<E>(acc);
  multiply_steps<E, P, NB, G, U>(acc, at, x, live, a.K, wave, (a.K + kStep - 1) / kStep, kWaves);
#pragma unroll
  for (int b = 0; b < NB; b++) {
    if (b > 0) {
      if (16 * b >= count) break;
      __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < P; p++) *(f32x4*)&part[wave][p][r][4 * q] = acc[p][b];
    __syncthreads();
    if (threadIdx.x < 16 * kCols) {  // whole waves
      const int row = threadIdx.x / kCols, col = threadIdx.x % kCols;
      const int m = __shfl(member, 16 * b + row);
      float v[2];
#pragma unroll
      for (int p = 0; p < 2; p++) {
        const int i = p * kCols + col;  // weight row of the workgroup
        v[p] = part[0][i / 16][row][i % 16];
#pragma unroll
        for (int k = 1; k < kWaves; k++) v[p] = add_sums<E>(v[p], part[k][i / 16][row][i % 16]);
      }
      if (16 * b + row < count && n0 + col < a.N) {
        const int64_t to = (int64_t)((m & 255) * a.top_k + (m >> 8)) * a.hld + n0 + col;
        if constexpr (E::kInt8) {
          float g[1] = {scaled(__float_as_int(v[0]), xs[b], ws[0])};
          const float u = scaled(__float_as_int(v[1]), xs[b], ws[1]);
          act_values<F32, 1>(g, a.act);
          ((float*)a.h)[to] = g[0] * u;
        } else {
          float g[1] = {v[0]};
          act_values<E, 1>(g, a.act);
          Inner<E>::put((typename E::T*)a.h + to, a.hlow, g[0] * v[1]);
        }
      }
    }
  }
}

template <class E, int P, int NB, int kWaves, bool kValues>
__global__ __launch_bounds__(kWaves * 64) void k_moe_up(MoeArgs a, int tiles, bool by_choice) {
  extern __shared__ __attribute__((aligned(16))) char quantized[];  // kValues: [T][pitch]
  __shared__ float part[kWaves][P][16][16], own_scale[kMoeValuesTokens];
  constexpr int ES = sizeof(typename E::X);
  const int lane = threadIdx.x & 63, r = lane & 15;
  const int slot = blockIdx.x / tiles, n0 = (int)(blockIdx.x % tiles) * (8 * P);
  const int e = by_choice ? expert_at(a, slot) : slot;
  if (e < 0) return;
  const uint32_t places = places_of(a, e);
  const uint64_t chose = __ballot(places != 0);
  const int count = __popcll(chose);
  if (count == 0) return;
  const int member = gathered(chose, member_of(lane, places ? __builtin_ctz(places) : 0));
  if (by_choice) {
    const int first = __builtin_amdgcn_readfirstlane(member);
    if ((first & 255) * a.top_k + (first >> 8) != slot) return;
  }
  const char* w[P];
#pragma unroll
  for (int p = 0; p < P; p++) {
    const int i = 16 * p + r;
    w[p] = (const char*)a.w[i / (8 * P)] + (e * a.w_expert + min(n0 + i % (8 * P), a.N - 1) * a.wld) * ES;
  }
  const int pitch = moe_pitch(a.K);
  const float* xscale = kValues ? own_scale : a.xscale;
  if constexpr (kValues) {
    for (int t = 0; t < a.T; t++)
      quantize_row<typename E::Values, kWaves * 64>((const typename E::T*)a.x + t * a.xld, a.K, pitch,
                                                    (lds_char*)quantized + t * pitch, &own_scale[t], (uint32_t*)part);
  }
  auto run = [&](auto blocks) {
    moe_up_rows<E, P, decltype(blocks)::value, kWaves, kValues>(a, w, member, count, e, n0, part, (lds_char*)quantized, pitch,
                                                             xscale);
  };
  if (NB == 1 || count <= 16)
    run(std::integral_constant<int, 1>());
  else if (NB == 2 || count <= 32)
    run(std::integral_constant<int, (NB < 2 ? NB : 2)>());
  else
    run(std::integral_constant<int, NB>());
}

// Second kernel: y = sum over the choices of weight * h wd^T, + residual.  A
// workgroup takes 16 P output columns for all tokens and experts; the waves take
// equal runs of the (expert, k step) pairs.  A fragment's rows are the tokens that
// chose the expert, as in the first kernel; when a wave leaves an expert it adds
// their weighted sums to its own row of every such token in LDS.  No atomics: the
// waves' rows are added in order.  Bound by reading the weights, and the inner rows
// again by every workgroup, in bf16 two numbers each: the same cases 17 us (3.9 TB/s), 104
// (4.5) and 48 (4.9).
template <class E, int P, int NB, bool kValues>
__device__ __forceinline__ void moe_down_rows(const MoeArgs& a, const char* const (&w)[P], int member, float factor,
                                              int count, int e, int n0, int k0, int k1, float* mine,
                                              const lds_char* inner, int pitch, const float* hscale) {
  constexpr int kParts = Inner<E>::kTwo ? 2 : 1, NX = NB * kParts;
  constexpr int G = NB <= 2 ? 2 : 1, U = P * NB * G > 4 ? 1 : 2, ES = sizeof(typename E::X);
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  typedef std::conditional_t<kValues, const lds_char, const char> Row;
  bool live[NX];
  Row* h[NX];
  int token[NB];
  float f[NB], hs[NB], ds[P][4];
#pragma unroll
  for (int b = 0; b < NB; b++) {
    live[b] = 16 * b + r < count;
    const int m = __shfl(member, 16 * b + r);
    f[b] = __shfl(factor, 16 * b + r);
    token[b] = m & 255;
    const int p = live[b] ? (m & 255) * a.top_k + (m >> 8) : 0;
    hs[b] = 1.f;
    if constexpr (E::kInt8) hs[b] = hscale[p];
    if constexpr (kValues)
      h[b] = inner + p * pitch + q * (16 * G);
    else
      h[b] = (const char*)a.h + p * a.hld * ES + q * (16 * G);
    if constexpr (kParts == 2) {
      live[NB + b] = live[b];
      h[NB + b] = h[b] + a.hlow * ES;
    }
  }
  const char* at[P];
#pragma unroll
  for (int p = 0; p < P; p++) at[p] = w[p] + q * (16 * G);
  // scales are fetched with the first operands and used after the last
#pragma unroll
  for (int p = 0; p < P; p++)
#pragma unroll
    for (int v = 0; v < 4; v++) {
      ds[p][v] = 1.f;
      if constexpr (E::kInt8) ds[p][v] = a.dscale[(int64_t)e * a.outs + min(n0 + 16 * p + 4 * q + v, a.outs - 1)];
    }
  f32x4 acc[P][NX];
  clear<E>(acc);
  // a step here is G chunks a lane; k0 and k1 count single ones
  multiply_steps<E, P, NX, G, U>(acc, at, h, live, a.N, k0 / G, (k1 + G - 1) / G, 1);
#pragma unroll
  for (int b = 0; b < NB; b++) {
    if (!live[b]) continue;
    if constexpr (E::kInt8) f[b] *= hs[b];
#pragma unroll
    for (int p = 0; p < P; p++) {
      f32x4* y = (f32x4*)(mine + (token[b] * P + p) * 16 + 4 * q);
      f32x4 sum = *y;
#pragma unroll
      for (int v = 0; v < 4; v++) {
        float c = acc[p][b][v];
        if constexpr (kParts == 2) c = Inner<E>::sum(c, acc[p][NB + b][v]);
        sum[v] = fmaf(f[b], E::kInt8 ? (float)__float_as_int(c) * ds[p][v] : c, sum[v]);
      }
      *y = sum;
    }
  }
}

template <class E, int P, int NB, int kWaves, bool kValues>
__global__ __launch_bounds__(kWaves * 64) void k_moe_down(MoeArgs a) {
  constexpr int ES = sizeof(typename E::X), kStep = 64 / ES, kEven = 2;  // waves' shares: whole pairs of chunks
  extern __shared__ __attribute__((aligned(16))) float part[];  // [kWaves][T][P][16]; kValues: and [choices][pitch]
  __shared__ uint32_t bits[kMoeExperts / 32], chosen[kMoeExperts][2];
  __shared__ int16_t ids[kMoeTokens * kMoeTopK], act[kMoeExperts];
  __shared__ float weights[kMoeTokens * kMoeTopK], own_scale[kValues ? kMoeValuesRows : 1];
  const int lane = threadIdx.x & 63, r = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int share = blockIdx.x % a.parts, n0 = (int)(blockIdx.x / a.parts) * (16 * P);
  const int choices = a.T * a.top_k, rows = a.T * P * 16;
  float* mine = part + wave * rows;
  for (int i = lane * 4; i < rows; i += 256) *(f32x4*)(mine + i) = f32x4{0.f, 0.f, 0.f, 0.f};
  // the experts that any token chose, in order, and for each the tokens
  const int words = (a.E + 31) / 32;
  if (threadIdx.x < words) bits[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < 2 * min(choices, a.E); i += kWaves * 64) (&chosen[0][0])[i] = 0;
  __syncthreads();
  for (int p = threadIdx.x; p < choices; p += kWaves * 64) {
    const int e = expert_at(a, p);
    ids[p] = (int16_t)e;
    weights[p] = a.weights[p];
    if (e >= 0) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  for (int p = threadIdx.x; p < choices; p += kWaves * 64) {
    const int e = ids[p], t = p / a.top_k;
    if (e < 0) continue;
    int rank = __popc(bits[e >> 5] & ((1u << (e & 31)) - 1));
    for (int i = 0; i < e >> 5; i++) rank += __popc(bits[i]);
    act[rank] = (int16_t)e;
    atomicOr(&chosen[rank][t >> 5], 1u << (t & 31));
  }
  int active = 0;
  for (int i = 0; i < words; i++) active += __popc(bits[i]);
  active = __builtin_amdgcn_readfirstlane(active);
  const int pitch = moe_pitch(a.N);
  lds_char* inner = (lds_char*)part + kWaves * rows * 4;
  const float* hscale = kValues ? own_scale : a.hscale;
  if constexpr (kValues) {
    // a row a wave; those of choices without an expert are whatever they were, and not used
    for (int p = wave; p < choices; p += kWaves)
      quantize_row<F32, 64>((const float*)a.h + p * a.hld, a.N, pitch, inner + p * pitch, &own_scale[p], nullptr);
  }
  __syncthreads();

  const int steps = (a.N + kEven * kStep - 1) / (kEven * kStep);  // pairs of chunks of one expert
  const int64_t all = (int64_t)active * steps, runs = (int64_t)a.parts * kWaves, run = share * kWaves + wave;
  int64_t s = all * run / runs;
  const int64_t s1 = all * (run + 1) / runs;
  while (s < s1) {
    const int i = (int)(s / steps), k0 = (int)(s - (int64_t)i * steps);
    const int k1 = (int)min((int64_t)steps, k0 + (s1 - s));
    s += k1 - k0;
    const int e = __builtin_amdgcn_readfirstlane(act[i]);
    const uint64_t chose = (uint64_t)__builtin_amdgcn_readfirstlane(chosen[i][1]) << 32 |
                           (uint32_t)__builtin_amdgcn_readfirstlane(chosen[i][0]);
    const int count = __popcll(chose);
    // the token's places of this expert: the first, and the sum of their weights
    int place = 0;
    float sum = 0.f;
    if (chose >> lane & 1) {
      bool found = false;
      for (int c0 = 0; c0 < a.top_k; c0 += 8) {
        int id[8];
        float weight[8];
#pragma unroll
        for (int c = 0; c < 8; c++) {
          const int at = lane * a.top_k + min(c0 + c, a.top_k - 1);
          id[c] = ids[at];
          weight[c] = weights[at];
        }
#pragma unroll
        for (int c = 0; c < 8; c++)
          if (id[c] == e && c0 + c < a.top_k) {
            sum += weight[c];
            if (!found) place = c0 + c;
            found = true;
          }
      }
    }
    const int member = gathered(chose, member_of(lane, place));
    const float factor = __int_as_float(gathered(chose, __float_as_int(sum)));
    const char* w[P];
#pragma unroll
    for (int p = 0; p < P; p++)
      w[p] = (const char*)a.wd + (e * a.d_expert + min(n0 + 16 * p + r, a.outs - 1) * a.dld) * ES;
    auto multiply = [&](auto blocks) {
      moe_down_rows<E, P, decltype(blocks)::value, kValues>(a, w, member, factor, count, e, n0, kEven * k0, kEven * k1, mine,
                                                            inner, pitch, hscale);
    };
    if (NB == 1 || count <= 16)
      multiply(std::integral_constant<int, 1>());
    else if (NB == 2 || count <= 32)
      multiply(std::integral_constant<int, (NB < 2 ? NB : 2)>());
    else
      multiply(std::integral_constant<int, NB>());
  }
  __syncthreads();
  typedef typename E::T T;
  for (int i = threadIdx.x; i < rows; i += kWaves * 64) {
    const int t = i / (16 * P), c = n0 + i % (16 * P);
    if (c >= a.outs) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWaves; k++) v += part[k * rows + i];
    if (a.parts > 1) {
      a.partial[((int64_t)share * a.T + t) * a.outs + c] = v;
      continue;
    }
    if (a.resid) v += E::to(((const T*)a.resid)[t * a.rld + c]);
    ((T*)a.out)[t * a.outld + c] = E::from(v);
  }
}

// The shares' sums, in their order, and the residual.
template <class E>
__global__ __launch_bounds__(256) void k_moe_join(MoeArgs a) {
  typedef typename E::T T;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, count = (int64_t)a.T * a.outs;
  if (i >= count) return;
  float v = 0.f;
#pragma unroll 8
  for (int s = 0; s < a.parts; s++) v += a.partial[s * count + i];
  const int64_t t = i / a.outs, c = i - t * a.outs;
  if (a.resid) v += E::to(((const T*)a.resid)[t * a.rld + c]);
  ((T*)a.out)[t * a.outld + c] = E::from(v);
}

// Eight waves a workgroup: two to four workgroups a CU cover each other's ends
// (1 token, 8 of 64 experts 4096 x 1024 bf16: both kernels 46 us against 49 with sixteen
// in the second; 48 tokens, 8 experts 8192 x 3584 int8: first 99 against 107).  Sixteen where
// there are too few workgroups for that (4 tokens, 2 of 16 experts 2048 x 512 fp32 17.5
// against 18.6).  And half the columns a workgroup where twice as many still get a CU
// each (both kernels, 1 token bf16, 2 of 8 experts 8192 x 448: 22.7 us against 29.4; 64
// tokens 4096 x 256 26.8 against 31; but 32 tokens 8192 x 448, 224 workgroups, 52.2
// against 47.2).
template <class E, int P, int kWaves>
hipError_t moe_up(const MoeArgs& a, bool values, bool by_choice, hipStream_t s) {
  const int64_t tiles = ((int64_t)a.N + 8 * P - 1) / (8 * P), groups = tiles * (by_choice ? a.T * a.top_k : a.E);
  if (groups == 0) return hipSuccess;
  if (!launchable(groups, kWaves * 64)) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)groups), block(kWaves * 64);
  if constexpr (E::kInt8) {
    if (values) {
      if (a.T > kMoeValuesTokens) return hipErrorInvalidConfiguration;
      k_moe_up<E, P, 1, kWaves, true><<<grid, block, a.T * moe_pitch(a.K), s>>>(a, (int)tiles, by_choice);
      return hipGetLastError();
    }
  }
  if (a.T <= 16)
    k_moe_up<E, P, 1, kWaves, false><<<grid, block, 0, s>>>(a, (int)tiles, by_choice);
  else if (a.T <= 32)
    k_moe_up<E, P, 2, kWaves, false><<<grid, block, 0, s>>>(a, (int)tiles, by_choice);
  else
    k_moe_up<E, P, 4, kWaves, false><<<grid, block, 0, s>>>(a, (int)tiles, by_choice);
  return hipGetLastError();
}
template <class E>
hipError_t moe_up(const MoeArgs& a, bool values, hipStream_t s) {
  const int64_t choices = (int64_t)a.T * a.top_k;
  const bool by_choice = choices <= a.E;
  const int64_t groups = ((int64_t)a.N + 15) / 16 * (by_choice ? choices : a.E);
  if (groups <= 128) return moe_up<E, 1, 16>(a, values, by_choice, s);
  return groups <= 320 ? moe_up<E, 2, 16>(a, values, by_choice, s) : moe_up<E, 2, 8>(a, values, by_choice, s);
}

template <class E, int P>
hipError_t moe_down(const MoeArgs& a, bool values, hipStream_t s) {
  constexpr int kWaves = 8;
  const int64_t groups = ((int64_t)a.outs + 16 * P - 1) / (16 * P) * a.parts;
  if (groups == 0 || a.T == 0) return hipSuccess;
  if (!launchable(groups, kWaves * 64)) return hipErrorInvalidConfiguration;
  const dim3 grid((uint32_t)groups), block(kWaves * 64);
  const uint32_t lds = kWaves * a.T * P * 16 * 4;
  if constexpr (E::kInt8) {
    if (values) {
      const int choices = a.T * a.top_k;
      if (choices > kMoeValuesRows || a.T > kMoeValuesRows) return hipErrorInvalidConfiguration;
      k_moe_down<E, P, 1, kWaves, true><<<grid, block, lds + choices * moe_pitch(a.N), s>>>(a);
      return hipGetLastError();
    }
  }
  if (a.T <= 16)
    k_moe_down<E, P, 1, kWaves, false><<<grid, block, lds, s>>>(a);
  else if (a.T <= 32)
    k_moe_down<E, P, 2, kWaves, false><<<grid, block, lds, s>>>(a);
  else
    k_moe_down<E, P, 4, kWaves, false><<<grid, block, lds, s>>>(a);
  return hipGetLastError();
}
// Every workgroup reads the inner rows again, so it takes 32 columns where that
// leaves enough workgroups (both kernels, 2 of 8 experts 8192 x 3584: 48 tokens int8 152 us
// against 163, 8 tokens bf16 253 against 261, 64 323 against 372; but 24 tokens, 4 of 32
// experts 4096 x 1024, 183 against 154).
bool moe_wide(int T, int64_t outs) { return T > 4 && outs >= 32 * 192; }

template <class E>
hipError_t moe_down(const MoeArgs& a, bool values, hipStream_t s) {
  const hipError_t e = moe_wide(a.T, a.outs) ? moe_down<E, 2>(a, values, s) : moe_down<E, 1>(a, values, s);
  if (e != hipSuccess || a.parts == 1) return e;
  const int64_t groups = ((int64_t)a.T * a.outs + 255) / 256;
  k_moe_join<E><<<dim3((uint32_t)groups), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

// How many workgroups share the experts of a column tile: with few outputs and many
// experts a wave would go from one expert to the next for long (59 tokens, 94 experts,
// 479 outputs int8 56 us, now 10.7 and 2.8 for the join; 1 token, 6 experts, 477 outputs
// fp16 12.7, now 7.0 and 1.8).  The costs in us: an expert, a pair of chunks, and the join
// with its launch.  From 128 column tiles on the weights' bytes are the bound, and a join
// only adds to them (24 tokens, 4 of 32 experts 4096 x 1024 bf16, both kernels 154 us, shared
// by two 163).
int moe_parts(int T, int64_t n, int64_t outs, int64_t experts, int top_k, int es) {
  const int64_t tiles = (outs + 15) / 16, choices = (int64_t)T * top_k;
  if (moe_wide(T, outs) || choices == 0 || n == 0 || tiles == 0) return 1;
  const int64_t steps = (n * es + 127) / 128, all = (choices < experts ? choices : experts) * steps;
  int best = 1;
  double least = 0;
  for (int parts = 1; parts <= 16 && (parts == 1 || tiles * parts <= 256); parts *= 2) {
    const double pairs = (double)all / (8 * parts);  // of a wave
    const double cost = (pairs / steps + 1) * 2 + pairs * 0.5 + (parts > 1 ? 4.5 : 0);
    if (parts == 1 || cost < least) {
      least = cost;
      best = parts;
    }
  }
  return best;
}

hipError_t launch_moe_up(int kind, bool int8, bool values, const MoeArgs& a, hipStream_t s) {
  if (int8)
    return kind == 0   ? moe_up<Int8<F32>>(a, values, s)
           : kind == 1 ? moe_up<Int8<F16>>(a, values, s)
                       : moe_up<Int8<BF16>>(a, values, s);
  return kind == 0 ? moe_up<F32>(a, false, s) : kind == 1 ? moe_up<F16>(a, false, s) : moe_up<BF16>(a, false, s);
}
hipError_t launch_moe_down(int kind, bool int8, bool values, const MoeArgs& a, hipStream_t s) {
  if (int8)
    return kind == 0   ? moe_down<Int8<F32>>(a, values, s)
           : kind == 1 ? moe_down<Int8<F16>>(a, values, s)
                       : moe_down<Int8<BF16>>(a, values, s);
  return kind == 0 ? moe_down<F32>(a, false, s) : kind == 1 ? moe_down<F16>(a, false, s) : moe_down<BF16>(a, false, s);
}

}  // namespace llar_ffn
