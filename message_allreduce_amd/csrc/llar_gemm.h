// llar_gemm.h -- the matrix product of the feed-forward operators on the
// gfx950 matrix units.  See llar_ffn.h for what one launch computes.
#pragma once
#include "llar_ffn.h"
#include "llar_ffn_math.h"

namespace llar_ffn {

#define LLAR_LDS __attribute__((address_space(3)))
typedef LLAR_LDS char lds_char;

constexpr uint32_t kNoLoad = 0x80000000u;  // beyond every descriptor: the load writes zeros

// A TM x TN tile by WM x WN waves; kGroups such groups of waves take the k
// tiles in turn, each with its own buffers, and their sums are joined in LDS:
// more waves where there are few tiles, without a second kernel.
template <int TM_, int TN_, int WM_, int WN_, int G_>
struct TileShape {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, kGroups = G_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;  // of a group
  static constexpr int kAllThreads = kThreads * kGroups;
  static constexpr int FM = TM / WM / 16;  // 16-row fragments of a wave along m
  static constexpr int FN = TN / WN / 16;  // and along n
  static constexpr bool kPaired = WM == 2 && WN == 4;
  // tile buffers of a group: what the CU's LDS holds, four at most
  static constexpr int kStages = kPaired || (TM > 64 && TN > 64) || G_ == 4 ? 2 : TM > 64 ? 3 : 4;
};
typedef TileShape<256, 256, 2, 4, 1> Shape256;
template <int G>
using Shape128 = TileShape<128, 128, 2, 2, G>;
typedef TileShape<128, 64, 2, 2, 2> Shape128x64;
template <int G>
using Shape64 = TileShape<64, 64, 2, 2, G>;

// ---- fragments -------------------------------------------------------------------
// A 16 x 32 operand fragment: lane l holds row l % 16, k = 8 (l / 16) .. + 7.
template <class E>
struct Frag {
  s16x8 v;
};
// binary32 as three bfloat16 whose sum is the value: each part is what the parts
// before it leave, rounded to 8 bits.  Every remainder is exact, and 8 bits at
// most are left for the third part, which is cut (below 2^-110 a value's last
// bits are less than a bfloat16 can hold, and up to 2^-133 is lost).  Rounding by
// an addition: the conversion instruction measured four times an ordinary one.
// A value that rounds to infinity leaves a NaN, as an infinity does (sum_again).
template <>
struct Frag<F32> {
  s16x8 hi, mid, lo;
};

template <class E>
__device__ __forceinline__ f32x4 mma(const Frag<E>& a, const Frag<E>& b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mma<BF16>(const Frag<BF16>& a, const Frag<BF16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c,
                                                 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mma<F16>(const Frag<F16>& a, const Frag<F16>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a.v), __builtin_bit_cast(f16x8, b.v), c, 0,
                                                0, 0);
}
// 16 x 64 fragments of 8-bit numbers: lane l holds row l % 16, k = 16 (l / 16) ..
// + 15, the same bytes of a row as 16-bit lanes hold.  c's bits are integers'.
#define LLAR_MMA_INT8(Out) \
  template <> \
  __device__ __forceinline__ f32x4 mma<Int8<Out>>(const Frag<Int8<Out>>& a, const Frag<Int8<Out>>& b, f32x4 c) { \
    return mma_int8(a.v, b.v, c); \
  }
__device__ __forceinline__ f32x4 mma_int8(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                                         __builtin_bit_cast(i32x4, b),
                                                                         __builtin_bit_cast(i32x4, c), 0, 0, 0));
}
LLAR_MMA_INT8(F32)
LLAR_MMA_INT8(F16)
LLAR_MMA_INT8(BF16)

// Six of the nine products of parts, small ones first: 6 bfloat16 products at 16
// times the binary32 unit's rate.  mid is at most 2^-8 of its value and lo 2^-17,
// so the three left out are at most 2^-24 of the whole, as much as binary32
// rounds a product by, and of either sign.  Parts cut and not rounded leave up to
// 2^-21 out, all towards zero, for 3 to 5 % less time (4096^3 618 against 647 us).
__device__ __forceinline__ f32x4 mma_part(int s, const Frag<F32>& a, const Frag<F32>& b, f32x4 c) {
  const s16x8 p = s == 0 || s == 3 ? a.mid : s == 1 ? a.lo : a.hi;
  const s16x8 q = s == 0 || s == 4 ? b.mid : s == 2 ? b.lo : b.hi;
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c, 0, 0,
                                                 0);
}
template <>
__device__ __forceinline__ f32x4 mma<F32>(const Frag<F32>& a, const Frag<F32>& b, f32x4 c) {
#pragma unroll
  for (int s = 0; s < 6; s++) c = mma_part(s, a, b, c);
  return c;
}

// The upper halves of two words, a's lower.
__device__ __forceinline__ uint32_t upper_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302);
}
// The value rounded to its leading 8 bits: the nearest such, up at halfway.
__device__ __forceinline__ float leading(uint32_t v) { return __uint_as_float((v + 0x8000u) & 0xffff0000u); }
__device__ __forceinline__ Frag<F32> split3(const float (&x)[8]) {
  union {
    s16x8 v;
    uint32_t u[4];
  } hi, mid, lo;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    float h[2], m[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const float v = x[2 * i + e];
      h[e] = leading(__float_as_uint(v));
      const float r = v - h[e];
      m[e] = leading(__float_as_uint(r));
      l[e] = r - m[e];
    }
    hi.u[i] = upper_halves(__float_as_uint(h[0]), __float_as_uint(h[1]));
    mid.u[i] = upper_halves(__float_as_uint(m[0]), __float_as_uint(m[1]));
    lo.u[i] = upper_halves(__float_as_uint(l[0]), __float_as_uint(l[1]));
  }
  Frag<F32> f;
  f.hi = hi.v;
  f.mid = mid.v;
  f.lo = lo.v;
  return f;
}

// ---- one 16-bit (or 8-bit) operand's tile in LDS ----------------------------------------
// R rows by 64 k (128), in one of two orders.
//
// k-contiguous source: [row][8 chunks of 16 bytes], chunk c of a row stored at
// position c ^ key(row), so that the 16 rows of a fragment read the same chunk
// from different banks.
// Row-contiguous source: [k][row], chunk c of a k line stored at c ^ key(k);
// fragments come out through the transposing LDS read, which gathers four k of
// one row into a lane.
//
// perm: fragment j's 16 rows are spread over the wave's rows as
// n = 4 F b + 4 j + i (b, i = 0..3, F fragments in a run), so that a lane's
// results of the run are 4 F neighbours of one output row.  Only the
// k-contiguous order is read that way; the other keeps n = 16 j + r.
template <class E, bool kRows, int R, int NT, int F, bool kPerm>
struct Operand {
  static constexpr bool kByRows = kRows, kSpread = kPerm;
  static constexpr int kRun = F;
  static constexpr int kThreads = NT;
  static constexpr int ES = sizeof(typename E::X);
  static constexpr int CE = 16 / ES;          // elements of a chunk
  static constexpr int BK = 128 / ES;         // k of a tile
  static constexpr int kBytes = R * 128;
  static constexpr int kLoads = R * 8 / NT;   // chunks a thread loads
  static_assert(R * 8 % NT == 0, "whole chunks per thread");
  static constexpr int kLine = R / CE;        // chunks of a k line (row-contiguous order)

  static __device__ __forceinline__ int key_row(int row) {
    return kPerm ? (row & 3) | (((row / (4 * F)) & 1) << 2) : row & 7;
  }
  static __device__ __forceinline__ int key_k(int k) {
    return 2 * (((k & 3) | (((k >> 3) & 1) << 2)) & (kLine / 2 - 1));
  }

  // chunk number of load i of this thread, in LDS order
  static __device__ __forceinline__ int slot(int i) { return i * NT + (int)(threadIdx.x % NT); }
  // its row (or first row) and its k (or first k) within the tile
  static __device__ __forceinline__ void where(int i, int& row, int& k) {
    const int s = slot(i);
    if constexpr (kRows) {
      k = s / kLine;
      row = ((s % kLine) ^ key_k(k)) * CE;
    } else {
      row = s / 8;
      k = ((s % 8) ^ key_row(row)) * CE;
    }
  }
};

// Waits until at most n of this wave's loads are on their way; they arrive in order.
template <int n>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}

// This thread's byte offsets from the tile's first element, kNoLoad where the
// row does not exist.
template <class Op>
__device__ __forceinline__ void direct_offsets(uint32_t (&voff)[Op::kLoads], int rows_left, int64_t ld) {
#pragma unroll
  for (int i = 0; i < Op::kLoads; i++) {
    int row, k;
    Op::where(i, row, k);
    const int64_t at = Op::kByRows ? k * ld + row : row * ld + k;
    voff[i] = row < rows_left ? (uint32_t)(at * Op::ES) : kNoLoad;
  }
}

// Loads 16 bytes a lane from base + off straight into LDS, the wave's 64 chunks
// back to back from `at`.  The compiler would count these loads against every
// later LDS read and wait for all of them; written as assembly they are this
// code's own to wait for (wait_loads).  They have no result registers.
__device__ __forceinline__ u32x4 describe(int64_t base) {
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)base),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(base >> 32)) & 0xffffu, 0x7fffffffu, 0x00020000u};
}
// m0 is declared, so that a value that the compiler keeps there for a use of its
// own is set again (it warns that it does not save it across the statement).
__device__ __forceinline__ void load_chunks(uint32_t at, uint32_t off, u32x4 desc) {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at),
      "v"(off), "s"(desc)
      : "memory", "m0");
#pragma clang diagnostic pop
}

// A whole tile that way.  krem: how many k of it exist.
template <class Op>
__device__ __forceinline__ void load_direct(lds_char* lds, int64_t base, const uint32_t (&voff)[Op::kLoads],
                                            int krem) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x % Op::kThreads >> 6);
  const u32x4 desc = describe(base);
  const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds + wave * 1024);
#pragma unroll
  for (int i = 0; i < Op::kLoads; i++) {
    int row, k;
    Op::where(i, row, k);
    load_chunks(at + i * (Op::kThreads * 16), k < krem ? voff[i] : kNoLoad, desc);
  }
}

// The lane's address of fragment 0 (first tile row `row0`), k step 0.
template <class Op>
__device__ __forceinline__ uint32_t frag_base(int row0) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  if constexpr (Op::kByRows) {
    const int k = q * 8 + (r >> 2), col = row0 + (r & 3) * 4;
    return (k * Op::kLine + ((col / 8) ^ Op::key_k(k))) * 16 + (col % 8) * 2;
  } else {
    const int row = row0 + (Op::kSpread ? (r >> 2) * 4 * Op::kRun + (r & 3) : r);
    return row * 128 + (q ^ Op::key_row(row)) * 16;
  }
}

// Fragment f (a constant after unrolling) of k step kk.
template <class Op, class E>
__device__ __forceinline__ Frag<E> read_frag(lds_char* lds, uint32_t base, int f, int kk) {
  Frag<E> out;
  if constexpr (Op::kByRows) {
    // lane i of 16 hands in row i / 4 of a 4 x 16 block and takes column i
    const uint32_t at = (base ^ (f * 32)) + kk * 32 * Op::kLine * 16;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LLAR_LDS s16x4*)(lds + at));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LLAR_LDS s16x4*)(lds + at + 4 * Op::kLine * 16));
    out.v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const uint32_t step = Op::kSpread ? 4 * 128 : 16 * 128;
    out.v = *(LLAR_LDS s16x8*)(lds + ((base ^ (kk * 64)) + f * step));
  }
  return out;
}

// What a whole sum stands for: three roundings of binary32.  The weight's scale, an
// ordinary number, comes first: a token's may be as large or as small as its values.
__device__ __forceinline__ float scaled(int sum, float xs, float ws) { return (float)sum * ws * xs; }

// Applies the epilogue to n neighbours of one output row and stores them.
// acc0: the sums (gated: of the first projection), acc1: of the second.
template <class E, bool kGated, int n>
__device__ __forceinline__ void finish(const GemmArgs& a, int b, int m, int col, const float* acc0,
                                       const float* acc1) {
  typedef typename E::T T;
  const int cnt = a.N - col;
  float y[n];
  if constexpr (kGated) {
    if (a.z[0]) {
      store_vals<E, n>((T*)a.z[0] + m * a.zld + col, acc0, cnt);
      store_vals<E, n>((T*)a.z[1] + m * a.zld + col, acc1, cnt);
    }
#pragma unroll
    for (int i = 0; i < n; i++) y[i] = acc0[i];
    act_values<E, n>(y, a.act);
#pragma unroll
    for (int i = 0; i < n; i++) y[i] *= acc1[i];
  } else {
#pragma unroll
    for (int i = 0; i < n; i++) y[i] = acc0[i];
    if (a.bias) {
      const Vals<E, n> v = load_vals<E, n>((const T*)a.bias + col, cnt);
#pragma unroll
      for (int i = 0; i < n; i++) y[i] += v.v[i];
    }
    if (a.z[0]) store_vals<E, n>((T*)a.z[0] + m * a.zld + col, y, cnt);
    act_values<E, n>(y, a.act);
    if (a.resid) {
      const Vals<E, n> v = load_vals<E, n>((const T*)a.resid + m * a.rld + col, cnt);
#pragma unroll
      for (int i = 0; i < n; i++) y[i] += v.v[i];
    }
  }
  store_vals<E, n>((T*)a.out[b] + m * a.outld + col, y, cnt);
}

// The product of parts turns an infinity into a NaN (infinity times a zero
// part, or infinity less infinity in a remainder), and a part rounded up may
// overflow where its value does not.  So a sum of binary32 inputs that is not
// finite is taken again from the inputs, in k order, up to the first true NaN.
// One lane a sum, 16 terms fetched together, which is slow next to the matrix
// units: with an infinity in one row of x, 512 x 2048 x 2048 takes 73 us instead of
// 33 (one term at a time 380), 4096^3 880 instead of 645.
__device__ __forceinline__ bool not_finite(float s) { return !(fabsf(s) < __builtin_inff()); }
template <bool kXRows, bool kWRows>
__device__ __forceinline__ float sum_again(const GemmArgs& a, int b, int p, int m, int col, int64_t k0, int64_t k1) {
  constexpr int U = 16;
  const int64_t xstep = kXRows ? a.xld : 1, wstep = kWRows ? a.wld : 1;
  const bool two = a.segs == 2;
  float s = 0.f;
  for (int seg = two ? 0 : b; seg <= (two ? 1 : b); seg++) {
    const int64_t before = two ? (int64_t)seg * a.K : 0;  // terms of the pairs before this one
    const int64_t end = two ? min(k1 - before, (int64_t)a.K) : k1;
    int64_t k = max(k0 - before, (int64_t)0);
    const float* x = (const float*)a.x[seg] + (kXRows ? m : m * a.xld);
    const float* w = (const float*)a.w[two || a.batch == 2 ? seg : p] + (kWRows ? col : col * a.wld);
#pragma clang loop unroll(disable)
    for (; k + U <= end && s == s; k += U) {
      float xv[U], wv[U];
#pragma unroll
      for (int i = 0; i < U; i++) {
        xv[i] = x[(k + i) * xstep];
        wv[i] = w[(k + i) * wstep];
      }
#pragma unroll
      for (int i = 0; i < U; i++) s = fmaf(xv[i], wv[i], s);
    }
#pragma clang loop unroll(disable)
    for (; k < end && s == s; k++) s = fmaf(x[k * xstep], w[k * wstep], s);
  }
  return s;
}

// Whether the residual can be in a sum from its start: begin (or the quarters)
// and store_results both ask here, so that exactly one of them adds it.
__device__ __forceinline__ bool starts_with_resid(const GemmArgs& a) {
  return a.resid && a.splits == 1 && !a.z[0] && a.act == kActNone;
}

// ---- results -------------------------------------------------------------------------
// The tile (m0, n0) of plane b: acc[part of x][part of w][fragment of x][of w].
// kSumsBegun: they began with the bias, and with the residual where nothing
// comes between (starts_with_resid), for either order of w.
template <class E, bool kXRows, bool kWRows, bool kGated, class Shape, int kXParts, int kWParts, bool kSpread, int kLds,
          bool kSumsBegun, int FX, int FW>
__device__ __forceinline__ void store_results(const GemmArgs& a, f32x4 (&acc)[kXParts][kWParts][FX][FW], lds_char* lds,
                                              int m0, int n0, int b, int split, int ktiles, int t0, int t1, int bk) {
  // of fragments (f, j) lane l holds row l % 16 and 4 neighbouring
  // columns.  Bare sums (a gradient, a partial plane, a product without
  // epilogue) are stored from there; everything else goes through LDS, where a
  // lane takes 8 columns of one row, so that the epilogue is one piece of code
  // and its accesses are whole lines.
  typedef typename E::T T;
  constexpr int P = kGated ? 2 : 1;
  constexpr int kXRowsPart = Shape::TM / kXParts, kWRowsPart = Shape::TN / kWParts;
  constexpr int kWStep = kGated ? 0 : kWRowsPart;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / Shape::WN, wn = wave % Shape::WN;
  const int mwave = m0 + wm * 16 * FX, nwave = n0 + wn * 16 * FW;
  const bool add_bias = !kGated && !kSumsBegun && a.bias;
  const bool add_resid = !kGated && a.resid && a.splits == 1 && !(kSumsBegun && starts_with_resid(a));
  bool bare = !kGated && kSpread &&
              (a.splits > 1 || (!a.z[0] && a.act == kActNone && !add_bias && !add_resid));
  bool again = false;
  if constexpr (E::kParts) {
#pragma unroll
    for (int h = 0; h < kXParts; h++)
#pragma unroll
      for (int p = 0; p < kWParts; p++)
#pragma unroll
        for (int f = 0; f < FX; f++)
#pragma unroll
          for (int j = 0; j < FW; j++) {
            const f32x4 c = acc[h][p][f][j];
            const float s = (c[0] + c[1]) + (c[2] + c[3]);
            again = again || not_finite(s);
          }
    again = __any(again);
    bare = bare && !again;
  }
  if (bare) {
    constexpr int kRunLen = kSpread ? (4 * FW < 8 ? 4 * FW : 8) : 4;
#pragma unroll
    for (int h = 0; h < kXParts; h++)
#pragma unroll
      for (int f = 0; f < FX; f++) {
        const int m = mwave + h * kXRowsPart + f * 16 + (lane & 15);
#pragma unroll
        for (int p = 0; p < kWParts; p++)
#pragma unroll
          for (int j = 0; j < FW; j += kRunLen / 4) {
            const int col = nwave + p * kWStep + (kSpread ? q * 4 * FW + 4 * j : 16 * j + 4 * q);
            if (m < a.M && col < a.N) {
              if (a.splits > 1) {
                float* d = a.partial + (((int64_t)split * a.batch + b) * a.M + m) * a.npad + col;
#pragma unroll
                for (int i = 0; i < kRunLen / 4; i++)
                  if (col + 4 * i < a.npad) *(f32x4*)(d + 4 * i) = acc[h][p][f][j + i];
              } else {
                float v[kRunLen];
#pragma unroll
                for (int i = 0; i < kRunLen; i++) v[i] = acc[h][p][f][j + i / 4][i % 4];
                store_vals<E, kRunLen>((T*)a.out[b] + m * a.outld + col, v, a.N - col);
              }
            }
          }
      }
    return;
  }
  // half of the wave's rows at a time (a part of x, or half of its one);
  // 16-byte chunk c of a row lies at c ^ row % 16
  constexpr int kCols = 16 * FW * kWParts, kHalf = kXParts * FX / 2, kRows = kHalf * 16;
  static_assert(Shape::kWaves * kRows * kCols * 4 <= kLds, "the waves' sums fit the tile buffers");
  lds_char* mine = lds + wave * (kRows * kCols * 4);
  auto chunk = [&](int row, int c) {
    return (LLAR_LDS f32x4*)(mine + (row * (kCols / 4) + (c ^ (row % 16 % (kCols / 4)))) * 16);
  };
  auto k_of = [&](int t) { return (int64_t)(t / ktiles) * a.K + min((t % ktiles) * bk, a.K); };
  auto settle = [] {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  __syncthreads();  // everyone is done with the tiles
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int mhalf = mwave + (kXParts == 2 ? h * kXRowsPart : h * kRows);
#pragma unroll
    for (int i = 0; i < kHalf; i++)
#pragma unroll
      for (int p = 0; p < kWParts; p++)
#pragma unroll
        for (int j = 0; j < FW; j++) {
          constexpr int kPer = kXParts == 2 ? 0 : kHalf;  // fragments of x before this half's in its part
          *chunk(i * 16 + (lane & 15), p * 4 * FW + (kSpread ? q * FW + j : 4 * j + q)) =
              acc[kXParts == 2 ? h : 0][p][i + h * kPer][j];
        }
    settle();
    if constexpr (E::kParts) {
      // most calls have no such sum: the wave looks before it goes through them
      if (again) {
#pragma clang loop unroll(disable)
        for (int i = lane; i < kRows * kCols; i += 64) {
          const int row = i / kCols, c = i % kCols, p = c / (16 * FW);
          const int m = mhalf + row, col = nwave + p * kWStep + c % (16 * FW);
          LLAR_LDS float* v = (LLAR_LDS float*)chunk(row, c / 4) + c % 4;
          if (not_finite(*v) && m < a.M && col < a.N)
            *v = sum_again<kXRows, kWRows>(a, b, kGated ? p : 0, m, col, k_of(t0), k_of(t1));
        }
        settle();
      }
    }
    // A lane takes the same 8 columns of every row it comes to (gated: of both
    // projections), two rows at a time so that their chains overlap.
    constexpr int kRuns = 2 * FW * (kGated ? 1 : kWParts), kPieces = kRows * kRuns, kStride = 64 / kRuns;
    constexpr int U = kPieces >= 128 && E::kind != 0 ? 2 : 1;  // binary32: a second workgroup must fit the registers
    static_assert(64 % kRuns == 0, "whole rows a wave");
    const int c = lane % kRuns, col = nwave + c / (2 * FW) * kWStep + 8 * (c % (2 * FW));
    const int cnt = a.N - col;
    auto row_of = [&](int i) { return lane / kRuns + i * kStride; };
    // The residual comes from memory: pieces ahead of their use, or a tile pays
    // that latency for each.
    typedef typename Wide<E, 8>::vec piece;
    const bool queue = add_resid && cnt >= 8;
    auto peek = [&](int i) {
      piece v = {};
      if (queue && row_of(i) < kRows && mhalf + row_of(i) < a.M)
        v = *(const typename Wide<E, 8>::loose*)((const T*)a.resid + (mhalf + row_of(i)) * a.rld + col);
      return v;
    };
    piece next[U];
#pragma unroll
    for (int u = 0; u < U; u++) next[u] = peek(u);
    Vals<E, 8> bias = {};
    if (add_bias && cnt > 0) bias = load_vals<E, 8>((const T*)a.bias + col, cnt);
#pragma clang loop unroll(disable)
    for (int i = 0; i * kStride < kRows; i += U) {
      piece now[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        now[u] = next[u];
        next[u] = peek(i + U + u);
      }
      float v[P][8 * U];
#pragma unroll
      for (int u = 0; u < U; u++)
#pragma unroll
        for (int p = 0; p < P; p++) {
          const int row = row_of(i + u) % kRows;  // a wave with fewer pieces than lanes comes back to the first
          const f32x4 lo = *chunk(row, p * 4 * FW + 2 * c), hi = *chunk(row, p * 4 * FW + 2 * c + 1);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            v[p][8 * u + e] = lo[e];
            v[p][8 * u + 4 + e] = hi[e];
          }
        }
      bool live[U];
      int64_t m[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        m[u] = mhalf + row_of(i + u);
        live[u] = row_of(i + u) < kRows && m[u] < a.M && cnt > 0;
      }
      if (a.splits > 1) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
          for (int p = 0; p < P; p++) {
            if (!live[u]) continue;
            float* d = a.partial + (((int64_t)split * (kGated ? 2 : a.batch) + (kGated ? p : b)) * a.M + m[u]) * a.npad + col;
            const float* s = &v[p][8 * u];
            *(f32x4*)d = f32x4{s[0], s[1], s[2], s[3]};
            *(f32x4*)(d + 4) = f32x4{s[4], s[5], s[6], s[7]};
          }
        continue;
      }
      if constexpr (!kSumsBegun && !kGated) {
#pragma unroll
        for (int e = 0; e < 8 * U; e++) v[0][e] += bias.v[e % 8];
      }
      if (a.z[0]) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
          for (int p = 0; p < P; p++)
            if (live[u]) store_vals<E, 8>((T*)a.z[p] + m[u] * a.zld + col, &v[p][8 * u], cnt);
      }
      act_values<E, 8 * U>(v[0], a.act);
      if constexpr (kGated) {
#pragma unroll
        for (int e = 0; e < 8 * U; e++) v[0][e] *= v[P - 1][e];
      } else if (add_resid) {
#pragma unroll
        for (int u = 0; u < U; u++) {
          Vals<E, 8> r;
#pragma unroll
          for (int e = 0; e < 8; e++) r.v[e] = E::to(now[u][e]);
          if (!queue && live[u]) r = load_vals<E, 8>((const T*)a.resid + m[u] * a.rld + col, cnt);
#pragma unroll
          for (int e = 0; e < 8; e++) v[0][8 * u + e] += r.v[e];
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++)
        if (live[u]) store_vals<E, 8>((T*)a.out[b] + m[u] * a.outld + col, &v[0][8 * u], cnt);
    }
    settle();
  }
}

// Adds the groups' sums, in their order, into the first group's; false for the
// others, which are done.
template <class E, class Shape, int kLds, int A, int B, int FX, int FW>
__device__ __forceinline__ bool join_groups(f32x4 (&acc)[A][B][FX][FW], lds_char* lds) {
  constexpr int G = Shape::kGroups, kFrags = A * B * FX * FW;
  if constexpr (G == 1) return true;
  static_assert((G - 1) * kFrags * Shape::kThreads * 16 <= kLds, "the groups' sums fit the tile buffers");
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / Shape::kThreads), t = threadIdx.x % Shape::kThreads;
  f32x4(&flat)[kFrags] = reinterpret_cast<f32x4(&)[kFrags]>(acc);
  __syncthreads();
  if (group > 0) {
#pragma unroll
    for (int i = 0; i < kFrags; i++)
      *(LLAR_LDS f32x4*)(lds + (((group - 1) * kFrags + i) * Shape::kThreads + t) * 16) = flat[i];
  }
  __syncthreads();
  if (group > 0) return false;
#pragma unroll
  for (int g = 0; g < G - 1; g++)
#pragma unroll
    for (int i = 0; i < kFrags; i++) {
      const f32x4 v = *(LLAR_LDS f32x4*)(lds + ((g * kFrags + i) * Shape::kThreads + t) * 16);
#pragma unroll
      for (int e = 0; e < 4; e++) {
        if constexpr (E::kInt8)
          flat[i][e] = __int_as_float(__float_as_int(flat[i][e]) + __float_as_int(v[e]));
        else
          flat[i][e] += v[e];
      }
    }
  return true;
}

// Which tile, plane and share of the k tiles workgroup `wg` of a product's
// `total` takes: those with the same wg % 8 run on one XCD; it takes a run of
// neighbouring tiles, in groups of 8 along m, so that its L2 holds what they share.
struct Place {
  int m0, n0, b, split, ktiles, t0, t1;
};
template <int TM, int TN>
__device__ __forceinline__ Place place(const GemmArgs& a, int BK, int wg, int total) {
  Place o;
  const int tm = (a.M + TM - 1) / TM, tn = (a.N + TN - 1) / TN;
  const int xcd = wg & 7, share = total >> 3, extra = total & 7;
  int id = xcd * share + (xcd < extra ? xcd : extra) + (wg >> 3);
  const int tiles = tm * tn;
  const int plane = id / tiles;
  id -= plane * tiles;
  o.b = plane % a.batch;
  o.split = plane / a.batch;
  const int group = id / (8 * tn), in = id - group * 8 * tn;
  const int gm = min(tm - group * 8, 8);
  o.m0 = (group * 8 + in % gm) * TM;
  o.n0 = in / gm * TN;
  o.ktiles = (a.K + BK - 1) / BK;
  const int64_t all = (int64_t)o.ktiles * a.segs;
  o.t0 = (int)(all * o.split / a.splits);
  o.t1 = (int)(all * (o.split + 1) / a.splits);
  return o;
}

// One workgroup computes a TM x TN tile of the output (gated: TM x TN/2 of both
// projections) over its share of the k tiles.  While a tile is multiplied the
// next ones' loads are on their way to the other LDS buffers.
//
// The tile's rows of w lie in LDS as kWParts operands (gated: one for each
// projection), those of x as kXParts; a wave owns FX fragments of every part
// of x and FW of every part of w.
//
// Which tile: a 256 x 256 one reads 12 KB of fragments a wave for 32 matrix
// instructions and keeps them 80 % busy at the clock that power leaves (8192^3
// bf16 1480 TF, of 1850 there), but 256 CUs want 256 tiles.  The smaller ones are
// bound by LDS reads (64 x 64: 4 KB for 4), then by their first loads; the
// groups of waves bring the waves that few tiles lack.  bf16, us, 256 / 128 /
// 128 x 64 / 64, best groups: 4096 x 2048 x 8192 119 / 130 / 171 / -, 2048 x 2048 x 2048
// 40 / 24 / 26 / 33, 1024 x 2048 x 2048 - / 21 / 16 / 18, 128 x 2048 x 2048 - / - / 13 / 10.5.
template <class Shape>
constexpr int kGemmLds = Shape::kGroups * Shape::kStages * (Shape::TM + Shape::TN) * 128;
// Room behind it: 8-bit operands' scales; the large tile's for a quarter of every
// wave's residual (kLater).
template <class E, class Shape>
constexpr int kScaleLds = E::kInt8 ? (Shape::TM + Shape::TN) * 4 : 0;
constexpr int kResidLds = 8 * 64 * 32 * 2;

template <class E, bool kXRows, bool kWRows, class Shape, bool kGated, bool kLater>
__device__ __forceinline__ void gemm_body(const GemmArgs& a, char* smem, int wg, int total) {
  typedef typename E::T T;
  constexpr bool kPaired = Shape::kPaired;
  constexpr int TM = Shape::TM, NT = Shape::kThreads;
  constexpr int P = kGated ? 2 : 1;              // projections
  constexpr int TN = Shape::TN / P;              // output columns of the tile
  constexpr int kXParts = kPaired ? 2 : 1, kWParts = kPaired ? 2 : P;
  constexpr int FX = Shape::FM / kXParts, FW = Shape::FN / kWParts;
  constexpr int kXRowsPart = TM / kXParts, kWRowsPart = Shape::TN / kWParts;
  constexpr int kWStep = kGated ? 0 : kWRowsPart;  // columns from one part of w to the next
  constexpr bool kSpread = !kWRows;
  typedef Operand<E, kXRows, kXRowsPart, NT, FX, false> X;
  typedef Operand<E, kWRows, kWRowsPart, NT, FW, kSpread> W;
  constexpr int BK = X::BK, ES = X::ES;
  constexpr int kBuf = kXParts * X::kBytes + kWParts * W::kBytes;
  constexpr int kStages = Shape::kStages;
  constexpr int G = Shape::kGroups;
  static_assert(G * kStages * kBuf == kGemmLds<Shape>, "the kernel's LDS");
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  lds_char* lds = (lds_char*)smem + group * kStages * kBuf;

  const Place at = place<TM, TN>(a, BK, wg, total);
  const int m0 = at.m0, n0 = at.n0, b = at.b, split = at.split, ktiles = at.ktiles, t0 = at.t0, t1 = at.t1;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x % NT >> 6);
  const int wm = wave / Shape::WN, wn = wave % Shape::WN;

  f32x4 acc[kXParts][kWParts][FX][FW];
#pragma unroll
  for (int h = 0; h < kXParts; h++)
#pragma unroll
    for (int p = 0; p < kWParts; p++)
#pragma unroll
      for (int f = 0; f < FX; f++)
#pragma unroll
        for (int j = 0; j < FW; j++) acc[h][p][f][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  uint32_t xoff[kXParts][X::kLoads], woff[kWParts][W::kLoads];
#pragma unroll
  for (int h = 0; h < kXParts; h++) direct_offsets<X>(xoff[h], a.M - m0 - h * kXRowsPart, a.xld);
#pragma unroll
  for (int p = 0; p < kWParts; p++) direct_offsets<W>(woff[p], a.N - n0 - p * kWStep, a.wld);
  const int64_t x1 = (int64_t)a.x[1], w1 = (int64_t)a.w[1];
  const int64_t x0 = b ? x1 : (int64_t)a.x[0], w0 = b ? w1 : (int64_t)a.w[0];
  const int64_t xnext = x1 - x0, wnext = w1 - w0;  // to the second pair's
  const int64_t xpart = (kXRows ? kXRowsPart : kXRowsPart * a.xld) * ES;
  const int64_t wpart = kGated ? wnext : (kWRows ? kWStep : kWStep * a.wld) * ES;
  const int64_t xfirst = kXRows ? m0 : m0 * a.xld, xstep = kXRows ? BK * a.xld : BK;
  const int64_t wfirst = kWRows ? n0 : n0 * a.wld, wstep = kWRows ? BK * a.wld : BK;
  // Neighbouring workgroups start up to three k tiles apart: the rows of a tile
  // can lie so that a k tile of all of them is in a few memory channels (8192 x
  // 8192 x 3584 bf16: 400 -> 333 us, other shapes within 2 %).
  const int shift = (n0 / TN % 4) % max(t1 - t0, 1);
  // k tile t's first elements and how many of its k exist (none beyond the last tile)
  int64_t xat, wat;
  int krem;
  auto aim = [&](int t) {
    const bool exists = t < t1;
    t += shift;
    if (t >= t1) t -= t1 - t0;
    const bool second = a.segs == 2 && t >= ktiles;
    const int kt = second ? t - ktiles : t;
    krem = exists ? a.K - kt * BK : 0;
    xat = x0 + (second ? xnext : 0) + (xfirst + kt * xstep) * ES;
    wat = w0 + (second ? wnext : 0) + (wfirst + kt * wstep) * ES;
  };
  auto load_x = [&](int slot, int h) {
    load_direct<X>(lds + slot * kBuf + h * X::kBytes, xat + h * xpart, xoff[h], krem);
  };
  auto load_w = [&](int slot, int p) {
    load_direct<W>(lds + slot * kBuf + kXParts * X::kBytes + p * W::kBytes, wat + p * wpart, woff[p], krem);
  };

  // The large tile takes the residual in quarters while it multiplies, if every
  // 8 columns of it are an aligned chunk and there are tiles enough (8192 x 8192 x
  // 3584 bf16 398 -> 384 us, x 1024 178 -> 147; without a residual 340 and 122).
  bool later = false;
  if constexpr (kLater)
    later = starts_with_resid(a) && t1 - t0 > 8 && ((a.N | a.rld | ((int64_t)a.resid / 2)) & 7) == 0 && a.rld < 1 << 23;

  // 8-bit operands' scales wait in LDS, behind the tiles: fetched at the end they cost
  // every tile their latency.
  lds_char* const scales = (lds_char*)smem + kGemmLds<Shape>;
  auto fetch_scales = [&] {
    if constexpr (E::kInt8) {
      if (a.splits > 1) return;
      for (int i = threadIdx.x; i < TM + Shape::TN; i += Shape::kAllThreads) {
        const int n = i - TM, p = kGated && n >= TN ? 1 : 0, col = n0 + n - p * TN;
        float v = 0.f;
        if (i < TM) {
          if (m0 + i < a.M) v = a.xscale[m0 + i];
        } else if (col < a.N) {
          v = a.wscale[p][col];
        }
        *(LLAR_LDS float*)(scales + i * 4) = v;
      }
    }
  };

  // The first group's sums start with the bias, and with the residual if only
  // sums follow: its loads then overlap the first tiles', and the results need
  // no pass through LDS (8192 x 8192 x 3584 bf16 with a bias: 361 us, now 334).
  auto begin = [&] {
    if (E::kInt8 || kGated || a.splits > 1 || group > 0) return;
    const int lane = threadIdx.x & 63, q = lane >> 4;
    constexpr int kRunLen = kSpread ? (4 * FW < 8 ? 4 * FW : 8) : 4;
    const bool resid = starts_with_resid(a) && !later;
#pragma unroll
    for (int p = 0; p < kWParts; p++)
#pragma unroll
      for (int j = 0; j < FW; j += kRunLen / 4) {
        const int col = n0 + wn * 16 * FW + p * kWStep + (kSpread ? q * 4 * FW + 4 * j : 16 * j + 4 * q);
        const int cnt = a.N - col;
        Vals<E, kRunLen> bias = {};
        if (a.bias && cnt > 0) bias = load_vals<E, kRunLen>((const T*)a.bias + col, cnt);
#pragma unroll
        for (int h = 0; h < kXParts; h++)
#pragma unroll
          for (int f = 0; f < FX; f++) {
            const int m = m0 + wm * 16 * FX + h * kXRowsPart + f * 16 + (lane & 15);
            Vals<E, kRunLen> r = {};
            if (resid && m < a.M && cnt > 0) r = load_vals<E, kRunLen>((const T*)a.resid + m * a.rld + col, cnt);
#pragma unroll
            for (int i = 0; i < kRunLen; i++) acc[h][p][f][j + i / 4][i % 4] = bias.v[i] + r.v[i];
          }
      }
  };

  const uint32_t xbase = frag_base<X>(wm * 16 * FX), wbase = frag_base<W>(wn * 16 * FW);
  constexpr int KK = BK * ES / 64;
  if constexpr (kPaired) {
    // Two groups of four waves (one a SIMD) take turns: while one multiplies a
    // quarter of its wave tiles (one part of x by one of w), the other reads its
    // next fragments and issues loads.  A barrier ends every half turn; the
    // second group runs half a turn behind.  The quarters go round so that each
    // turn reads one part of one operand, and a tile starts with the part of w
    // that the tile before ended with:
    //   turn 0: x0 wa   turn 1: x0 wb   turn 2: x1 wb   turn 3: x1 wa
    // where turn 0 reads x0, turn 1 wb, turn 2 x1 and turn 3 the next tile's
    // first part of w (wb's registers).  Each turn loads, into the part that
    // the turn before read for the last time, what lies two tiles on, and so
    // has seven turns to arrive.
    Frag<E> xf[FX][KK], wf[2][FW][KK];
    auto read_x = [&](int slot, int h) {
#pragma unroll
      for (int kk = 0; kk < KK; kk++)
#pragma unroll
        for (int f = 0; f < FX; f++) xf[f][kk] = read_frag<X, E>(lds + slot * kBuf + h * X::kBytes, xbase, f, kk);
    };
    auto read_w = [&](int slot, int p) {
#pragma unroll
      for (int kk = 0; kk < KK; kk++)
#pragma unroll
        for (int j = 0; j < FW; j++)
          wf[p][j][kk] = read_frag<W, E>(lds + slot * kBuf + kXParts * X::kBytes + p * W::kBytes, wbase, j, kk);
    };
    auto multiply = [&](int h, int p) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int kk = 0; kk < KK; kk++)
#pragma unroll
        for (int f = 0; f < FX; f++)
#pragma unroll
          for (int j = 0; j < FW; j++) acc[h][p][f][j] = mma<E>(wf[p][j][kk], xf[f][kk], acc[h][p][f][j]);
      __builtin_amdgcn_s_setprio(0);
    };
    auto turn = [] {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    auto read_done = [] { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); };
    static_assert(X::kLoads == W::kLoads, "a turn's loads");
    constexpr int kAhead = 6 * X::kLoads;  // loads of the six turns that may still be on their way
    if (t0 < t1) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        aim(t0 + i);
        load_w(i, i);  // in the order of their use: tile t0 starts with part 0 of w, the next with part 1
        load_x(i, 0);
        load_w(i, 1 - i);
        load_x(i, 1);
      }
      begin();
      fetch_scales();
      wait_loads<kAhead>();
      turn();
      read_w(0, 0);
      read_done();
      turn();
      if (wm == 1) turn();
      // Quarter i of the residual is sent for at tile 2 i, into this wave's own
      // LDS, and added at tile 2 i + 2: eight turns' loads are behind it then, and
      // the waits for those have covered it.  Row r's chunk c lies at c ^ r / 2 % 4.
      auto quarter = [&](auto number) {
        constexpr int i = decltype(number)::value;
        if constexpr (kLater) {
          static_assert(FX == 4 && FW == 2, "a quarter is 64 rows of 4 chunks");
          // kept here: what depends on them would wait in registers through the loop
          int lane = threadIdx.x & 63, my = wave;
          asm volatile("" : "+v"(lane), "+s"(my));
          const int r = lane & 15, q = lane >> 4, wm = my / Shape::WN, wn = my % Shape::WN;
          lds_char* mine = (lds_char*)smem + kGemmLds<Shape> + my * (kResidLds / 8);
          if constexpr (i > 0) {
#pragma unroll
            for (int f = 0; f < FX; f++) {
              const auto v =
                  *(LLAR_LDS typename Wide<E, 8>::vec*)(mine + (f * 16 + r) * 64 + (q ^ (r / 2 % 4)) * 16);
#pragma unroll
              for (int e = 0; e < 8; e++) acc[(i - 1) / 2][(i - 1) % 2][f][e / 4][e % 4] += E::to(v[e]);
            }
            read_done();
          }
          if constexpr (i < 4) {
            const int m = m0 + wm * 16 * FX + i / 2 * kXRowsPart, n = n0 + wn * 16 * FW + i % 2 * kWStep;
            const u32x4 desc = describe((int64_t)a.resid + (m * a.rld + n) * ES);
            const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)mine);
#pragma unroll
            for (int g = 0; g < 4; g++) {
              const int row = g * 16 + lane / 4, c = (lane & 3) ^ (row / 2 % 4);
              load_chunks(to + g * 1024, m + row < a.M && n + c * 8 < a.N ? (row * (uint32_t)a.rld + c * 8) * ES : kNoLoad,
                          desc);
            }
          }
        }
      };
      auto tile = [&](int t, auto first) {
        constexpr int wa = decltype(first)::value, wb = 1 - wa, slot = wa;
        if constexpr (kLater && wa == 0) {
          if (later) {
            if (t == t0) quarter(std::integral_constant<int, 0>());
            if (t == t0 + 2) quarter(std::integral_constant<int, 1>());
            if (t == t0 + 4) quarter(std::integral_constant<int, 2>());
            if (t == t0 + 6) quarter(std::integral_constant<int, 3>());
            if (t == t0 + 8) quarter(std::integral_constant<int, 4>());
          }
        }
        auto ready = [&] {
          wait_loads<kAhead>();
          read_done();
          turn();
        };
        aim(t + 2);
        read_x(slot, 0);
        load_w(slot, wa);
        ready();
        multiply(0, wa);
        turn();
        read_w(slot, wb);
        load_x(slot, 0);
        ready();
        multiply(0, wb);
        turn();
        read_x(slot, 1);
        load_w(slot, wb);
        ready();
        multiply(1, wb);
        turn();
        read_w(1 - slot, wb);  // beyond the last tile: zeros, and not used
        load_x(slot, 1);
        ready();
        multiply(1, wa);
        turn();
      };
      int t = t0;
      for (; t + 1 < t1; t += 2) {
        tile(t, std::integral_constant<int, 0>());
        tile(t + 1, std::integral_constant<int, 1>());
      }
      if (t < t1) tile(t, std::integral_constant<int, 0>());
      if (wm == 0) turn();
      wait_loads<0>();
    } else {
      begin();
      fetch_scales();
    }
  } else {
    // a ring of buffers: all but one are on their way while one is multiplied
    constexpr int S = kStages, kLoads = kXParts * X::kLoads + kWParts * W::kLoads;
    auto load = [&](int t, int slot) {
      aim(t);
#pragma unroll
      for (int p = 0; p < kWParts; p++) load_w(slot, p);
#pragma unroll
      for (int h = 0; h < kXParts; h++) load_x(slot, h);
    };
    // group g takes the tiles t0 + g, t0 + g + G, ...; all groups go round
    // equally often, loading nothing beyond the last tile
    const int rounds = (t1 - t0 + G - 1) / G;
    for (int i = 0; i < S - 1; i++) load(t0 + group + i * G, i);
    begin();
    fetch_scales();
    int slot = 0;
    for (int r = 0; r < rounds; r++) {
      wait_loads<(S - 2) * kLoads>();
      __syncthreads();  // this tile has arrived; everyone is done with the one before
      load(t0 + group + (r + S - 1) * G, slot == 0 ? S - 1 : slot - 1);
      lds_char* tile = lds + slot * kBuf;
      slot = slot == S - 1 ? 0 : slot + 1;
#pragma unroll
      for (int kk = 0; kk < KK; kk++) {
        Frag<E> wf[kWParts][FW];
#pragma unroll
        for (int p = 0; p < kWParts; p++)
#pragma unroll
          for (int j = 0; j < FW; j++)
            wf[p][j] = read_frag<W, E>(tile + kXParts * X::kBytes + p * W::kBytes, wbase, j, kk);
#pragma unroll
        for (int f = 0; f < FX; f++) {
          const Frag<E> xf = read_frag<X, E>(tile, xbase, f, kk);
#pragma unroll
          for (int p = 0; p < kWParts; p++)
#pragma unroll
            for (int j = 0; j < FW; j++) acc[0][p][f][j] = mma<E>(wf[p][j], xf, acc[0][p][f][j]);
        }
      }
    }
    wait_loads<0>();
  }

  if (!join_groups<E, Shape, G * kStages * kBuf>(acc, (lds_char*)smem)) return;
  if constexpr (E::kInt8) {
    // whole sums become values; a share of them is joined with the others' first
    if (a.splits == 1) {
      if (t0 >= t1) __syncthreads();  // no tile's barrier has made the scales visible
      int lane = threadIdx.x & 63;
      asm volatile("" : "+v"(lane));  // what depends on it would wait in registers through the loop
      const int q = lane >> 4;
      float xs[kXParts][FX];
#pragma unroll
      for (int h = 0; h < kXParts; h++)
#pragma unroll
        for (int f = 0; f < FX; f++)
          xs[h][f] = *(LLAR_LDS float*)(scales + (wm * 16 * FX + h * kXRowsPart + f * 16 + (lane & 15)) * 4);
#pragma unroll
      for (int p = 0; p < kWParts; p++)
#pragma unroll
        for (int j = 0; j < FW; j++) {
          const int n = wn * 16 * FW + p * (kGated ? TN : kWStep) + (kSpread ? q * 4 * FW + 4 * j : 16 * j + 4 * q);
          const f32x4 ws = *(LLAR_LDS f32x4*)(scales + (TM + n) * 4);
#pragma unroll
          for (int h = 0; h < kXParts; h++)
#pragma unroll
            for (int f = 0; f < FX; f++)
#pragma unroll
              for (int i = 0; i < 4; i++)
                acc[h][p][f][j][i] = scaled(__float_as_int(acc[h][p][f][j][i]), xs[h][f], ws[i]);
        }
    }
  }
  store_results<E, kXRows, kWRows, kGated, Shape, kXParts, kWParts, kSpread, G * kStages * kBuf, !E::kInt8>(
      a, acc, (lds_char*)smem, m0, n0, b, split, ktiles, t0, t1, BK);
}

template <class E, bool kXRows, bool kWRows, class Shape, bool kGated>
__global__ __launch_bounds__(Shape::kAllThreads) void k_gemm(GemmArgs a) {
  constexpr bool kLater = Shape::kPaired && !kGated && !kWRows && !E::kInt8;
  __shared__ __attribute__((aligned(1024))) char smem[kGemmLds<Shape> + kScaleLds<E, Shape> + (kLater ? kResidLds : 0)];
  gemm_body<E, kXRows, kWRows, Shape, kGated, kLater>(a, smem, blockIdx.x, gridDim.x);
}

// ---- binary32 ----------------------------------------------------------------------
// R rows by 32 k of one operand, as three planes of bfloat16 parts in LDS:
// [plane][row][4 chunks of 8 k], chunk c of a row at c ^ key(row).  A thread
// fetches its share of the tile into registers one tile ahead, and splits it into
// parts when it writes it, once for all the waves that multiply it.
template <bool kRows, int R, int NT, int F, bool kPerm>
struct Parts {
  static constexpr bool kAll = R * 4 >= NT;  // else threads from R * 4 on have no share
  static constexpr int C = kAll ? R * 4 / NT : 1;  // 8-k chunks of a thread (row-contiguous: of neighbouring rows)
  static constexpr int kPlane = R * 64, kBytes = 3 * kPlane;
  static_assert(C == 1 || C == 2 || C == 4, "whole chunks");
  float raw[C][8];

  static __device__ __forceinline__ int key(int row) {
    return kPerm ? ((row >> 1) & 1) | (((row / (4 * F)) & 1) << 1) : (row >> 1) & 3;
  }
  static __device__ __forceinline__ void where(int c, int& row, int& kc) {
    const int t = threadIdx.x % NT;
    if constexpr (kRows) {
      row = t % (R / C) * C + c;
      kc = t / (R / C);
    } else {
      row = (c * NT + t) / 4;
      kc = (c * NT + t) % 4;
    }
  }
  // rows and k that exist, counted from the tile's first
  __device__ __forceinline__ void fetch(int64_t base, int64_t ld, int rows_left, int krem) {
    if (!kAll && threadIdx.x % NT >= R * 4) krem = 0;
    const uint64_t first = (uint32_t)__builtin_amdgcn_readfirstlane((int)base) |
                           (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(base >> 32)) << 32;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)first, (short)0, 0x7fffffff, 0x00020000);
    if constexpr (kRows) {
      int row, kc;
      where(0, row, kc);
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int k = kc * 8 + e;
        const uint32_t off = row < rows_left && k < krem ? (uint32_t)((k * ld + row) * 4) : kNoLoad;
        if constexpr (C == 1) {
          raw[0][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
        } else if constexpr (C == 2) {
          const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0);
          raw[0][e] = __uint_as_float(v[0]);
          raw[1][e] = __uint_as_float(v[1]);
        } else {
          const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
#pragma unroll
          for (int c = 0; c < 4; c++) raw[c][e] = __uint_as_float(v[c]);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; c++) {
        int row, kc;
        where(c, row, kc);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int k = kc * 8 + 4 * h;
          const uint32_t off = row < rows_left && k < krem ? (uint32_t)((row * ld + k) * 4) : kNoLoad;
          const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; e++) raw[c][4 * h + e] = __uint_as_float(v[e]);
        }
      }
    }
  }
  __device__ __forceinline__ void write(lds_char* lds) const {
    if (!kAll && threadIdx.x % NT >= R * 4) return;
#pragma unroll
    for (int c = 0; c < C; c++) {
      int row, kc;
      where(c, row, kc);
      const Frag<F32> f = split3(raw[c]);
      lds_char* at = lds + row * 64 + (kc ^ key(row)) * 16;
      *(LLAR_LDS s16x8*)at = f.hi;
      *(LLAR_LDS s16x8*)(at + kPlane) = f.mid;
      *(LLAR_LDS s16x8*)(at + 2 * kPlane) = f.lo;
    }
  }
  static __device__ __forceinline__ uint32_t frag_at(int row0) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const int row = row0 + (kPerm ? (r >> 2) * 4 * F + (r & 3) : r);
    return row * 64 + (q ^ key(row)) * 16;
  }
  static __device__ __forceinline__ Frag<F32> read(lds_char* lds, uint32_t base, int f) {
    lds_char* at = lds + base + f * (kPerm ? 4 * 64 : 16 * 64);
    Frag<F32> o;
    o.hi = *(LLAR_LDS s16x8*)at;
    o.mid = *(LLAR_LDS s16x8*)(at + kPlane);
    o.lo = *(LLAR_LDS s16x8*)(at + 2 * kPlane);
    return o;
  }
};

// The same product for binary32: one LDS buffer, registers one tile ahead; the
// other workgroups of the CU multiply while this one writes.  Bound by the six
// products (matrix units 61 % busy) and the splitting beside them: 4096^3 647 us (212
// TF), 512 x 2048 x 2048 33 us, 2048^3 89, 128 x 2048 x 2048 17.  us, 128 / 64, best
// groups (with parts cut): 2048 x 2048 x 2048 90 / 110, 512 x 4096 x 2048 56 / 57.
template <class Shape>
constexpr int kGemm32Lds = Shape::kGroups * (Shape::TM + Shape::TN) * 192;

template <bool kXRows, bool kWRows, class Shape, bool kGated>
__device__ __forceinline__ void gemm32_body(const GemmArgs& a, char* smem, int wg, int total) {
  constexpr int TM = Shape::TM, NT = Shape::kThreads, BK = 32;
  constexpr int P = kGated ? 2 : 1;
  constexpr int TN = Shape::TN / P;
  constexpr int FX = Shape::FM, FW = Shape::FN / P;
  typedef Parts<kXRows, TM, NT, FX, false> X;
  typedef Parts<kWRows, TN, NT, FW, true> W;
  constexpr int kBuf = X::kBytes + P * W::kBytes;
  constexpr int G = Shape::kGroups;
  static_assert(G * kBuf == kGemm32Lds<Shape>, "the kernel's LDS");
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  lds_char* lds = (lds_char*)smem + group * kBuf;
  const Place at = place<TM, TN>(a, BK, wg, total);
  const int m0 = at.m0, n0 = at.n0, b = at.b, ktiles = at.ktiles, t0 = at.t0, t1 = at.t1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x % NT >> 6);
  const int wm = wave / Shape::WN, wn = wave % Shape::WN;

  f32x4 acc[1][P][FX][FW];
#pragma unroll
  for (int p = 0; p < P; p++)
#pragma unroll
    for (int f = 0; f < FX; f++)
#pragma unroll
      for (int j = 0; j < FW; j++) acc[0][p][f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t x1 = (int64_t)a.x[1], w1 = (int64_t)a.w[1];
  const int64_t x0 = b ? x1 : (int64_t)a.x[0], w0 = b ? w1 : (int64_t)a.w[0];
  const int64_t xnext = x1 - x0, wnext = w1 - w0;
  const int64_t xfirst = kXRows ? m0 : m0 * a.xld, xstep = kXRows ? BK * a.xld : BK;
  const int64_t wfirst = kWRows ? n0 : n0 * a.wld, wstep = kWRows ? BK * a.wld : BK;
  X xr;
  W wr[P];
  auto fetch = [&](int t) {
    const bool second = a.segs == 2 && t >= ktiles;
    const int kt = second ? t - ktiles : t;
    const int krem = t < t1 ? a.K - kt * BK : 0;
    xr.fetch(x0 + (second ? xnext : 0) + (xfirst + kt * xstep) * 4, a.xld, a.M - m0, krem);
#pragma unroll
    for (int p = 0; p < P; p++)
      wr[p].fetch(w0 + (second || p ? wnext : 0) + (wfirst + kt * wstep) * 4, a.wld, a.N - n0, krem);
  };
  const uint32_t xbase = X::frag_at(wm * 16 * FX), wbase = W::frag_at(wn * 16 * FW);
  // group g takes the tiles t0 + g, t0 + g + G, ...; the second half of the
  // groups runs half a round behind, splitting while the first half multiplies
  const int rounds = (t1 - t0 + G - 1) / G;
  const bool late = group >= (G + 1) / 2;
  fetch(t0 + group);
  if (late) __syncthreads();
  for (int r = 0; r < rounds; r++) {
    __syncthreads();  // everyone is done with the tile before
    xr.write(lds);
#pragma unroll
    for (int p = 0; p < P; p++) wr[p].write(lds + X::kBytes + p * W::kBytes);
    fetch(t0 + group + (r + 1) * G);
    __syncthreads();
    Frag<F32> wf[P][FW];
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
      for (int j = 0; j < FW; j++) wf[p][j] = W::read(lds + X::kBytes + p * W::kBytes, wbase, j);
#pragma unroll
    for (int f = 0; f < FX; f++) {
      const Frag<F32> xf = X::read(lds, xbase, f);
      // small products first; neighbours in the sequence have different sums
#pragma unroll
      for (int s = 0; s < 6; s++)
#pragma unroll
        for (int p = 0; p < P; p++)
#pragma unroll
          for (int j = 0; j < FW; j++) acc[0][p][f][j] = mma_part(s, wf[p][j], xf, acc[0][p][f][j]);
    }
  }
  if (G > 1 && !late) __syncthreads();
  if (!join_groups<F32, Shape, G * kBuf>(acc, (lds_char*)smem)) return;
  store_results<F32, kXRows, kWRows, kGated, Shape, 1, P, true, G * kBuf, false>(a, acc, (lds_char*)smem, m0, n0, b, at.split,
                                                                        ktiles, t0, t1, BK);
}

template <bool kXRows, bool kWRows, class Shape, bool kGated>
__global__ __launch_bounds__(Shape::kAllThreads) void k_gemm32(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[kGemm32Lds<Shape>];
  gemm32_body<kXRows, kWRows, Shape, kGated>(a, smem, blockIdx.x, gridDim.x);
}

// Both products of a backward pass in one launch, the one with more k a tile
// first: the other's tiles fill the CUs as they come free, so the pass has one
// last round that is not full, not two, and one launch less (against two
// launches: gated bf16 2394 x 1920 x 2240 129 -> 96 us, fp16 90 x 2560 x 1280
// 18 -> 13, 44 random sizes 9 % on average).
template <class E, bool kWRows, class Shape>
__global__ __launch_bounds__(Shape::kAllThreads) void k_gemm_pair(PairArgs a) {
  constexpr bool k32 = E::kind == 0;
  __shared__ __attribute__((aligned(1024))) char smem[k32 ? kGemm32Lds<Shape> : kGemmLds<Shape>];
  const bool later = (int)blockIdx.x >= a.first;
  const int wg = later ? blockIdx.x - a.first : blockIdx.x, total = later ? gridDim.x - a.first : a.first;
  if (later == a.dw_first) {
    if constexpr (k32)
      gemm32_body<false, kWRows, Shape, false>(a.dx, smem, wg, total);
    else
      gemm_body<E, false, kWRows, Shape, false, false>(a.dx, smem, wg, total);
  } else {
    if constexpr (k32)
      gemm32_body<true, true, Shape, false>(a.dw, smem, wg, total);
    else
      gemm_body<E, true, true, Shape, false, false>(a.dw, smem, wg, total);
  }
}

}  // namespace llar_ffn
