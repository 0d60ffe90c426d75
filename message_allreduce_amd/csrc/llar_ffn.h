// llar_ffn.h -- argument blocks and launchers shared by the host side of the
// feed-forward operators (llar_ffn.hip) and their kernels (not public).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace llar_ffn {

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// One matrix product, or two that share their shape and strides:
//
//   out[b][i][j] = epilogue( sum over s, k of x[s or b][i][k] * w[s or b][j][k] )
//
// i < M, j < N, k < K.  `segs` = 2 adds the products of both pairs (x[0],
// w[0]) and (x[1], w[1]); `batch` = 2 keeps them apart in out[0] and out[1].
// A gated product takes w[0] and w[1] with the same x and combines both sums
// of an element in its epilogue.
// A matrix lies k-contiguous (rows `ld` elements apart) or row-contiguous
// (consecutive k `ld` elements apart); out, resid and z rows are contiguous.
// The tiled kernel reads both operands in whole, 16-byte aligned chunks: lines
// whose length is no multiple of one are followed by zeros up to it.
struct GemmArgs {
  const void* x[2];
  const void* w[2];
  void* out[2];
  void* z[2];           // linear: z[0] keeps the value before the activation; gated: both projections
  const void* bias;     // N elements or null
  const void* resid;    // M x N or null
  float* partial;       // split over k: [split][plane][M][npad] sums, else null
  int64_t xld, wld, outld, zld, rld;
  int M, N, K;
  int segs, batch, splits;
  int act;
  int npad;             // row length of a partial plane
  const float* xscale;  // 8-bit operands: of every row of x, and of w[0] and w[1]
  const float* wscale[2];
};

// Whether a launch stays below 2^32 threads.  The runtime counts them in 32 bits,
// and what is beyond would be left out without an error, so every launcher asks.
inline bool launchable(int64_t groups, int threads) { return groups * threads < (1ll << 32); }

// Tile shapes of the product kernel (rows of x by rows of w by workgroup);
// see llar_gemm.h.
enum Tile : int { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTile128x64 = 3, kTileCount = 4 };
constexpr int kTileM[kTileCount] = {256, 128, 64, 128};
constexpr int kTileN[kTileCount] = {256, 128, 64, 64};

struct GemmPlan {
  int kind;        // llar_dtype
  int tile, groups;
  bool x_rows;     // x is row-contiguous
  bool w_rows;
  bool gated;
};

hipError_t launch_gemm(const GemmPlan& p, const GemmArgs& a, hipStream_t s);
// The same with 8-bit operands, both k-contiguous, and outputs of type p.kind.
hipError_t launch_gemm_int8(const GemmPlan& p, const GemmArgs& a, hipStream_t s);

// The products of a backward pass together: dx from k-contiguous rows of dz, dw
// from dz and x both row-contiguous.
struct PairArgs {
  GemmArgs dx, dw;
  int first;  // workgroups of the one that goes first
  bool dw_first;
};
hipError_t launch_pair(int kind, int tile, int groups, bool w_rows, PairArgs a, hipStream_t s);

// A product with M <= kFewRows rows of k-contiguous x and N <= kFewColumns (up to
// 128 threads a column: 2^31), any alignment; a.batch is 1.
constexpr int kFewRows = 16;
constexpr int64_t kFewColumns = 1 << 24;
hipError_t launch_few(int kind, bool w_rows, bool gated, const GemmArgs& a, hipStream_t s);

// Copies of matrices in whole chunks: lines of `width` elements, `ld` apart,
// written `dld` apart (a multiple of 8) with zeros behind them.
constexpr int kRepackMax = 4;
struct RepackArgs {
  const void* src[kRepackMax];
  void* dst[kRepackMax];
  int64_t ld[kRepackMax], dld[kRepackMax], lines[kRepackMax], width[kRepackMax];
  int64_t first[kRepackMax + 1];  // workgroup that starts each
  int count;
};
hipError_t launch_repack(int kind, const RepackArgs& a, hipStream_t s);

// Sums the partial planes of a product split over k and applies its epilogue.
hipError_t launch_join(int kind, bool gated, const GemmArgs& a, hipStream_t s);

// dg = dh u act'(g), du = dh act(g), element by element (rows contiguous, but for
// dh's, whose columns are `dhcs` apart; rows of dg and du `dld` apart, a multiple
// of 8, with zeros behind column N).
struct GateGradArgs {
  const void *dh, *g, *u;
  void *dg, *du;
  int64_t dhld, dhcs, gld, uld, dld;
  int M, N;
  int act;
};
hipError_t launch_gate_grad(int kind, const GateGradArgs& a, hipStream_t s);

// dz = dy act'(z) (z null: no activation; dz null: not written) and the sum of dz
// over the rows: part[c][j] = sum over row chunk c, then db[j] = sum over c in
// order.  dz rows as for the gated block, dy's columns `dycs` apart.
struct ActGradArgs {
  const void *dy, *z;
  void* dz;
  void* db;
  float* part;
  int64_t dyld, dycs, zld, dzld;
  int M, N;
  int act;
  int chunks;
};
hipError_t launch_act_grad(int kind, const ActGradArgs& a, hipStream_t s);

}  // namespace llar_ffn
