// llar_moe.h -- argument blocks and launchers of the mixture-of-experts operators
// (not public).
#pragma once
#include "llar_ffn.h"

namespace llar_ffn {

constexpr int kMoeTokens = 64;     // of one pair of launches: a lane each
constexpr int kMoeExperts = 1024;
constexpr int kMoeTopK = 32;

// Logits of M tokens (rows of x) and E experts (rows of w), both k-contiguous.
struct RouteArgs {
  const void *x, *w;
  double* logits;  // [splits][M][E]
  int64_t xld, wld;
  int M, E, K, top_k;
  int splits;  // shares of k
  bool small;  // one kernel
  bool sigmoid, normalize;
  float* weights;
  int32_t* experts;
};
// Tokens of one pair of launches: room for their logits (binary64, 512 MiB at most), and far from 2^32 threads.
constexpr int64_t kRouteTokens = 1 << 16;
constexpr int64_t kRouteSmallTokens = 256, kRouteSmall = 1 << 17;
bool route_small(int64_t m, int64_t experts, int64_t k);  // one kernel, no logits in memory
int route_splits(int64_t m, int64_t experts, int64_t k);
hipError_t launch_route(int kind, const RouteArgs& a, hipStream_t s);

// At most kMoeTokens tokens.  A choice is place j of token t's list, p = t top_k + j;
// h holds a row for every choice that has an expert and is the first of its token
// with that expert.
struct MoeArgs {
  const void* x;         // T rows of k elements: of the I/O type, or int8
  const float* xscale;   // int8: of every token
  const void* w[2];      // gate, up: [E][n][k]
  const float* wscale[2];
  const void* wd;        // [E][outs][n]
  const float* dscale;
  void* h;               // first kernel's output (int8: binary32); second kernel's input (int8: whole numbers)
  int64_t hlow;          // 16-bit types: from a value to what its rounding left
  const float* hscale;   // int8: of every choice
  const void* ids;
  const float* weights;
  const void* resid;
  void* out;
  float* partial;        // [parts][T][outs], with more than one part
  int64_t xld, w_expert, wld, d_expert, dld, hld, rld, outld;
  int T, K, N, outs, E, top_k;
  int id_bytes, act;
  int parts;
};
// int8 with `values`: the kernel's own workgroups quantise its rows, x (up to
// kMoeValuesTokens of kMoeValuesK) and the inner ones (up to
// kMoeValuesRows choices of kMoeValuesBytes together: two rows a wave).
constexpr int kMoeValuesTokens = 2, kMoeValuesK = 8192, kMoeValuesRows = 16, kMoeValuesBytes = 16384;
hipError_t launch_moe_up(int kind, bool int8, bool values, const MoeArgs& a, hipStream_t s);
bool moe_wide(int T, int64_t outs);  // 32 columns a workgroup in the second kernel, else 16
int moe_parts(int T, int64_t n, int64_t outs, int64_t experts, int top_k, int es);
hipError_t launch_moe_down(int kind, bool int8, bool values, const MoeArgs& a, hipStream_t s);

}  // namespace llar_ffn
