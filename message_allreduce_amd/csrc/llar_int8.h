// llar_int8.h -- argument blocks and launchers of the 8-bit products (not public).
#pragma once
#include "llar_ffn.h"

namespace llar_ffn {

// Rows of whole numbers from rows of values: q rows `qld` apart, with zeros behind
// them up to column `qpad`; x's columns `cs` apart.
struct QuantArgs {
  const void* x;
  int8_t* q;
  float* scale;
  int64_t xld, xcs, qld;
  int64_t M;
  int K, qpad;
};

// 8-bit rows copied so that they start, and are, whole 16-byte chunks.
constexpr int kPack8Threads = 256;
struct Pack8Args {
  const int8_t* src[3];
  int8_t* dst[3];
  int64_t ld[3], dld, lines[3];
  int64_t first[4];  // workgroup that starts each
  int width, count;
};
hipError_t launch_pack8(const Pack8Args& a, hipStream_t s);

// Both in one launch (copies.first is set here).
hipError_t launch_quantize(int kind, const QuantArgs& a, const Pack8Args& copies, hipStream_t s);

// Products with M <= kFewRows8 rows of x, any alignment.  kind: the results' type.
// values: x is of that type and not quantised yet, M <= kFewValuesRows, K <= kFewValuesK.
constexpr int kFewRows8 = 32;
constexpr int kFewValuesRows = 2, kFewValuesK = 8192;
// Pairs of 16 weight rows, what its wider workgroups take.
inline int64_t few_pairs(int64_t n, bool gated) { return (n + (gated ? 15 : 31)) / (gated ? 16 : 32); }
hipError_t launch_few_int8(int kind, bool gated, bool values, const GemmArgs& a, hipStream_t s);

// The join of a product split over k: whole sums, then scales and epilogue.
hipError_t launch_join_int8(int kind, bool gated, const GemmArgs& a, hipStream_t s);

// A sum of products of whole numbers of -128 .. 127 fits 32 bits up to this k.
constexpr int64_t kMaxInt8K = (1 << 17) - 1;

}  // namespace llar_ffn
