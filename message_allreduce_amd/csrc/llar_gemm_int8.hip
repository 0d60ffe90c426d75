// llar_gemm_int8.hip -- instances of the product kernel for 8-bit operands;
// compiled once for each type of the results (LLAR_ELEM: F32, F16 or BF16).
// The tiles are the 16-bit operands' (the same bytes, twice the k) with whole-number
// sums.  The large one is bound by the matrix units: 8192^3 407 us, 2700 TOPS, 74 % busy
// at the clock that power leaves; 8192 x 3584 -> 8192 bf16 208 us, 134 MB of results with
// it.  The small ones by their first loads: 512 x 2048 x 2048 9.1 us.
#include "llar_gemm.h"

namespace llar_ffn {

template <class E, class Shape, bool kGated>
hipError_t launch_one(const GemmArgs& a, hipStream_t s) {
  const int tn_cols = Shape::TN / (kGated ? 2 : 1);
  const int64_t tiles = ((int64_t)a.M + Shape::TM - 1) / Shape::TM * (((int64_t)a.N + tn_cols - 1) / tn_cols);
  const int64_t grid = tiles * a.splits;
  if (grid <= 0) return hipSuccess;
  if (!launchable(grid, Shape::kAllThreads)) return hipErrorInvalidConfiguration;
  k_gemm<E, false, false, Shape, kGated><<<dim3((uint32_t)grid), dim3(Shape::kAllThreads), 0, s>>>(a);
  return hipGetLastError();
}

template <class E, bool kGated>
hipError_t launch_shape(const GemmPlan& p, const GemmArgs& a, hipStream_t s) {
  if (p.tile == kTile256) return launch_one<E, Shape256, kGated>(a, s);
  if (p.tile == kTile128x64) return launch_one<E, Shape128x64, kGated>(a, s);
  if (p.tile == kTile128) {
    if (p.groups == 1) return launch_one<E, Shape128<1>, kGated>(a, s);
    return launch_one<E, Shape128<2>, kGated>(a, s);
  }
  if (p.groups == 1) return launch_one<E, Shape64<1>, kGated>(a, s);
  if (p.groups == 2) return launch_one<E, Shape64<2>, kGated>(a, s);
  return launch_one<E, Shape64<4>, kGated>(a, s);
}

#define LLAR_CAT_(a, b) a##_##b
#define LLAR_CAT(a, b) LLAR_CAT_(a, b)

hipError_t LLAR_CAT(launch_gemm_int8, LLAR_ELEM)(const GemmPlan& p, const GemmArgs& a, hipStream_t s) {
  if (p.gated) return launch_shape<Int8<LLAR_ELEM>, true>(p, a, s);
  return launch_shape<Int8<LLAR_ELEM>, false>(p, a, s);
}

}  // namespace llar_ffn
