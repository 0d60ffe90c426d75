// llar_gemm_inst.hip -- instances of the product kernel for one element type
// and one pair of operand orders; compiled once for each (LLAR_ELEM: F32, F16
// or BF16; LLAR_XR, LLAR_WR: 1 where the operand is row-contiguous).
#include "llar_gemm.h"

namespace llar_ffn {

template <class E, bool kXRows, bool kWRows, class Shape, bool kGated>
hipError_t launch_one(const GemmArgs& a, hipStream_t s) {
  const int tn_cols = Shape::TN / (kGated ? 2 : 1);
  const int64_t tiles = ((int64_t)a.M + Shape::TM - 1) / Shape::TM * (((int64_t)a.N + tn_cols - 1) / tn_cols);
  const int64_t grid = tiles * a.batch * a.splits;
  if (grid <= 0) return hipSuccess;
  if (!launchable(grid, Shape::kAllThreads)) return hipErrorInvalidConfiguration;
  if constexpr (E::kind == 0)
    k_gemm32<kXRows, kWRows, Shape, kGated><<<dim3((uint32_t)grid), dim3(Shape::kAllThreads), 0, s>>>(a);
  else
    k_gemm<E, kXRows, kWRows, Shape, kGated><<<dim3((uint32_t)grid), dim3(Shape::kAllThreads), 0, s>>>(a);
  return hipGetLastError();
}

template <class E, bool kXRows, bool kWRows, bool kGated>
hipError_t launch_shape(const GemmPlan& p, const GemmArgs& a, hipStream_t s) {
  if constexpr (E::kind != 0) {
    if (p.tile == kTile256) return launch_one<E, kXRows, kWRows, Shape256, kGated>(a, s);
    if (p.tile == kTile128x64) return launch_one<E, kXRows, kWRows, Shape128x64, kGated>(a, s);
  }
  if (p.tile == kTile128) {
    if (p.groups == 1) return launch_one<E, kXRows, kWRows, Shape128<1>, kGated>(a, s);
    return launch_one<E, kXRows, kWRows, Shape128<2>, kGated>(a, s);
  }
  if (p.groups == 1) return launch_one<E, kXRows, kWRows, Shape64<1>, kGated>(a, s);
  if (p.groups == 2) return launch_one<E, kXRows, kWRows, Shape64<2>, kGated>(a, s);
  return launch_one<E, kXRows, kWRows, Shape64<4>, kGated>(a, s);
}

#define LLAR_CAT_(a, b, c, d) a##_##b##_##c##d
#define LLAR_CAT(a, b, c, d) LLAR_CAT_(a, b, c, d)

hipError_t LLAR_CAT(launch_gemm, LLAR_ELEM, LLAR_XR, LLAR_WR)(const GemmPlan& p, const GemmArgs& a, hipStream_t s) {
  if (p.gated) return launch_shape<LLAR_ELEM, LLAR_XR, LLAR_WR, true>(p, a, s);
  return launch_shape<LLAR_ELEM, LLAR_XR, LLAR_WR, false>(p, a, s);
}

}  // namespace llar_ffn
