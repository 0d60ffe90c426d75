// llar_gemm_pair.hip -- instances of the kernel for both products of a backward
// pass, for one element type and one order of the weights; compiled once for
// each (LLAR_ELEM: F32, F16 or BF16; LLAR_WR: 1 where dx's weights are
// row-contiguous).
#include "llar_gemm.h"

namespace llar_ffn {

template <class Shape>
int64_t workgroups(const GemmArgs& a) {
  return ((int64_t)a.M + Shape::TM - 1) / Shape::TM * (((int64_t)a.N + Shape::TN - 1) / Shape::TN) * a.batch * a.splits;
}

template <class E, bool kWRows, class Shape>
hipError_t launch_one(PairArgs& a, hipStream_t s) {
  const int64_t first = workgroups<Shape>(a.dw_first ? a.dw : a.dx);
  const int64_t grid = first + workgroups<Shape>(a.dw_first ? a.dx : a.dw);
  if (!launchable(grid, Shape::kAllThreads)) return hipErrorInvalidConfiguration;
  a.first = (int)first;
  k_gemm_pair<E, kWRows, Shape><<<dim3((uint32_t)grid), dim3(Shape::kAllThreads), 0, s>>>(a);
  return hipGetLastError();
}

#define LLAR_CAT_(a, b, c) a##_##b##_##c
#define LLAR_CAT(a, b, c) LLAR_CAT_(a, b, c)

template <class E, bool kWRows>
hipError_t launch_shape(int tile, int groups, PairArgs& a, hipStream_t s) {
  if constexpr (E::kind != 0) {
    if (tile == kTile256) return launch_one<E, kWRows, Shape256>(a, s);
    if (tile == kTile128x64) return launch_one<E, kWRows, Shape128x64>(a, s);
  }
  if (tile == kTile128) {
    if (groups == 1) return launch_one<E, kWRows, Shape128<1>>(a, s);
    return launch_one<E, kWRows, Shape128<2>>(a, s);
  }
  if (groups == 1) return launch_one<E, kWRows, Shape64<1>>(a, s);
  if (groups == 2) return launch_one<E, kWRows, Shape64<2>>(a, s);
  return launch_one<E, kWRows, Shape64<4>>(a, s);
}

hipError_t LLAR_CAT(launch_pair, LLAR_ELEM, LLAR_WR)(int tile, int groups, PairArgs& a, hipStream_t s) {
  return launch_shape<LLAR_ELEM, LLAR_WR>(tile, groups, a, s);
}

}  // namespace llar_ffn
