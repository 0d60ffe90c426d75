// llar_gemm_inst.hip -- instances of the product kernel for one element type
// and one pair of operand orders; compiled once for each (LLAR_ELEM: F32, F16
// or BF16; LLAR_XR, LLAR_WR: 1 where the operand is row-contiguous).
#include "llar_gemm.h"

namespace llar_ffn {

#define LLAR_CAT_(a, b, c, d) a##_##b##_##c##d
#define LLAR_CAT(a, b, c, d) LLAR_CAT_(a, b, c, d)

hipError_t LLAR_CAT(launch_gemm, LLAR_ELEM, LLAR_XR, LLAR_WR)(const GemmPlan& p, const GemmArgs& a, hipStream_t s) {
  if (p.gated) return launch_shape<LLAR_ELEM, LLAR_XR, LLAR_WR, true>(p, a, s);
  return launch_shape<LLAR_ELEM, LLAR_XR, LLAR_WR, false>(p, a, s);
}

}  // namespace llar_ffn
