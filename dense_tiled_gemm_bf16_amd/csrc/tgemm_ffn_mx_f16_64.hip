// The products of MXFP4 operands with float16 outputs on tiles of 64 rows
// (tgemm_ffn_mx_tiles.hpp).
#include "tgemm_ffn_mx_tiles.hpp"

namespace tgemm {
namespace ffn {

template <>
hipError_t launch_mx_64<1>(const MxGemm &g, bool two) {
  return two ? launch_mx_aligned<1, 64, 64, true>(g) : launch_mx_aligned<1, 64, 64, false>(g);
}

}  // namespace ffn
}  // namespace tgemm
