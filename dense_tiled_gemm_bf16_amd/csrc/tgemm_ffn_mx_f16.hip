// The products of MXFP4 operands with float16 outputs on tiles of 128 and 256 rows
// (tgemm_ffn_mx_tiles.hpp).
#include "tgemm_ffn_mx_tiles.hpp"

namespace tgemm {
namespace ffn {

template <>
hipError_t launch_mx_large<1>(const MxGemm &g, int tm) {
  return tm == 256 ? launch_mx_gated<1, 256, 256, false, true>(g) : launch_mx_aligned<1, 128, 128, true>(g);
}

}  // namespace ffn
}  // namespace tgemm
