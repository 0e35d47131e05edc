// The products of MXFP4 operands with bfloat16 outputs on tiles of 64 rows, and the
// K split of either type (tgemm_ffn_mx_tiles.hpp).
#include "tgemm_ffn_mx_tiles.hpp"

namespace tgemm {
namespace ffn {

template <>
hipError_t launch_mx_64<0>(const MxGemm &g, bool two) {
  return two ? launch_mx_aligned<0, 64, 64, true>(g) : launch_mx_aligned<0, 64, 64, false>(g);
}

hipError_t launch_mx_split(const MxGemm &g) { return launch_mx_split_tiles(g); }

}  // namespace ffn
}  // namespace tgemm
