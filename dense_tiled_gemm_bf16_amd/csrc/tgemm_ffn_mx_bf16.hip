// The tiled products of MXFP4 operands with bfloat16 outputs, and the
// K split of either (tgemm_ffn_mx_tiles.hpp).
#include "tgemm_ffn_mx_tiles.hpp"

namespace tgemm {
namespace ffn {

hipError_t launch_mx_bf16(const MxGemm &g, int tm, bool two) { return launch_mx_tiles_dt<0>(g, tm, two); }

hipError_t launch_mx_split(const MxGemm &g) { return launch_mx_split_tiles(g); }

}  // namespace ffn
}  // namespace tgemm
