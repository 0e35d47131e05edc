// The tiled products of MXFP4 operands with bfloat16 outputs (tgemm_ffn_mx_tiles.hpp).
#include "tgemm_ffn_mx_tiles.hpp"

namespace tgemm {
namespace ffn {

hipError_t launch_mx_bf16(const MxGemm &g, int tm, bool two) { return launch_mx_tiles_dt<0>(g, tm, two); }

}  // namespace ffn
}  // namespace tgemm
