// The tiled products of MXFP4 operands with float16 outputs (tgemm_ffn_mx_tiles.hpp).
#include "tgemm_ffn_mx_tiles.hpp"

namespace tgemm {
namespace ffn {

hipError_t launch_mx_f16(const MxGemm &g, int tm, bool two) { return launch_mx_tiles_dt<1>(g, tm, two); }

}  // namespace ffn
}  // namespace tgemm
