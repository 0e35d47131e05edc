// The feed-forward products' tiled kernels on fp16 (tgemm_ffn_tiles.hpp).
#include "tgemm_ffn_tiles.hpp"

namespace tgemm {
namespace ffn {

hipError_t launch_gemm_f16(const Gemm &g, int tm, int tn) { return launch_layouts<kF16>(g, tm, tn); }
hipError_t launch_split_f16(const Gemm &g) { return launch_split<kF16>(g); }
hipError_t launch_tn_f16(const GroupedTn &g, int tm, int tn) { return launch_tn<kF16>(g, tm, tn); }

}  // namespace ffn
}  // namespace tgemm
