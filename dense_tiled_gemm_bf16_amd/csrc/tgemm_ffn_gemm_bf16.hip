// The feed-forward products' tiled kernels on bfloat16 (tgemm_ffn_tiles.hpp).
#include "tgemm_ffn_tiles.hpp"

namespace tgemm {
namespace ffn {

hipError_t launch_gemm_bf16(const Gemm &g, int tm, int tn) { return launch_layouts<kBf16>(g, tm, tn); }
hipError_t launch_split_bf16(const Gemm &g) { return launch_split<kBf16>(g); }
hipError_t launch_tn_bf16(const GroupedTn &g, int tm, int tn) { return launch_tn<kBf16>(g, tm, tn); }

}  // namespace ffn
}  // namespace tgemm
