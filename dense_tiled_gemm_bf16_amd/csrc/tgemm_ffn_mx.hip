// Which kernel a product of MXFP4 operands takes (host code).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tgemm_ffn_internal.hpp"

namespace tgemm {
namespace ffn {

bool mx_tile_supported(const MxGemm &, int tm, int tn) { return tm == 16 && tn == 16; }

int mx_splits(int64_t, int64_t, int64_t) { return 1; }

hipError_t launch_mx(const MxGemm &g) { return launch_mx_rows(g); }

}  // namespace ffn
}  // namespace tgemm
