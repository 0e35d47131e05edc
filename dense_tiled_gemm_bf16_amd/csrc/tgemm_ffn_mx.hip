// Which kernel a product of MXFP4 operands takes (host code).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tgemm_ffn_internal.hpp"

namespace tgemm {
namespace ffn {

// 256 x 256 tiles take whole slices of 256 elements and scale rows that start
// on a dword.
static bool big_tile(const MxGemm &g) { return g.K > 0 && g.K % 256 == 0 && mx_scales_aligned(g); }

bool mx_tile_supported(const MxGemm &g, int tm, int tn) {
  return tm == tn && (tm == 16 || tm == 64 || tm == 128 || (tm == 256 && big_tile(g)));
}

int mx_splits(int64_t, int64_t, int64_t) { return 1; }

hipError_t launch_mx(const MxGemm &g) {
  int tm = g.tile_m;
  if (tm == 0) {
    const int64_t per = g.groups ? g.M / std::min(g.groups, g.M) : g.M;
    tm = per <= 16 ? 16 : per <= 96 ? 64 : big_tile(g) && per > 192 ? 256 : 128;
  }
  if (tm == 16) return launch_mx_rows(g);
  return g.dtype == 1 ? launch_mx_f16(g, tm) : launch_mx_bf16(g, tm);
}

}  // namespace ffn
}  // namespace tgemm
