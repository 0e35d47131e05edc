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

namespace {

// A round is one tile a CU, or two of 128 x 128; it takes about base + slice *
// (K / 256) us, and more with an epilogue that is not the rounding alone
// (tile 128: half a round of tiles takes 0.72 of one).  Measured, us, the rounding
// alone | bias, gelu and residual | swiglu alone:
//   M     N     K      64                   128                 256
//   256   4096  4096   9.4   11.5  9.6      14.7  18.4  14.1    25.5  39.5  30.2
//   512   4096  4096   16.9  19.4  17.6     14.9  18.6  15.0    25.8  39.3  30.5
//   2048  4096  4096   60    69    60       23.0  29.2  22.1    27.0  43.1  33.2
//   4096  4096  1024   57    76    58       17.3  28.3  14.5    14.1  29.4  19.6
//   4096  4096  2048   80    96    79       25.0  34.9  22.7    20.3  35.3  25.6
//   4096  4096  8192   184   202   182      79.2  88.5  78.5    60.1  74.9  65.8
//   8192  8192  4096   457   544   454      177   223   170     134   187   147
struct MxShape {
  int tm, per_round;
  double base, slice, fused, gated;
};
constexpr MxShape kMxShapes[] = {
    {256, 256, 7.5, 1.64, 15.4, 6.0}, {128, 512, 4.6, 1.10, 5.0, -0.8}, {64, 256, 3.0, 0.27, 1.0, 0.0}};

int pick(const MxGemm &g) {
  int best = 0;
  double best_t = 0;
  const bool gated = is_gated(g.act), fused = g.bias || g.residual || g.preact || (!gated && g.act != kNone);
  const int64_t hit = std::min(g.groups, g.M);
  for (const MxShape &s : kMxShapes) {
    if (s.tm == 256 && !big_tile(g)) continue;
    double rounds;
    if (g.groups) {
      // A group's last tile is half full on average, and the groups' tiles do not
      // fill their last round.
      const double tiles = ((double)g.M / s.tm + 0.5 * (double)hit) * (double)((g.N + s.tm - 1) / s.tm);
      rounds = tiles / s.per_round;
      rounds = rounds < 0.5 ? (s.per_round > 256 ? 0.72 : 1.0) : rounds < 1.0 ? 1.0 : rounds + 0.5;
    } else {
      const int64_t tiles = ((g.M + s.tm - 1) / s.tm) * ((g.N + s.tm - 1) / s.tm);
      const int64_t rest = tiles % s.per_round;
      rounds = (double)(tiles / s.per_round) + (rest == 0 ? 0.0 : rest <= 256 && s.per_round > 256 ? 0.72 : 1.0);
    }
    const double t = rounds * (s.base + s.slice * (double)g.K / 256.0 + (gated ? s.gated : 0.0) + (fused ? s.fused * (gated ? 0.5 : 1.0) : 0.0));
    if (best == 0 || t < best_t) {
      best = s.tm;
      best_t = t;
    }
  }
  return best;
}

}  // namespace

hipError_t launch_mx(const MxGemm &g) {
  int tm = g.tile_m;
  if (tm == 0) tm = g.M <= (g.groups ? 10 * g.groups : 16) ? 16 : pick(g);
  if (tm == 16) return launch_mx_rows(g);
  bool two = false;
  if (tm == 64) {
    const int64_t tiles = g.groups ? g.M / 64 + std::min(g.groups, g.M) : (g.M + 63) / 64;
    two = tiles * ((g.N + 63) / 64) > 256;
  }
  return g.dtype == 1 ? launch_mx_f16(g, tm, two) : launch_mx_bf16(g, tm, two);
}

}  // namespace ffn
}  // namespace tgemm
