// Which kernel a product of MXFP4 operands takes (host code).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "tgemm_ffn_internal.hpp"

namespace tgemm {
namespace ffn {

// 256 x 256 tiles take whole slices of 256 elements and scale rows that start
// on a dword.
static bool big_tile(const MxGemm &g) { return g.K > 0 && g.K % 256 == 0 && mx_scales_aligned(g); }

bool mx_tile_supported(const MxGemm &g, int tm, int tn) {
  return tm == tn && (tm == 16 || tm == 64 || tm == 128 || (tm == 256 && big_tile(g)));
}

// K is split where 64 x 64 tiles leave at least half the compute units idle and
// K is so deep that each is spared nine slices of 512 or more (0.45 us each): as
// many splits as fill the units once.  The second launch and the sums on their
// way cost about 4 us.  us, unsplit -> split, rows read from memory:
//   M    N     K                          M    N     K
//   48   8192  28672  29.3 -> 23.9 (2)    48   8192  8192   11.2 -> 11.3 (2)
//   48   4096  14336  15.9 -> 11.6 (4)    512  1024  8192   11.2 -> 11.8 (2)
//   64   1024  8192   10.9 -> 8.7 (4)     64   1024  4096    7.3 -> 7.9 (2)
//   100  256   8192   11.0 -> 8.7 (4)     200  2048  4096    7.6 -> 9.7 (2)
// (256 compute units: the workspace's size is asked for where there may be no
// device.  Up to 16 rows the kernel for few rows splits K among its waves.)
int mx_splits(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64), slices = (K + 511) / 512;
  if (M <= 16 || tiles == 0 || tiles * 2 > 256 || slices < 8) return 1;
  const int64_t n = std::min<int64_t>({256 / tiles, slices / 4, 16});
  const int64_t each = (slices + n - 1) / n;
  return slices - each >= 9 ? (int)((slices + each - 1) / each) : 1;
}

namespace {

// A round is one 256 x 256 tile a CU or two of the smaller ones; it takes about base +
// slice * (K / 256) us, and more with an epilogue that is not the rounding
// alone; up to one smaller tile a CU take 0.6 of a round.  Measured, us, with the
// rounding alone | bias, gelu and residual | swiglu alone:
//   M     N     K      64                   128                 256
//   256   4096  4096   7.7   9.0   7.8      12.1  15.7  11.7    25.4  39.0  30.3
//   512   4096  4096   11.8  13.5  11.7     12.5  16.2  12.1    25.4  39.3  30.4
//   1024  4096  4096   20.9  24.1  20.7     14.7  18.8  13.8    25.7  39.8  30.6
//   2048  4096  4096   38.8  42.7  36.8     22.8  28.4  21.8    26.6  41.5  31.5
//   4096  4096  1024   27.5  39.0  28.0     16.4  26.7  14.2    13.8  28.5  18.8
//   4096  4096  2048   40.5  49.6  39.4     23.9  33.2  21.9    19.6  33.6  24.7
//   4096  4096  8192   136   137   129      78.5  86.6  78.4    58.7  72.8  63.8
//   8192  8192  4096   285   335   275      168   221   160     129   201   142
struct MxShape {
  int tm, per_round;
  double base, slice, fused, gated;
};
constexpr MxShape kMxShapes[] = {
    {256, 256, 5.0, 1.63, 14.5, 6.0}, {128, 512, 3.3, 1.085, 4.5, -1.0}, {64, 512, 1.5, 0.48, 0.8, -0.3}};

// Tiles of tm x tm, of groups of any sizes: a group's last one is half full on
// average, and every group that has rows has one.
double tiles_of(const MxGemm &g, int tm) {
  const double across = (double)((g.N + tm - 1) / tm);
  if (!g.groups) return (double)((g.M + tm - 1) / tm) * across;
  const double hit = (double)std::min(g.groups, g.M);
  return std::max(hit, (double)g.M / tm + 0.5 * hit) * across;
}

int pick(const MxGemm &g) {
  int best = 0;
  double best_t = 0;
  const bool gated = is_gated(g.act), fused = g.bias || g.residual || g.preact || (!gated && g.act != kNone);
  for (const MxShape &s : kMxShapes) {
    if (s.tm == 256 && !big_tile(g)) continue;
    const double tiles = tiles_of(g, s.tm), whole = std::floor(tiles / s.per_round), rest = tiles - whole * s.per_round;
    double rounds = whole + (rest <= 0 ? 0.0 : rest <= 256 && s.per_round > 256 ? 0.6 : 1.0);
    if (g.groups && whole > 0) rounds = tiles / s.per_round + 0.5;  // (the groups end at different times)
    const double t = rounds * (s.base + s.slice * (double)g.K / 256.0 + (gated ? s.gated : 0.0) + (fused ? s.fused * (gated ? 0.5 : 1.0) : 0.0));
    if (best == 0 || t < best_t) {
      best = s.tm;
      best_t = t;
    }
  }
  return best;
}

// Whether a product takes the kernel for few rows: up to 16 rows of one
// weight, up to 10 a group on average, where 64 x 64 tiles are fewer than half
// the CUs or K is short; with more of them those read the weights faster, or (at the
// border, 8192 x 8192) soon will.  us between launches of a graph, weights from
// memory, this kernel and 64 x 64 tiles:
//   one row: 4096 x 4096 4.9 and 7.5, 1024 x 8192 6.0 and 10.4, 4096 x 1024 2.9 and
//   4.0, 8192 x 8192 10.6 and 12.3, 32768 x 4096 18.1 and 16.3; 16 rows of 8192 x
//   4096 8.6 and 8.2; 64 gated experts of 2048 x 2048 by 6 rows 6.4 and 6.2, by
//   220 32.7 and 32.8; 64 of 2048 x 1024 by 220 19.5 and 24.2.
bool few_rows(const MxGemm &g) {
  if (g.M > (g.groups ? 10 * g.groups : 16)) return false;
  return g.K <= 1024 || tiles_of(g, 64) < 0.5 * g.cus;
}

}  // namespace

hipError_t launch_mx(const MxGemm &g) {
  if (g.splits > 1) {
    const hipError_t e = launch_mx_split(g);
    if (e != hipSuccess) return e;
    Gemm j{};
    j.dtype = g.dtype;
    j.M = g.M;
    j.N = g.N;
    j.bias = g.bias;
    j.residual = g.residual;
    j.ldr = g.ldr;
    j.preact = g.preact;
    j.ldp = g.ldp;
    j.C = g.C;
    j.ldc = g.ldc;
    j.act = g.act;
    j.ws = g.ws;
    j.splits = g.splits;
    j.stream = g.stream;
    return launch_join(j);
  }
  int tm = g.tile_m;
  if (tm == 0) tm = few_rows(g) ? 16 : pick(g);
  if (tm == 16) return launch_mx_rows(g);
  // 64 x 64 tiles: one a CU with a deep ring while they are that few, else two.
  const bool two = tm == 64 && tiles_of(g, 64) > (double)g.cus;
  if (tm == 64) return g.dtype == 1 ? launch_mx_64<1>(g, two) : launch_mx_64<0>(g, two);
  return g.dtype == 1 ? launch_mx_large<1>(g, tm) : launch_mx_large<0>(g, tm);
}

}  // namespace ffn
}  // namespace tgemm
