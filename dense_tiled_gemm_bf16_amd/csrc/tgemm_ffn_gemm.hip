// Which kernel a feed-forward product takes (host code).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tgemm_ffn_internal.hpp"
#include "tgemm_shapes.hpp"

namespace tgemm {
namespace ffn {

bool tile_supported(const Gemm &g, int tm, int tn) {
  if (tm == 16 && tn == 16) return !g.trans_a && g.trans_b;
  if (tm == 256 && tn == 192) return g.trans_b && !is_gated(g.act) && g.groups == 0;
  return (tm == 256 && tn == 256) || (tm == 128 && tn == 128) || (tm == 64 && tn == 64);
}

namespace {

// Whether a product takes the kernel for few rows, where its layout does.  One
// weight: up to 16 rows, one tile of it (4096 x 4096: 1 row 8.5 us, 64 x 64
// tiles 13.0; 16 rows 10.2 and 13.2; 32 rows 19.4 and 13.4).  Groups: up to 10
// rows on average (64 experts of 2048 x 2048 gated: 3.5 rows 85 us, 64 x 64
// tiles 104; 9.4 rows 118 and 122; 16 rows 145 and 124).
// Not where 64 x 64 tiles are between half and all of one a compute unit, which
// then stream the weights at the same rate with fewer fixed costs: 6 of 64
// gated experts of 2048 x 2048 (192 tiles) 14.8 us and 12.7, 8 (256) 15.8 and
// 13.9, but 4 (128) 9.9 and 11.1, 12 (384) 21.5 and 23.8; one weight, 16 rows of
// 16384 x 4096 (256 tiles) 38.7 and 30.8, 16384 x 1024 10.4 and 8.9, but one
// row of 16384 x 2048 15.9 and 17.5, so from more than 8 rows on.
bool few_rows(const Gemm &g) {
  if (g.trans_a || !g.trans_b || g.M > (g.groups ? 10 * g.groups : 16)) return false;
  if (g.groups == 0 && g.M <= 8) return true;
  const int64_t tiles = (g.N + 63) / 64 * (g.groups ? std::min(g.groups, g.M) : 1);
  return 2 * tiles <= g.cus || tiles > g.cus;
}

// The shape with the least estimated time (as pick_shape), over groups of any
// sizes, whose last row tile is half full on average (256-row tiles: half of
// the last ones are short tiles of 0.6 of the time, so 0.3 of a tile is lost).
template <size_t NS>
Shape pick_grouped(const Shape (&shapes)[NS], int64_t M, int64_t N, int64_t groups, int cus) {
  Shape best{};
  double best_t = 0;
  const int64_t hit = std::min(groups, M);
  for (const Shape &s : shapes) {
    if (s.tn == 192) continue;
    const double tiles = ((double)M / s.tm + (s.tm == 256 ? 0.3 : 0.5) * (double)hit) * (double)((N + s.tn - 1) / s.tn);
    const double waves = tiles / cus < 1.0 ? 1.0 : tiles / cus + 0.5;
    const double t = waves * s.tm * s.tn / s.rel;
    if (best.tm == 0 || t < best_t) {
      best = s;
      best_t = t;
    }
  }
  return best;
}

// Compute units of an MI355X: the workspace's size is asked for on the host, where
// there may be no device, and the call has to split as that said.
constexpr int kCus = 256;
constexpr int kMostSplits = 16;

}  // namespace

// K is split where 64 x 64 tiles leave at least half the compute units idle
// and K is deep: as many splits as fill them once, of 8 slices of 64 or more.
// us, NT with bias, gelu and residual but where noted, unsplit -> split:
//   M     N     K                          M    N     K
//   48    2048  2048   8.4 -> 7.9 (4)      48   4096  2048, swiglu  8.0 -> 9.1 (4)
//   256   1024  4096  12.0 -> 10.1 (4)     512  512   2048   8.0 -> 9.1 (4)
//   553   896   4016  19.9 -> 16.2 (2)     24   1024  8192  20.1 -> 8.8 (16)
//   512   512   8192  23.3 -> 13.8 (4)     704  704   8192  24.4 -> 18.7 (2)
// More splits than fill the chip lose (704 x 704 x 8192: 3 take 24.2), and so
// do any where more than half of it is busy (1138 x 736 x 7296: 24.7 -> 29.8).
// The bound on M + N can only tell in one row of tiles with more than 7104
// columns (or one column with as many rows), and goes by weights that the caches
// hold (K = 4096: 48 x 6144 gated 14.3 -> 13.9, 48 x 7168 14.6 -> 14.6, 48 x
// 8192 gated 14.9 -> 15.9).  Weights from beyond them would be read faster by
// two splits there too: 48 x 8192 x 4096 gated 22.0 -> 20.5, 17 x 8192 x 2112
// 12.1 -> 11.3, 64 x 8192 x 8192 43.1 -> 34.0, NN 48 x 7680 x 4096 26.5 -> 19.5.
// At up to 16 rows NT the kernel for few rows splits K among its waves, and
// this split beats it from deeper on (16 x 1024: 4096 9.8 -> 8.0, 8192 16.8 ->
// 8.8; one row: 4096 7.2 -> 7.5, 8192 11.5 -> 8.3).
int epilogue_splits(bool trans_a, bool trans_b, int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((M + 63) / 64) * ((N + 63) / 64), slices = (K + 63) / 64;
  const bool rows = !trans_a && trans_b && M <= 16;
  if (tiles == 0 || tiles * 2 > kCus || M + N > 28 * kCus || slices <= (rows ? 64 : 32)) return 1;
  const int64_t n = std::min<int64_t>({kCus / tiles, slices / 8, kMostSplits});
  const int64_t each = (slices + n - 1) / n;
  return (int)((slices + each - 1) / each);
}

hipError_t launch_gemm(const Gemm &g) {
  int tm = g.tile_m, tn = g.tile_n;
  if (g.splits > 1) {
    const hipError_t e = g.dtype == 1 ? launch_split_f16(g) : launch_split_bf16(g);
    return e != hipSuccess ? e : launch_join(g);
  }
  if (tm == 0) {
    if (few_rows(g)) {
      tm = tn = 16;
    } else {
      Shape s;
      if (g.groups)
        s = pick_grouped(kShapesBK, g.M, g.N, g.groups, g.cus);
      else if (g.trans_b && !is_gated(g.act))
        s = pick_shape(kShapesBK, g.M, g.N, g.cus);
      else
        s = pick_shape(kShapesBN, g.M, g.N, g.cus);
      tm = s.tm;
      tn = s.tn;
    }
  }
  if (tm == 16) return launch_rows(g);
  return g.dtype == 1 ? launch_gemm_f16(g, tm, tn) : launch_gemm_bf16(g, tm, tn);
}

hipError_t launch_grouped_tn(const GroupedTn &g) {
  int tm = g.tile_m, tn = g.tile_n;
  if (tm == 0) {
    const Shape s = pick_shape(kShapesBN, g.P * g.groups, g.Q, g.cus);
    tm = s.tm;
    tn = s.tn;
  }
  return g.dtype == 1 ? launch_tn_f16(g, tm, tn) : launch_tn_bf16(g, tm, tn);
}

}  // namespace ffn
}  // namespace tgemm
