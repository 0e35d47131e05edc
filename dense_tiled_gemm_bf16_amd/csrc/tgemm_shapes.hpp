// The choice of the 16-bit kernels' tile shape (host code).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace tgemm {
namespace {

// Tile shapes per kind, largest first, each with a rate relative to
// 256 x 256 per unit of tile area in a wave of workgroups (one workgroup
// per CU).  The rates are fitted to sustained measurements on MI355X
// (bf16 NT unless noted, us):
//                        256x256  256x192  128x128  64x64
//   4096 x 4096 x 8192     193      --       251      --   (rate 0.77 here)
//   3072 x 3072 x 3072      65      --        74      --
//   4000 x 3000 x 5000     118     117       156      --
//   2048 x 2048 x 4096      78      63        35      --
//   2048 x 1024 x 4096      77      --        27      --
//   512 x 512 x 4096        --      --        25.8    12.2
//   fp16 NN 2048 x 1024^2   --      --        12.0    11.1
//   fp16 NN 1024^3          31      --        11.8     6.2
//   256^3                   --      --         5.9     3.7
// 0.70 for 128 x 128 sits between the first two rows: a partly filled last
// wave runs at a higher clock under the power cap than whole ones.  0.35
// for 64 x 64 fits the rows below it, where a slice's loads and barrier,
// not its 8 MFMAs per wave, set the pace.
struct Shape {
  int tm, tn;
  double rel;
};
constexpr Shape kShapesBK[] = {{256, 256, 1.0}, {256, 192, 0.92}, {128, 128, 0.70}, {64, 64, 0.35}};  // B K-contiguous
constexpr Shape kShapesBN[] = {{256, 256, 1.0}, {128, 128, 0.70}, {64, 64, 0.35}};                     // B N-contiguous

// The shape with the least estimated time: whole waves of tiles over the
// CUs, each wave costing its tile area over the shape's relative rate.
template <size_t NS>
Shape pick_shape(const Shape (&shapes)[NS], int64_t M, int64_t N, int cus) {
  Shape best = shapes[0];
  double best_t = 0;
  for (size_t i = 0; i < NS; ++i) {
    const Shape &s = shapes[i];
    const int64_t tiles = ((M + s.tm - 1) / s.tm) * ((N + s.tn - 1) / s.tn);
    const int64_t slots = cus;  // one workgroup per CU
    const int64_t waves = (tiles + slots - 1) / slots;
    const double t = (double)waves * s.tm * s.tn / s.rel;
    if (i == 0 || t < best_t) {
      best = s;
      best_t = t;
    }
  }
  return best;
}

}  // namespace
}  // namespace tgemm
