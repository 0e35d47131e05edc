// The feed-forward products' tiled kernels for gfx950: the K loop of
// tgemm_kernel.hpp under a fused epilogue (bias, activation, residual, the
// values before the activation kept for a backward pass), for one weight
// (dense) or one weight for each group of rows (grouped), and the grouped
// product over rows that gives each group's weight gradient.
//
// Sums, bias, activation and residual are binary32; C is rounded once, to the
// element type, which is what the matrix instruction behind it takes as an
// operand.  The values before the activation are kept in that type too: two bytes
// a value on the way out and back in instead of four (33.5 MB less each way, 6 us
// at a copy's rate, of 4096 x 4096), for a derivative that is taken half a step of Z
// away (2^-8 of Z at most in bf16, as the rounding of the dZ made from it).
//
// What bounds them is the K loop: a 256 x 256 tile at K = 4096 is 64 slices of
// about 1.2 us each, and the epilogue's traffic (residual, values before the
// activation) streams at the end of each tile.  4096 x 4096 x 8192, inputs from
// memory: 196 us with bias, gelu and residual (1.40 PFLOP/s), 185 without any
// of them; the plain product 203, without the prefetch.  What the epilogue costs
// there, inputs in the caches: through LDS 6 us, relu 1.7 more, gelu 8.2 (about
// 0.9 for each VALU instruction a value), the residual 1.2, the values before the
// activation 1.5.
//
// The epilogue goes through LDS: the accumulators are indexed statically, so
// work on them directly would be unrolled 512 times for every activation
// (code of hundreds of KB a kernel), while a rolled loop over LDS rows keeps
// one copy of each activation and gives every global access 256 contiguous
// bytes of a row.  The round trip is about 4096 LDS clocks (2 us) a
// 256 x 256 tile.
#pragma once

#include "tgemm_ffn_math.hpp"
#include "tgemm_kernel.hpp"
#include "tgemm_shapes.hpp"

namespace tgemm {
namespace ffn {
namespace {

// The epilogue's operands (device pointers of the element type; grouped:
// already at the group's first row or its own entry).
struct Tail {
  const uint8_t *bias;  // or nullptr
  const uint8_t *res;   // or nullptr
  uint8_t *pre;         // or nullptr
  int ldr, ldp;
  int act;
  int half;  // gated: columns of one half (the second half's offset); else 0
};

struct Groups {
  const int32_t *offsets;
  const int32_t *rows;  // or nullptr
  int groups, R, src_rows;
  int64_t stride_b, stride_bias;  // elements
  int tiles_n;
};

// AREA: bytes of each of the four LDS areas (slots 0 and 1 of A and of B).
template <int DT, bool GATED, bool GROUPED, int AREA>
struct FfnExt {
  static constexpr bool kOn = true, kGated = GATED, kGather = GROUPED;
  // (Grouped ones with operands of the epilogue, as in training, find much of
  // theirs in the caches: 16 experts' training step 551 us, with it 558.)
  static constexpr bool kPrefetch = !GROUPED;
  int m0, n0;
  int half;
  const int32_t *rows;
  int src_rows;
  Tail t;

  // 64 rows of the wave tile at a time (32 for 64 x 64 tiles) go through the
  // wave's own LDS area as binary32, 16-byte chunk k of row r at place (k / 2
  // + k % 2 * half the chunks) ^ (r % 8): the writes (16 rows at one chunk)
  // and the reads (a row's even chunks, then its odd ones) each spread over
  // all banks.  A lane then takes pieces of 8 output columns, 64 pieces of
  // the wave side by side, kBatch of them at once without a branch between,
  // so that their LDS reads are in flight together; the residual's loads go
  // two batches ahead, the first before the accumulators are even in LDS
  // (one wave a SIMD has nothing else to hide them behind).
  template <class K>
  struct Shape {
    static constexpr int kWM = K::kWM, kWN = K::kWN;
    static constexpr int kRows = kWM < 64 ? kWM : 64;       // of one phase
    static constexpr int kOutN = GATED ? kWN / 2 : kWN;     // output columns of the wave tile
    static constexpr int kPer = kOutN / 8;                  // pieces of a row
    static constexpr int kPieces = kRows * kPer / 64;       // pieces of a lane and phase
    // (Gated pieces hold both halves: four of them would spill.)
    static constexpr int kBatch = kPieces % 4 == 0 && !GATED ? 4 : kPieces % 2 == 0 ? 2 : 1;
    static constexpr bool kOneColumn = 64 % kPer == 0;      // all of a lane's pieces are in one column
    static_assert(kRows * kPer % 64 == 0, "whole passes");
  };

  template <class K>
  __device__ __forceinline__ void store(K &k) const {
    using S = Shape<K>;
    constexpr int kWN = K::kWN, kNBn = K::kNBn, kChunks = kWN / 4, kRows = S::kRows;
    static_assert(K::kBlk == 16 && kChunks % 8 == 0 && kRows * kWN * 4 <= AREA, "staging area");
    const int lane = k.lane;
    LDS_AS uint8_t *area = k.wave == 0   ? k.slots.a[0]
                           : k.wave == 1 ? k.slots.a[1]
                           : k.wave == 2 ? k.slots.b[0]
                                         : k.slots.b[1];
    v4u r0[S::kBatch] = {}, r1[S::kBatch] = {};
    if (t.res) {
      load_res(k, 0, r0);
      load_res(k, 1, r1);
    }
    // Every wave's reads of the slots and loads into them are done.
    barrier();
#pragma unroll
    for (int ph = 0; ph < K::kWM / kRows; ++ph) {
#pragma unroll
      for (int j = 0; j < kRows / 16; ++j) {
        const int r = 16 * j + (lane & 15);
#pragma unroll
        for (int i = 0; i < kNBn; ++i) {
          const int c = 4 * i + (lane >> 4);
          const int at = ((c >> 1) + (c & 1) * (kChunks / 2)) ^ (r & 7);
          *(LDS_AS f32x4 *)(area + r * (kWN * 4) + at * 16) = k.acc[i][ph * (kRows / 16) + j];
        }
      }
      asm volatile("" ::: "memory");
      with_act<GATED>(t.act, [&](auto act) { rows_out<decltype(act)::value>(k, area, ph, r0, r1); });
      asm volatile("" ::: "memory");
    }
  }

  // Piece of batch `batch` (of the whole wave tile), number b: its row and
  // output column in the wave tile.
  template <class K>
  __device__ static __forceinline__ void piece(const K &k, int batch, int b, int &row, int &col) {
    using S = Shape<K>;
    const int idx = (batch * S::kBatch + b) * 64 + k.lane;
    row = idx / S::kPer;
    col = (idx - row * S::kPer) * 8;
  }
  template <class K, int N>
  __device__ __forceinline__ void load_res(const K &k, int batch, v4u (&r)[N]) const {
    const int mb = m0 + k.wave_m * K::kWM, nb = n0 + k.wave_n * Shape<K>::kOutN;
#pragma unroll
    for (int b = 0; b < N; ++b) {
      int row, col;
      piece(k, batch, b, row, col);
      // (Past the edge: the last valid piece again, unused.)
      const int m = min(mb + row, k.a.M - 1), n = min(nb + col, k.a.N - 8);
      r[b] = *(const v4u *)(t.res + ((size_t)m * t.ldr + n) * 2);
    }
  }

  __device__ static __forceinline__ void read8(const LDS_AS uint8_t *row, int r7, int c, int odd, float (&v)[8]) {
    const f32x4 lo = *(const LDS_AS f32x4 *)(row + ((c ^ r7) << 4));
    const f32x4 hi = *(const LDS_AS f32x4 *)(row + (((c + odd) ^ r7) << 4));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = lo[q];
      v[4 + q] = hi[q];
    }
  }
  __device__ __forceinline__ void add_bias(int n, float (&z)[8]) const {
    float v[8];
    unpack8<DT>(*(const v4u *)(t.bias + (size_t)n * 2), v);
#pragma unroll
    for (int q = 0; q < 8; ++q) z[q] += v[q];
  }

  template <int ACT, class K, int N>
  __device__ __forceinline__ void rows_out(K &k, const LDS_AS uint8_t *area, int ph, v4u (&r0)[N], v4u (&r1)[N]) const {
    using S = Shape<K>;
    constexpr int kWN = K::kWN, kOdd = kWN / 8, kBatches = S::kPieces / N;
    const int mb = m0 + k.wave_m * K::kWM, nb = n0 + k.wave_n * S::kOutN;
    const int M = k.a.M, Nc = k.a.N;
    float b0[8] = {}, b1[8] = {};
    if constexpr (S::kOneColumn)
      if (t.bias) {
        int row, col;
        piece(k, 0, 0, row, col);
        const int n = min(nb + col, Nc - 8);
        add_bias(n, b0);
        if constexpr (GATED) add_bias(t.half + n, b1);
      }
#pragma unroll 1
    for (int i = 0; i < kBatches; ++i) {
      const int batch = ph * kBatches + i;
      v4u res[N];
#pragma unroll
      for (int b = 0; b < N; ++b) {
        res[b] = r0[b];
        r0[b] = r1[b];
      }
      if (t.res && batch + 2 < kBatches * (K::kWM / S::kRows)) load_res(k, batch + 2, r1);
      float z[N][8], u[N][8];
      int m[N], n[N];
#pragma unroll
      for (int b = 0; b < N; ++b) {
        int row, col;
        piece(k, batch, b, row, col);
        m[b] = mb + row;
        n[b] = nb + col;
        row -= ph * S::kRows;
        const LDS_AS uint8_t *lr = area + row * (kWN * 4);
        if constexpr (GATED) {
          const int c = 4 * (col >> 4) + ((col >> 3) & 1);
          read8(lr, row & 7, c, kOdd, z[b]);
          read8(lr, row & 7, c + 2, kOdd, u[b]);
        } else {
          read8(lr, row & 7, col >> 3, kOdd, z[b]);
        }
      }
      if (t.bias) {
#pragma unroll
        for (int b = 0; b < N; ++b) {
          if constexpr (S::kOneColumn) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              z[b][q] += b0[q];
              if constexpr (GATED) u[b][q] += b1[q];
            }
          } else {
            add_bias(min(n[b], Nc - 8), z[b]);
            if constexpr (GATED) add_bias(t.half + min(n[b], Nc - 8), u[b]);
          }
        }
      }
      if (t.pre) {
#pragma unroll
        for (int b = 0; b < N; ++b) {
          uint8_t *p = t.pre + ((size_t)m[b] * t.ldp + n[b]) * 2;
          const v4u zw = pack8<DT>(z[b]);
          v4u uw;
          if constexpr (GATED) uw = pack8<DT>(u[b]);
          if (m[b] < M && n[b] < Nc) {
            *(v4u *)p = zw;
            if constexpr (GATED) *(v4u *)(p + (size_t)t.half * 2) = uw;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < N; ++b) {
        float rv[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          z[b][q] = act_fwd<ACT>(z[b][q]);
          if constexpr (GATED) z[b][q] *= u[b][q];
        }
        if (t.res) {
          unpack8<DT>(res[b], rv);
#pragma unroll
          for (int q = 0; q < 8; ++q) z[b][q] += rv[q];
        }
      }
#pragma unroll
      for (int b = 0; b < N; ++b) {
        const v4u w = pack8<DT>(z[b]);
        if (m[b] < M && n[b] < Nc) *(v4u *)(k.a.C + ((size_t)m[b] * k.a.ldc + n[b]) * 2) = w;
      }
    }
  }
};

// Products with nothing to do but the rounding: the plain epilogue, straight
// from the accumulators.  (An instance of its own: as a branch in FfnExt's it
// made the compiler spill accumulators, and lose one.)
struct PlainExt {
  static constexpr bool kOn = true, kGated = false, kGather = true, kPrefetch = true;
  int m0, n0;
  int half;
  const int32_t *rows;
  int src_rows;
  Tail t;
  template <class K>
  __device__ __forceinline__ void store(K &k) const {
    k.epilogue();
  }
};

// A gated activation alone: both values of an output lie in one lane's
// accumulators (blocks i and i + 1), so it goes straight from them, as the
// plain epilogue does.
template <int DT, bool GROUPED>
struct GatedExt {
  static constexpr bool kOn = true, kGated = true, kGather = GROUPED, kPrefetch = true;
  int m0, n0;
  int half;
  const int32_t *rows;
  int src_rows;
  Tail t;

  template <class K>
  __device__ __forceinline__ void store(K &k) const {
    with_act<true>(t.act, [&](auto act) { store_act<decltype(act)::value>(k); });
  }
  template <int ACT>
  __device__ static __forceinline__ u32x2 value4(const f32x4 &g, const f32x4 &u) {
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = act_fwd<ACT>(g[r]) * u[r];
    return u32x2{pack2<DT>(y[0], y[1]), pack2<DT>(y[2], y[3])};
  }
  template <int ACT, class K>
  __device__ __forceinline__ void store_act(K &k) const {
    const int q = k.lane >> 4;
#pragma unroll
    for (int j = 0; j < K::kNBm; ++j) {
      const int m = m0 + k.wave_m * K::kWM + j * 16 + (k.lane & 15);
      uint8_t *crow = k.a.C + (size_t)m * k.a.ldc * 2;
      const int nb = n0 + k.wave_n * (K::kWN / 2);
      if constexpr (K::kNBn == 2) {
        const u32x2 x = value4<ACT>(k.acc[0][j], k.acc[1][j]);
        const int n = nb + 4 * q;
        if (m < k.a.M && n < k.a.N) *(u32x2 *)(crow + (size_t)n * 2) = x;
      } else {
        // Two blocks of outputs: lane swaps leave each lane 8 columns of them
        // (as the plain epilogue's).
#pragma unroll
        for (int i = 0; i < K::kNBn; i += 4) {
          const u32x2 x = value4<ACT>(k.acc[i][j], k.acc[i + 1][j]), y = value4<ACT>(k.acc[i + 2][j], k.acc[i + 3][j]);
          uint32_t xo[2], yo[2];
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const auto h = __builtin_amdgcn_permlane32_swap(x[d], y[d], false, false);
            const auto r = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
            xo[d] = r[0];
            yo[d] = r[1];
          }
          const int n = nb + (i / 2) * 16 + 8 * q;
          if (m < k.a.M && n < k.a.N) store_c(crow + (size_t)n * 2, u32x4{xo[0], xo[1], yo[0], yo[1]});
        }
      }
    }
  }
};

// The grouped product over rows: the plain epilogue.
struct TnExt {
  static constexpr bool kOn = true, kGated = false, kGather = false, kPrefetch = true;
  int m0, n0;
  template <class K>
  __device__ __forceinline__ void store(K &k) const {
    k.epilogue();
  }
};

// Workgroups that share an XCD take consecutive tiles (as tile_of).
__device__ __forceinline__ int xcd_order(int wg, int total) {
  const int xcd = wg & 7, base = total >> 3, rem = total & 7;
  return xcd * base + min(xcd, rem) + (wg >> 3);
}

// Tile v of a group's tiles_m x tiles_n: groups of kGroupM tile rows, column
// by column (as tile_of).
__device__ __forceinline__ void tile_in_group(int v, int tiles_m, int tiles_n, int &tm, int &tn) {
  const int strip = v / (kGroupM * tiles_n);
  const int first = strip * kGroupM;
  const int rows = min(tiles_m - first, kGroupM);
  const int in = v - strip * kGroupM * tiles_n;
  tm = first + in % rows;
  tn = in / rows;
}

#define TGEMM_FFN_SLOTS(TM, TN)                                                \
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[TM * kRowBytes];       \
  __shared__ __attribute__((aligned(1024))) uint8_t sA1[TM * kRowBytes];       \
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[TN * kRowBytes];       \
  __shared__ __attribute__((aligned(1024))) uint8_t sB1[TN * kRowBytes];       \
  Slots slots;                                                                 \
  slots.a[0] = (LDS_AS uint8_t *)sA0;                                          \
  slots.a[1] = (LDS_AS uint8_t *)sA1;                                          \
  slots.b[0] = (LDS_AS uint8_t *)sB0;                                          \
  slots.b[1] = (LDS_AS uint8_t *)sB1;                                          \
  __shared__ __attribute__((aligned(256))) uint8_t junk[4 * 256];              \
  slots.junk = (LDS_AS uint8_t *)junk;                                         \
  slots.stage = nullptr;                                                       \
  if constexpr (kSlots<T, TM, TN> == 4) {                                      \
    __shared__ __attribute__((aligned(1024))) uint8_t sA2[TM * kRowBytes];     \
    __shared__ __attribute__((aligned(1024))) uint8_t sA3[TM * kRowBytes];     \
    __shared__ __attribute__((aligned(1024))) uint8_t sB2[TN * kRowBytes];     \
    __shared__ __attribute__((aligned(1024))) uint8_t sB3[TN * kRowBytes];     \
    slots.a[2] = (LDS_AS uint8_t *)sA2;                                        \
    slots.a[3] = (LDS_AS uint8_t *)sA3;                                        \
    slots.b[2] = (LDS_AS uint8_t *)sB2;                                        \
    slots.b[3] = (LDS_AS uint8_t *)sB3;                                        \
  }

// FUSED: with the operands of the epilogue (bias, residual, preact); else only
// its activation, gated, or (grouped) none.
template <class T, int TM, int TN, bool GATED, bool FUSED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void epilogue_kernel(const Args a, const Tail t) {
#if defined(__HIP_DEVICE_COMPILE__)
  TGEMM_FFN_SLOTS(TM, TN)
  int tm, tn;
  tile_of((int)blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, tm, tn);
  using X = typename std::conditional<FUSED, FfnExt<T::kDt, GATED, false, (TM < TN ? TM : TN) * kRowBytes>,
                                      GatedExt<T::kDt, false>>::type;
  const X x{tm * TM, tn * (GATED ? TN / 2 : TN), t.half, nullptr, 0, t};
  Kernel<T, TM, TN, false, X> k(a, slots, x);
  k.run();
#endif
}

// A group's rows are cut into tiles of TM rows; with 256-row tiles a last one
// of at most 128 rows is a tile of 128 x TN of its own (about 0.6 of the
// time), and those come after all the others, to fill the last wave of
// workgroups.  (16 groups of 152 to 1152 rows, 2048 columns, K = 1536: 40 row
// tiles, 9 of them short: 77 -> 69 us.)
template <int TM>
struct GroupTiles {
  static constexpr int kShort = TM == 256 ? 128 : 0;  // rows of a short tile; 0: there are none
  const Groups &g;
  int lane;
  // Units (tiles) of a group of n rows: whole ones, or the short one.
  template <bool SHORT>
  __device__ __forceinline__ int units(int n) const {
    const int rest = n % TM;
    const bool has = rest > 0 && rest <= kShort;
    if (SHORT) return has ? g.tiles_n : 0;
    return ((n + TM - 1) / TM - (has ? 1 : 0)) * g.tiles_n;
  }
  template <bool SHORT>
  __device__ __forceinline__ int total() const {
    return sum_units(g.offsets, g.groups, g.R, lane, [&](int n) { return units<SHORT>(n); });
  }
  template <bool SHORT>
  __device__ __forceinline__ Found find(int index) const {
    return find_in(g.offsets, g.groups, g.R, index, lane, [&](int n) { return units<SHORT>(n); });
  }
};

// One tile of a group: M0 its first row in the group.
template <class T, int TM, int TN, bool GATED, bool FUSED, int AREA>
__device__ __forceinline__ void group_tile(const Args &a0, const Tail &t0, const Groups &g, const Slots &slots, const Found &f,
                                           int m0, int n0) {
  // The group's own product: its rows, its weight, its bias.
  Args a = a0;
  Tail t = t0;
  a.M = f.hi - f.lo;
  a.B += (size_t)f.e * (size_t)g.stride_b * 2;
  a.C += (size_t)f.lo * a.ldc * 2;
  if (!g.rows) a.A += (size_t)f.lo * a.lda * 2;
  if (t.bias) t.bias += (size_t)f.e * (size_t)g.stride_bias * 2;
  if (t.pre) t.pre += (size_t)f.lo * t.ldp * 2;
  using Bare = typename std::conditional<GATED, GatedExt<T::kDt, true>, PlainExt>::type;
  using X = typename std::conditional<FUSED, FfnExt<T::kDt, GATED, true, AREA>, Bare>::type;
  const X x{m0, n0, t.half, g.rows ? g.rows + f.lo : nullptr, g.src_rows, t};
  Kernel<T, TM, TN, false, X> k(a, slots, x);
  k.run();
}

template <class T, int TM, int TN, bool GATED, bool FUSED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void grouped_kernel(const Args a0, const Tail t0, const Groups g) {
#if defined(__HIP_DEVICE_COMPILE__)
  TGEMM_FFN_SLOTS(TM, TN)
  constexpr int kArea = (TM < TN ? TM : TN) * kRowBytes, kCols = GATED ? TN / 2 : TN;
  const GroupTiles<TM> tiles{g, (int)(threadIdx.x & 63)};
  const int wg = (int)blockIdx.x, whole = tiles.template total<false>();
  if (wg < whole) {
    const Found f = tiles.template find<false>(xcd_order(wg, whole));
    if (f.e < 0) return;
    int tm, tn;
    tile_in_group(f.unit, tiles.template units<false>(f.hi - f.lo) / g.tiles_n, g.tiles_n, tm, tn);
    group_tile<T, TM, TN, GATED, FUSED, kArea>(a0, t0, g, slots, f, __builtin_amdgcn_readfirstlane(tm * TM),
                                        __builtin_amdgcn_readfirstlane(tn * kCols));
  } else if constexpr (GroupTiles<TM>::kShort > 0) {
    const int shorts = tiles.template total<true>();
    if (wg - whole >= shorts) return;
    const Found f = tiles.template find<true>(xcd_order(wg - whole, shorts));
    if (f.e < 0) return;
    group_tile<T, GroupTiles<TM>::kShort, TN, GATED, FUSED, kArea>(a0, t0, g, slots, f, (f.hi - f.lo) / TM * TM, f.unit * kCols);
  }
#endif
}

struct TnGroups {
  const int32_t *offsets;
  int R, groups;
};

// The group of rank r by falling rows, for at most 64 groups (lane l's group
// is l); r itself with more, whose groups then go out in their own order.  The
// rank is a loop over the groups in every workgroup: it gains where groups are
// long (1024 x 1024, 64 groups of 36 to 1838 rows 129 us in their own order, 111 so;
// 16 of 32 to 1034, 2048 x 1536 83 and 82) and loses where they are many and short
// (64 of 7 to 375 rows 47 and 56).  Past 64: 72 groups of 5 to 291 rows 67, 128 of 8
// to 406 120.
__device__ __forceinline__ int group_of_rank(const TnGroups &g, int r, int lane) {
  if (g.groups > 64) return r;
  const Range own = group_rows(g.offsets, min(lane, g.groups - 1), g.R);
  const int n = lane < g.groups ? own.hi - own.lo : -1;
  int rank = 0;
  for (int e = 0; e < g.groups; ++e) {
    const int o = __builtin_amdgcn_readlane(n, e);
    rank += o > n || (o == n && e < lane);
  }
  return (int)__builtin_ctzll(__ballot(lane < g.groups && rank == r));
}

// A tile takes time with its group's rows, so tiles go out group by group,
// most rows first, and every XCD (workgroups 8 apart share one) gets an eighth
// of each group's tiles: consecutive ones of the group's order, which share
// panels in its L2.  (16 groups of 152 to 1152 rows, 1536 x 2048: groups given
// whole to an XCD 80 us, so 62 us.)
template <class T, int TM, int TN>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void grouped_tn_kernel(const Args a0, const TnGroups g) {
#if defined(__HIP_DEVICE_COMPILE__)
  TGEMM_FFN_SLOTS(TM, TN)
  const int lane = threadIdx.x & 63;
  const int tiles = a0.tiles_m * a0.tiles_n, wg = (int)blockIdx.x;
  const int rank = wg / tiles, i = wg - rank * tiles;
  // XCD x = wg % 8 gets tiles / 8 of the group's tiles, or one more for the
  // first tiles % 8 XCDs from that of the group's first workgroup on.
  const int x = wg & 7, s = (wg - i) & 7, base = tiles >> 3, more = tiles & 7;
  int v = x * base + (i >> 3);
#pragma unroll
  for (int o = 0; o < 7; ++o) v += o < x && ((o - s) & 7) < more;
  const int e = group_of_rank(g, rank, lane);
  int tm, tn;
  tile_in_group(v, a0.tiles_m, a0.tiles_n, tm, tn);
  const Range r = group_rows(g.offsets, e, g.R);
  const int lo = __builtin_amdgcn_readfirstlane(r.lo), n = __builtin_amdgcn_readfirstlane(r.hi - r.lo);
  Args a = a0;
  a.A += (size_t)lo * a.lda * 2;
  a.B += (size_t)lo * a.ldb * 2;
  a.C += (size_t)e * (size_t)a.M * (size_t)a.N * 2;
  if (n == 0) {
    // An empty group: zeros, a row of the tile at a time by TN / 8 lanes (64 empty
    // groups of 2048 x 2048: 92 us, 5.8 TB/s; through the K loop 202).
    constexpr int kPer = TN / 8;
    const int col = tn * TN + (int)threadIdx.x % kPer * 8, m1 = min(a.M, tm * TM + TM);
    if (col < a.N)
      for (int m = tm * TM + (int)threadIdx.x / kPer; m < m1; m += kThreads / kPer)
        *(v4u *)(a.C + ((size_t)m * a.N + col) * 2) = v4u{};
    return;
  }
  a.K = n;
  a.ksteps = (n + 63) / 64;
  Kernel<T, TM, TN, false, TnExt> k(a, slots, TnExt{tm * TM, tn * TN});
  k.run();
#endif
}

inline Args gemm_args(const Gemm &g) {
  Args a{};
  a.A = static_cast<const uint8_t *>(g.A);
  a.B = static_cast<const uint8_t *>(g.B);
  a.C = static_cast<uint8_t *>(g.C);
  a.M = (int)g.M;
  a.N = (int)(is_gated(g.act) ? g.N / 2 : g.N);  // output columns
  a.K = (int)g.K;
  a.lda = (int)g.lda;
  a.ldb = (int)g.ldb;
  a.ldc = (int)g.ldc;
  a.ksteps = (int)((g.K + 63) / 64);
  a.splits = 1;
  return a;
}
inline Tail gemm_tail(const Gemm &g) {
  return Tail{static_cast<const uint8_t *>(g.bias), static_cast<const uint8_t *>(g.residual),
              static_cast<uint8_t *>(g.preact), (int)g.ldr, (int)g.ldp, g.act,
              is_gated(g.act) ? (int)(g.N / 2) : 0};
}

// (A dispatch holds fewer than 2^32 work-items per dimension.)
inline bool grid_ok(int64_t wgs) { return wgs <= (int64_t)(UINT32_MAX / kThreads); }

template <class T, int TM, int TN, bool GATED>
hipError_t launch_tile(const Gemm &g) {
  Args a = gemm_args(g);
  Tail t = gemm_tail(g);
  constexpr int kCols = GATED ? TN / 2 : TN;
  a.tiles_n = (a.N + kCols - 1) / kCols;
  const bool bare = !g.bias && !g.residual && !g.preact && (GATED || g.act == kNone);
  if (g.groups == 0) {
    a.tiles_m = (int)((g.M + TM - 1) / TM);
    const int64_t wgs = (int64_t)a.tiles_m * a.tiles_n;
    if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
    void *args[] = {&a, &t};
    const void *fn = reinterpret_cast<const void *>(&epilogue_kernel<T, TM, TN, GATED, true>);
    if constexpr (GATED)
      if (bare) fn = reinterpret_cast<const void *>(&epilogue_kernel<T, TM, TN, true, false>);
    return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(kThreads), args, 0, g.stream);
  }
  if constexpr (T::kAK && !(TM == 256 && TN == 192)) {
    // The most tiles the groups can have: each one's last may be partial.
    const int64_t wgs = (g.M / TM + (g.groups < g.M ? g.groups : g.M)) * (int64_t)a.tiles_n;
    if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
    Groups gr{g.offsets, g.rows, (int)g.groups, (int)g.M, (int)g.src_rows, g.stride_b, g.stride_bias, a.tiles_n};
    void *args[] = {&a, &t, &gr};
    const void *fn = bare ? reinterpret_cast<const void *>(&grouped_kernel<T, TM, TN, GATED, false>)
                          : reinterpret_cast<const void *>(&grouped_kernel<T, TM, TN, GATED, true>);
    return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(kThreads), args, 0, g.stream);
  }
  return hipErrorInvalidValue;
}

// The K split: workgroup w computes tile w % tiles over its range of slices and
// leaves its sums in plane w / tiles of the workspace.
template <class T, int TM, int TN>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void split_kernel(const Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  TGEMM_FFN_SLOTS(TM, TN)
  Kernel<T, TM, TN, true> k(a, slots);
  k.run();
#endif
}

template <class T, int TM, int TN>
hipError_t launch_split_tile(const Gemm &g) {
  Args a = gemm_args(g);
  a.N = (int)g.N;  // the product's columns, gated or not
  a.tiles_m = (int)((g.M + TM - 1) / TM);
  a.tiles_n = (int)((g.N + TN - 1) / TN);
  a.ws = g.ws;
  a.kq = (a.ksteps + g.splits - 1) / g.splits;  // (epilogue_splits leaves no split empty)
  a.splits = g.splits;
  const int64_t wgs = (int64_t)a.tiles_m * a.tiles_n * a.splits;
  if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
  void *args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void *>(&split_kernel<T, TM, TN>), dim3((unsigned)wgs), dim3(kThreads),
                         args, 0, g.stream);
}

template <int DT>
hipError_t launch_split(const Gemm &g) {
  const bool ak = !g.trans_a, bk = g.trans_b;
  if (ak && bk) return launch_split_tile<Traits<DT, true, true>, 64, 64>(g);
  if (ak) return launch_split_tile<Traits<DT, true, false>, 64, 64>(g);
  if (bk) return launch_split_tile<Traits<DT, false, true>, 64, 64>(g);
  return launch_split_tile<Traits<DT, false, false>, 64, 64>(g);
}

template <int DT, bool AK, bool BK>
hipError_t launch_tiles(const Gemm &g, int tm, int tn) {
  using T = Traits<DT, AK, BK>;
  if constexpr (AK) {
    if (is_gated(g.act)) {
      if (tm == 256 && tn == 256) return launch_tile<T, 256, 256, true>(g);
      if (tm == 128 && tn == 128) return launch_tile<T, 128, 128, true>(g);
      if (tm == 64 && tn == 64) return launch_tile<T, 64, 64, true>(g);
      return hipErrorInvalidValue;
    }
  }
  if (tm == 256 && tn == 256) return launch_tile<T, 256, 256, false>(g);
  if constexpr (BK)
    if (tm == 256 && tn == 192) return launch_tile<T, 256, 192, false>(g);
  if (tm == 128 && tn == 128) return launch_tile<T, 128, 128, false>(g);
  if (tm == 64 && tn == 64) return launch_tile<T, 64, 64, false>(g);
  return hipErrorInvalidValue;
}

template <int DT>
hipError_t launch_layouts(const Gemm &g, int tm, int tn) {
  const bool ak = !g.trans_a, bk = g.trans_b;
  if (ak && bk) return launch_tiles<DT, true, true>(g, tm, tn);
  if (ak) return launch_tiles<DT, true, false>(g, tm, tn);
  if (bk) return launch_tiles<DT, false, true>(g, tm, tn);
  return launch_tiles<DT, false, false>(g, tm, tn);
}

template <int DT, int TM, int TN>
hipError_t launch_tn_tile(const GroupedTn &g) {
  using T = Traits<DT, false, false>;
  Args a{};
  a.A = static_cast<const uint8_t *>(g.X);
  a.B = static_cast<const uint8_t *>(g.Y);
  a.C = static_cast<uint8_t *>(g.out);
  a.M = (int)g.P;
  a.N = (int)g.Q;
  a.lda = (int)g.ldx;
  a.ldb = (int)g.ldy;
  a.ldc = (int)g.Q;
  a.splits = 1;
  a.tiles_m = (int)((g.P + TM - 1) / TM);
  a.tiles_n = (int)((g.Q + TN - 1) / TN);
  const int64_t wgs = g.groups * a.tiles_m * a.tiles_n;
  if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
  TnGroups gr{g.offsets, (int)g.R, (int)g.groups};
  void *args[] = {&a, &gr};
  return hipLaunchKernel(reinterpret_cast<const void *>(&grouped_tn_kernel<T, TM, TN>), dim3((unsigned)wgs),
                         dim3(kThreads), args, 0, g.stream);
}

template <int DT>
hipError_t launch_tn(const GroupedTn &g, int tm, int tn) {
  if (tm == 256 && tn == 256) return launch_tn_tile<DT, 256, 256>(g);
  if (tm == 128 && tn == 128) return launch_tn_tile<DT, 128, 128>(g);
  if (tm == 64 && tn == 64) return launch_tn_tile<DT, 64, 64>(g);
  return hipErrorInvalidValue;
}

}  // namespace
}  // namespace ffn
}  // namespace tgemm
