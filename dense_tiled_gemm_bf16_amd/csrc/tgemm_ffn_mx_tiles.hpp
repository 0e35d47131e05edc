// Tiled products of MXFP4 operands with a fused epilogue for gfx950, dense and
// grouped.  256 x 256 tiles take the MXFP4 K loop of tgemm_kernel.hpp; MxTile
// here is the kernel of smaller tiles, and of scale rows that do not start on
// a dword.  The epilogues are those of the 16-bit products
// (tgemm_ffn_tiles.hpp): sums, bias, activation and residual are binary32, C is
// rounded once.
#pragma once

#include "tgemm_ffn_tiles.hpp"

namespace tgemm {
namespace ffn {
namespace {

// The MXFP4 operands of the 256 x 256 kernel, C in bf16 or fp16.
template <bool F16>
struct MxTraits : Traits<kFp4, true, true, true> {
  static constexpr bool kOutF16 = F16;
};

typedef __attribute__((ext_vector_type(8))) int v8i;

struct MxSlots {
  LDS_AS uint8_t *a[4], *b[4];  // kNS slots of TM, TN rows x 256 bytes
  LDS_AS uint8_t *s[4];         // their scales: 256 bytes per 16 rows (B's blocks first), then the dwords behind them
};

// MxTile: TM x TN of C by 4 waves (2 x 2), K in slices of 512 elements (256
// bytes of a row) through a ring of kNS slots, rows and scales loaded into LDS
// directly.
//
// Lane l of the scaled v_mfma 16x16x128 takes row l % 16 and one block of 32
// elements.  Over the four products of a slice lane group g = l / 16 takes
// blocks 4 g .. 4 g + 3, block 4 g + s in product s, of both operands alike:
// its four scales of a slice are then one dword, byte s for product s, and no
// scale moves between lanes.  A slot row keeps block 4 g + s at 16-byte chunk
// (4 s + g) ^ (row % 16): 16 rows at one chunk, and 4 chunks of 4 rows, fall
// on different LDS banks.
//
// ALIGNED: every row's scales start on a dword.  If not, a lane loads the
// dword that holds its first scale and the one behind, and shifts.
template <int DT, int TM, int TN, bool ALIGNED, class EXT>
struct MxTile {
  static constexpr int kBlk = 16;
  static constexpr int kWM = TM / 2, kWN = TN / 2, kNBm = kWM / 16, kNBn = kWN / 16;
  static constexpr int kNS = TM * TN <= 64 * 64 ? 4 : 2;
  static constexpr int kLA = TM / 16, kLB = TN / 16;     // row load instructions of a wave and slice (4 rows each)
  static constexpr int kScaleBlocks = (TM + TN) / 16;    // scale load instructions of a slice, 16 rows each
  static constexpr int kLS = kScaleBlocks / 4, kPlanes = ALIGNED ? 1 : 2;
  static constexpr int kLoads = kLA + kLB + kLS * kPlanes;
  static constexpr int kScaleBytes = kScaleBlocks * 256 * kPlanes;
  static_assert(kLA % 4 == 0 && kLB % 4 == 0 && kScaleBlocks % 4 == 0, "whole instructions");
  static_assert((kNS - 1) * kLoads < 64, "vmcnt is 6 bits");

  const Args &a;
  MxSlots slots;
  EXT x;
  int lane, wave, wave_m, wave_n, m0, n0;
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  uint32_t offa[kLA], offb[kLB];
  int kcol[4];             // this lane's byte in a slice row, by instruction % 4
  uint32_t offs[kLS];      // aligned offset of this lane's scales in slice 0
  uint32_t sh_x[2], sh_y[EXT::kGather ? kNBm : 1];  // where this lane's scales start in their dword
  uint32_t frag;           // this lane's chunk of product 0
  f32x4 acc[kNBn][kNBm];

  __device__ __forceinline__ MxTile(const Args &args, const MxSlots &s, const EXT &ext) : a(args), slots(s), x(ext) {}

  // Row of B (from the tile's first on) that LDS row r holds, or -1.
  __device__ __forceinline__ int b_row(int r) const {
    if constexpr (EXT::kGated) {
      const int c = ((r >> 5) << 4) + (r & 15);
      return c < min(a.N - n0, TN / 2) ? c + ((r >> 4) & 1 ? x.half : 0) : -1;
    } else {
      return r < min(a.N - n0, TN) ? r : -1;
    }
  }
  // Row of A (of the array if gathered, else from the tile's first on) that
  // LDS row r holds, or -1.
  __device__ __forceinline__ int a_row(int r) const {
    if (r >= min(a.M - m0, TM)) return -1;
    if constexpr (EXT::kGather)
      if (x.rows) {
        const int s = x.rows[m0 + r];
        return s >= 0 && s < x.src_rows ? s : -1;
      }
    return r;
  }

  __device__ __forceinline__ void init() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    wave_m = wave >> 1;
    wave_n = wave & 1;
    m0 = x.m0;
    n0 = x.n0;
    bool gather = false;
    if constexpr (EXT::kGather) gather = x.rows != nullptr;
    int src = min(a.M - m0, TM);
    if constexpr (EXT::kGather) src = gather ? x.src_rows : src;
    const int brows = EXT::kGated ? ext_half() + min(a.N - n0, TN / 2) : min(a.N - n0, TN);
    ra = make_rsrc(a.A + (gather ? (size_t)0 : (size_t)m0 * a.lda),
                   src > 0 ? (uint32_t)(src - 1) * (uint32_t)a.lda + (uint32_t)a.K : 0u);
    rb = make_rsrc(a.B + (size_t)n0 * a.ldb, (uint32_t)(brows - 1) * (uint32_t)a.ldb + (uint32_t)a.K);
    // Scales: based at the dword that holds the first byte, up to the one that
    // holds the last.
    const uintptr_t pa = (uintptr_t)(a.SA + (gather ? (size_t)0 : (size_t)m0 * a.kb));
    const uintptr_t pb = (uintptr_t)(a.SB + (size_t)n0 * a.kb);
    const uint32_t mis_a = (uint32_t)(pa & 3), mis_b = (uint32_t)(pb & 3);
    rsa = make_rsrc((const void *)(pa - mis_a), src > 0 ? (mis_a + (uint32_t)src * (uint32_t)a.kb + 3u) & ~3u : 0u);
    rsb = make_rsrc((const void *)(pb - mis_b), (mis_b + (uint32_t)brows * (uint32_t)a.kb + 3u) & ~3u);

    const int r = lane & 15, g = lane >> 4;
    // Rows: lane l of instruction i writes chunk l % 16 of row 4 i + l / 16 of
    // the wave's rows, whose number % 16 goes by i % 4.
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int q = r ^ (4 * p + g);                  // chunk before the row's permutation: 4 s + g
      kcol[p] = 16 * (4 * (q & 3) + (q >> 2));
    }
#pragma unroll
    for (int i = 0; i < kLA; ++i) {
      const int row = a_row(4 * (wave * kLA + i) + g);
      offa[i] = row >= 0 ? (uint32_t)row * (uint32_t)a.lda + (uint32_t)kcol[i & 3] : kOOB;
    }
#pragma unroll
    for (int i = 0; i < kLB; ++i) {
      const int row = b_row(4 * (wave * kLB + i) + g);
      offb[i] = row >= 0 ? (uint32_t)row * (uint32_t)a.ldb + (uint32_t)kcol[i & 3] : kOOB;
    }
    // Scales: instruction i of wave w takes 16-row block kLS w + i, lane l the
    // dword of row l % 16 and lane group l / 16.
#pragma unroll
    for (int i = 0; i < kLS; ++i) {
      const int b = wave * kLS + i;
      const bool isb = b < kLB;
      const int row = isb ? b_row(16 * b + r) : a_row(16 * (b - kLB) + r);
      offs[i] = row >= 0 ? ((isb ? mis_b : mis_a) + (uint32_t)row * (uint32_t)a.kb + 4u * (uint32_t)g) & ~3u : kOOB;
    }
    if constexpr (!ALIGNED) {
      // (16 rows are 16 kb bytes: one shift for all blocks, of each half.)
      sh_x[0] = (mis_b + (uint32_t)r * (uint32_t)a.kb) & 3u;
      sh_x[1] = (mis_b + (uint32_t)(r + ext_half()) * (uint32_t)a.kb) & 3u;
      if constexpr (EXT::kGather) {
#pragma unroll
        for (int j = 0; j < kNBm; ++j)
          sh_y[j] = (mis_a + (uint32_t)max(a_row(wave_m * kWM + 16 * j + r), 0) * (uint32_t)a.kb) & 3u;
      } else {
        sh_y[0] = (mis_a + (uint32_t)r * (uint32_t)a.kb) & 3u;
      }
    }
    frag = (uint32_t)(r * 256 + ((g ^ r) << 4));
#pragma unroll
    for (int i = 0; i < kNBn; ++i)
#pragma unroll
      for (int j = 0; j < kNBm; ++j) acc[i][j] = f32x4{};
  }
  __device__ __forceinline__ int ext_half() const {
    if constexpr (EXT::kGated) return x.half;
    return 0;
  }

  // Every load of slice kt into slot S.  Slices past whole ones check columns:
  // what lies past K arrives as zeros, and a slice past the last is all zeros.
  template <int S>
  __device__ __forceinline__ void load(int kt) const {
    const uint32_t so = (uint32_t)kt * 256u;
    const int left = a.K - kt * 256;  // bytes of a row from this slice on
    const bool whole = left >= 256;
#pragma unroll
    for (int i = 0; i < kLA; ++i) {
      const uint32_t v = whole || kcol[i & 3] < left ? offa[i] : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LDS_AS void *)(slots.a[S] + (wave * kLA + i) * 1024), 16, v, so, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kLB; ++i) {
      const uint32_t v = whole || kcol[i & 3] < left ? offb[i] : kOOB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LDS_AS void *)(slots.b[S] + (wave * kLB + i) * 1024), 16, v, so, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kLS; ++i) {
      const int b = wave * kLS + i;
      const __amdgpu_buffer_rsrc_t rs = b < kLB ? rsb : rsa;
      const uint32_t v = left > 0 ? offs[i] : kOOB;
#pragma unroll
      for (int p = 0; p < kPlanes; ++p)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDS_AS void *)(slots.s[S] + (p * kScaleBlocks + b) * 256), 4, v,
                                                 (uint32_t)kt * 16u + 4u * (uint32_t)p, 0, 0);
    }
  }

  // This lane's scales of 16-row block b in slot S.
  template <int S>
  __device__ __forceinline__ uint32_t scale(int b, uint32_t sh, uint32_t keep) const {
    const LDS_AS uint8_t *p = slots.s[S] + b * 256 + lane * 4;
    uint32_t w = *(const LDS_AS uint32_t *)p;
    if constexpr (!ALIGNED) w = __builtin_amdgcn_alignbyte(*(const LDS_AS uint32_t *)(p + kScaleBlocks * 256), w, sh);
    return w & keep;
  }
  template <int SEL>
  __device__ static __forceinline__ f32x4 mma(const u32x4 &p, const u32x4 &q, const f32x4 &c, uint32_t sp, uint32_t sq) {
    const v8i p8 = {(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
    const v8i q8 = {(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p8, q8, c, 4, 4, SEL, (int)sp, SEL, (int)sq);
  }
  template <int S, int P>
  __device__ __forceinline__ void product(const uint32_t (&sx)[kNBn], const uint32_t (&sy)[kNBm]) {
    u32x4 px[kNBn], py[kNBm];
    const uint32_t at = frag ^ (uint32_t)(P << 6);
#pragma unroll
    for (int i = 0; i < kNBn; ++i) px[i] = *(const LDS_AS u32x4 *)(slots.b[S] + (wave_n * kWN + 16 * i) * 256 + at);
#pragma unroll
    for (int j = 0; j < kNBm; ++j) py[j] = *(const LDS_AS u32x4 *)(slots.a[S] + (wave_m * kWM + 16 * j) * 256 + at);
#pragma unroll
    for (int i = 0; i < kNBn; ++i)
#pragma unroll
      for (int j = 0; j < kNBm; ++j) acc[i][j] = mma<P>(px[i], py[j], acc[i][j], sx[i], sy[j]);
  }

  // Slice kt from slot S: its loads have landed in every wave behind the
  // barrier, and every wave's reads of the slot before it lie in front.
  template <int S>
  __device__ __forceinline__ void step(int kt) {
    wait_vm_lgkm0<(kNS - 2) * kLoads>();
    barrier();
    load<(S + kNS - 1) % kNS>(kt + kNS - 1);
    // The scales of the row from this lane's first on (behind them lies the
    // next row's: a NaN among them would meet the zeros past K).
    const int left = a.kb - 16 * kt - 4 * (lane >> 4);
    const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : ~0u >> (32 - 8 * left);
    uint32_t sx[kNBn], sy[kNBm];
#pragma unroll
    for (int i = 0; i < kNBn; ++i) sx[i] = scale<S>(wave_n * kNBn + i, sh_x[EXT::kGated ? i & 1 : 0], keep);
#pragma unroll
    for (int j = 0; j < kNBm; ++j) sy[j] = scale<S>(kLB + wave_m * kNBm + j, sh_y[EXT::kGather ? j : 0], keep);
    product<S, 0>(sx, sy);
    product<S, 1>(sx, sy);
    product<S, 2>(sx, sy);
    product<S, 3>(sx, sy);
  }

  __device__ __forceinline__ void run() {
    init();
    const int nk = (a.K + 255) >> 8;
    load<0>(0);
    if constexpr (kNS == 4) {
      load<1>(1);
      load<2>(2);
    }
    int kt = 0;
    if constexpr (kNS == 4) {
      for (; kt + 3 < nk; kt += 4) {
        step<0>(kt);
        step<1>(kt + 1);
        step<2>(kt + 2);
        step<3>(kt + 3);
      }
      if (kt < nk) step<0>(kt);
      if (kt + 1 < nk) step<1>(kt + 1);
      if (kt + 2 < nk) step<2>(kt + 2);
    } else {
      for (; kt + 1 < nk; kt += 2) {
        step<0>(kt);
        step<1>(kt + 1);
      }
      if (kt < nk) step<0>(kt);
    }
    // The loads still in flight into the slots.
    wait_vm_lgkm0<0>();
    x.store(*this);
  }

  // The rounding alone (see the plain products' epilogue): lane swaps leave a
  // lane 8 columns of a row.
  __device__ __forceinline__ void epilogue() {
    static_assert(kNBn % 2 == 0, "blocks pair up along N");
    const int q = lane >> 4;
#pragma unroll
    for (int j = 0; j < kNBm; ++j) {
      const int m = m0 + wave_m * kWM + j * 16 + (lane & 15);
      uint8_t *crow = a.C + (size_t)m * a.ldc * 2;
#pragma unroll
      for (int i = 0; i < kNBn; i += 2) {
        const f32x4 &u = acc[i][j], &v = acc[i + 1][j];
        const uint32_t us[2] = {pack2<DT>(u[0], u[1]), pack2<DT>(u[2], u[3])};
        const uint32_t vs[2] = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
        uint32_t xo[2], yo[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const auto h = __builtin_amdgcn_permlane32_swap(us[d], vs[d], false, false);
          const auto r = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
          xo[d] = r[0];
          yo[d] = r[1];
        }
        const int n = n0 + wave_n * kWN + i * 16 + 8 * q;
        if (m < a.M && n < a.N) store_c(crow + (size_t)n * 2, u32x4{xo[0], xo[1], yo[0], yo[1]});
      }
    }
  }
};

#define TGEMM_MX_SLOTS(TM, TN, NS, SCALES)                                  \
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[TM * 256];          \
  __shared__ __attribute__((aligned(1024))) uint8_t sA1[TM * 256];          \
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[TN * 256];          \
  __shared__ __attribute__((aligned(1024))) uint8_t sB1[TN * 256];          \
  __shared__ __attribute__((aligned(1024))) uint8_t sS0[SCALES];            \
  __shared__ __attribute__((aligned(1024))) uint8_t sS1[SCALES];            \
  MxSlots slots;                                                            \
  slots.a[0] = (LDS_AS uint8_t *)sA0;                                       \
  slots.a[1] = (LDS_AS uint8_t *)sA1;                                       \
  slots.b[0] = (LDS_AS uint8_t *)sB0;                                       \
  slots.b[1] = (LDS_AS uint8_t *)sB1;                                       \
  slots.s[0] = (LDS_AS uint8_t *)sS0;                                       \
  slots.s[1] = (LDS_AS uint8_t *)sS1;                                       \
  if constexpr (NS == 4) {                                                  \
    __shared__ __attribute__((aligned(1024))) uint8_t sA2[TM * 256];        \
    __shared__ __attribute__((aligned(1024))) uint8_t sA3[TM * 256];        \
    __shared__ __attribute__((aligned(1024))) uint8_t sB2[TN * 256];        \
    __shared__ __attribute__((aligned(1024))) uint8_t sB3[TN * 256];        \
    __shared__ __attribute__((aligned(1024))) uint8_t sS2[SCALES];          \
    __shared__ __attribute__((aligned(1024))) uint8_t sS3[SCALES];          \
    slots.a[2] = (LDS_AS uint8_t *)sA2;                                     \
    slots.a[3] = (LDS_AS uint8_t *)sA3;                                     \
    slots.b[2] = (LDS_AS uint8_t *)sB2;                                     \
    slots.b[3] = (LDS_AS uint8_t *)sB3;                                     \
    slots.s[2] = (LDS_AS uint8_t *)sS2;                                     \
    slots.s[3] = (LDS_AS uint8_t *)sS3;                                     \
  }

// FUSED: with the operands of the epilogue or an activation that is not gated;
// else a gated activation alone, or none.
template <int DT, bool GATED, bool GROUPED, bool FUSED, int AREA>
using MxExt = typename std::conditional<
    FUSED, FfnExt<DT, GATED, GROUPED, AREA>,
    typename std::conditional<GATED, GatedExt<DT, GROUPED>, PlainExt>::type>::type;

// One tile with its first row m0 and first column n0, by the kernel of its size.
template <int DT, int TM, int TN, bool ALIGNED, class X>
__device__ __forceinline__ void mx_tile(const Args &a, const X &x) {
  if constexpr (TM == 256) {
    using T = MxTraits<DT == 1>;
    __shared__ __attribute__((aligned(1024))) uint8_t sA0[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sA1[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sB0[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sB1[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t st[Kernel<T, 256, 256, false, X>::kStageBytes];
    Slots slots;
    slots.a[0] = (LDS_AS uint8_t *)sA0;
    slots.a[1] = (LDS_AS uint8_t *)sA1;
    slots.b[0] = (LDS_AS uint8_t *)sB0;
    slots.b[1] = (LDS_AS uint8_t *)sB1;
    slots.junk = nullptr;
    slots.stage = (LDS_AS uint8_t *)st;
    Kernel<T, 256, 256, false, X> k(a, slots, x);
    k.run();
  } else {
    using K = MxTile<DT, TM, TN, ALIGNED, X>;
    TGEMM_MX_SLOTS(TM, TN, K::kNS, K::kScaleBytes)
    K k(a, slots, x);
    k.run();
  }
}

template <int DT, int TM, int TN, bool ALIGNED, bool GATED, bool FUSED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mx_epilogue_kernel(const Args a, const Tail t) {
#if defined(__HIP_DEVICE_COMPILE__)
  int tm, tn;
  tile_of((int)blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, tm, tn);
  constexpr int kArea = (TM < TN ? TM : TN) * (TM == 256 ? 128 : 256);
  const MxExt<DT, GATED, false, FUSED, kArea> x{tm * TM, tn * (GATED ? TN / 2 : TN), t.half, nullptr, 0, t};
  mx_tile<DT, TM, TN, ALIGNED>(a, x);
#endif
}

struct MxGroups {
  const int32_t *offsets;
  const int32_t *rows;  // or nullptr
  int groups, R, src_rows;
  int64_t stride_b, stride_sb, stride_bias;  // bytes, bytes, elements
};

template <int DT, int TM, int TN, bool ALIGNED, bool GATED, bool FUSED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mx_grouped_kernel(const Args a0, const Tail t0, const MxGroups g) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63;
  const int wg = (int)blockIdx.x, total = total_units(g.offsets, g.groups, g.R, TM, a0.tiles_n, lane);
  if (wg >= total) return;
  const Found f = find_unit(g.offsets, g.groups, g.R, xcd_order(wg, total), TM, a0.tiles_n, lane);
  if (f.e < 0) return;
  int tm, tn;
  tile_in_group(f.unit, (f.hi - f.lo + TM - 1) / TM, a0.tiles_n, tm, tn);
  // The group's own product: its rows, its weight, its bias.
  Args a = a0;
  Tail t = t0;
  a.M = f.hi - f.lo;
  a.B += (size_t)f.e * (size_t)g.stride_b;
  a.SB += (size_t)f.e * (size_t)g.stride_sb;
  a.C += (size_t)f.lo * a.ldc * 2;
  if (!g.rows) {
    a.A += (size_t)f.lo * a.lda;
    a.SA += (size_t)f.lo * a.kb;
  }
  if (t.bias) t.bias += (size_t)f.e * (size_t)g.stride_bias * 2;
  if (t.pre) t.pre += (size_t)f.lo * t.ldp * 2;
  constexpr int kArea = (TM < TN ? TM : TN) * (TM == 256 ? 128 : 256);
  const MxExt<DT, GATED, true, FUSED, kArea> x{__builtin_amdgcn_readfirstlane(tm * TM),
                                               __builtin_amdgcn_readfirstlane(tn * (GATED ? TN / 2 : TN)), t.half,
                                               g.rows ? g.rows + f.lo : nullptr, g.src_rows, t};
  mx_tile<DT, TM, TN, ALIGNED>(a, x);
#endif
}

template <int DT, int TM, int TN, bool ALIGNED, bool GATED>
hipError_t launch_mx_tile(const MxGemm &g) {
  Args a{};
  a.A = static_cast<const uint8_t *>(g.A);
  a.B = static_cast<const uint8_t *>(g.B);
  a.SA = static_cast<const uint8_t *>(g.SA);
  a.SB = static_cast<const uint8_t *>(g.SB);
  a.C = static_cast<uint8_t *>(g.C);
  a.M = (int)g.M;
  a.N = (int)(GATED ? g.N / 2 : g.N);
  a.K = (int)(g.K / 2);  // bytes
  a.lda = (int)g.lda;
  a.ldb = (int)g.ldb;
  a.ldc = (int)g.ldc;
  a.kb = (int)(g.K / 32);
  a.ksteps = (int)(g.K / 256);  // (256-row tiles)
  a.splits = 1;
  constexpr int kCols = GATED ? TN / 2 : TN;
  a.tiles_m = (int)((g.M + TM - 1) / TM);
  a.tiles_n = (a.N + kCols - 1) / kCols;
  Tail t{static_cast<const uint8_t *>(g.bias), static_cast<const uint8_t *>(g.residual), static_cast<uint8_t *>(g.preact),
         (int)g.ldr, (int)g.ldp, g.act, GATED ? a.N : 0};
  // (A gated 256 x 256 tile straight from the accumulators would spill.)
  const bool fused = g.bias || g.residual || g.preact || (GATED ? TM == 256 : g.act != kNone);
  constexpr bool kBare = !(GATED && TM == 256);
  if (g.groups == 0) {
    const int64_t wgs = (int64_t)a.tiles_m * a.tiles_n;
    if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
    void *args[] = {&a, &t};
    const void *fn = reinterpret_cast<const void *>(&mx_epilogue_kernel<DT, TM, TN, ALIGNED, GATED, true>);
    if constexpr (kBare)
      if (!fused) fn = reinterpret_cast<const void *>(&mx_epilogue_kernel<DT, TM, TN, ALIGNED, GATED, false>);
    return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(kThreads), args, 0, g.stream);
  }
  // The most tiles the groups can have: each one's last may be partial.
  const int64_t wgs = (g.M / TM + (g.groups < g.M ? g.groups : g.M)) * (int64_t)a.tiles_n;
  if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
  MxGroups gr{g.offsets, g.rows, (int)g.groups, (int)g.M, (int)g.src_rows, g.stride_b, g.stride_sb, g.N};
  void *args[] = {&a, &t, &gr};
  const void *fn = reinterpret_cast<const void *>(&mx_grouped_kernel<DT, TM, TN, ALIGNED, GATED, true>);
  if constexpr (kBare)
    if (!fused) fn = reinterpret_cast<const void *>(&mx_grouped_kernel<DT, TM, TN, ALIGNED, GATED, false>);
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(kThreads), args, 0, g.stream);
}

template <int DT, int TM, int TN, bool ALIGNED>
hipError_t launch_mx_gated(const MxGemm &g) {
  return is_gated(g.act) ? launch_mx_tile<DT, TM, TN, ALIGNED, true>(g) : launch_mx_tile<DT, TM, TN, ALIGNED, false>(g);
}

template <int DT>
hipError_t launch_mx_tiles_dt(const MxGemm &g, int tm) {
  if (tm == 256) return launch_mx_gated<DT, 256, 256, true>(g);
  const bool aligned = mx_scales_aligned(g);
  if (tm == 128) return aligned ? launch_mx_gated<DT, 128, 128, true>(g) : launch_mx_gated<DT, 128, 128, false>(g);
  return aligned ? launch_mx_gated<DT, 64, 64, true>(g) : launch_mx_gated<DT, 64, 64, false>(g);
}

}  // namespace
}  // namespace ffn
}  // namespace tgemm
