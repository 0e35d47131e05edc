// Products of MXFP4 operands with few rows and an epilogue, dense or grouped,
// for gfx950: single tokens and small batches against 4-bit weights (N x K).
//
// What bounds such a product is reading the weight once, 17 bytes per 32
// elements (220 rows of 64 experts of 2048 x 1024 19.5 us, 3.5 TB/s), and below some
// megabytes the latency of a launch and one load (4096 x 1024 2.9).  A workgroup
// takes 16 NB rows of the weight (columns of C) and up to 16 rows of A, and its W waves divide K: wave w takes units of 512 K
// elements (256 bytes of each row) w, w + W, ...  Rows and scales go from
// memory straight into the registers of the scaled v_mfma 16x16x128: in
// product s of a unit lane l holds row l % 16 and block 4 s + l / 16 of 32
// elements.  A lane loads its row's 16 scale bytes of the unit and picks every
// fourth, one for each product.  (Blocks 4 (l / 16) + s instead, whose scales are a
// dword as it lies, made a lane's loads 64 bytes of one row: 10% slower.)  The
// waves' sums meet in LDS, are added in wave order (the result does not depend
// on timing) and pass through the epilogue.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tgemm_ffn_math.hpp"

namespace tgemm {
namespace ffn {
namespace {

typedef __attribute__((ext_vector_type(8))) int v8i;

constexpr uint32_t kOOB = 0x80000000u;  // an offset past every resource

struct MxRowsArgs {
  const uint8_t *A, *SA, *B, *SB;
  uint8_t *C;
  const uint8_t *bias, *res;
  uint8_t *pre;
  int M, N, K;  // N: output columns
  int lda, ldb, ldc, ldr, ldp;
  int kb;  // scales of a row
  int act, half;
  int tiles_m, tiles_n;  // dense
  // grouped
  const int32_t *offsets, *rows;
  int groups, src_rows;
  int64_t stride_b, stride_sb;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, 0x00020000);
}

// Product S of a unit: byte S of the scale dwords.
template <int S>
__device__ __forceinline__ v4f mfma(const v4u &x, const v4u &y, const v4f &c, uint32_t sx, uint32_t sy) {
  const v8i x8 = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  const v8i y8 = {(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x8, y8, c, 4, 4, S, (int)sx, S, (int)sy);
}

template <int DT>
__device__ __forceinline__ void store4(uint8_t *p, const float (&v)[4]) {
  *(v2u *)p = v2u{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}

constexpr int kTM = 16;

// The scale rows of one operand.  A row's 16 scales of a unit need not start
// on a dword (rows of K / 32 bytes, from any address): a lane loads from the
// dword that holds the first on, one more, and shifts.  The resource is based
// at the dword that holds the first row's first byte and ends with the one that
// holds the last row's last.
struct ScaleRows {
  __amdgpu_buffer_rsrc_t r;
  uint32_t mis;
  // rows: as many as the resource spans.
  __device__ __forceinline__ void init(const uint8_t *p, uint32_t rows, int kb) {
    const uintptr_t at = (uintptr_t)p;
    mis = (uint32_t)(at & 3);
    r = rsrc_of((const void *)(at - mis), rows ? (mis + rows * (uint32_t)kb + 3u) & ~3u : 0u);
  }
};
struct ScaleWords {
  v4u w;
  uint32_t next;
};
struct ScaleLane {
  uint32_t off, sh;  // the row's aligned offset in unit 0 (or kOOB), the byte it starts at
  __device__ __forceinline__ void init(const ScaleRows &s, bool in, uint32_t row, int kb) {
    const uint32_t pos = s.mis + row * (uint32_t)kb;
    off = in ? pos & ~3u : kOOB;
    sh = pos & 3u;
  }
  __device__ __forceinline__ ScaleWords load(const ScaleRows &s, uint32_t u) const {
    return {__builtin_amdgcn_raw_buffer_load_b128(s.r, off, 16u * u, 0),
            __builtin_amdgcn_raw_buffer_load_b32(s.r, off, 16u * u + 16u, 0)};
  }
  // pick: bytes g and 4 + g of two dwords.
  __device__ __forceinline__ uint32_t get(const ScaleWords &c, uint32_t pick, uint32_t keep) const {
    const uint32_t w0 = __builtin_amdgcn_alignbyte(c.w[1], c.w[0], sh), w1 = __builtin_amdgcn_alignbyte(c.w[2], c.w[1], sh);
    const uint32_t w2 = __builtin_amdgcn_alignbyte(c.w[3], c.w[2], sh), w3 = __builtin_amdgcn_alignbyte(c.next, c.w[3], sh);
    const uint32_t lo = __builtin_amdgcn_perm(w1, w0, pick), hi = __builtin_amdgcn_perm(w3, w2, pick);
    return (lo | hi << 16) & keep;
  }
};

template <int DT, int W, int NB, bool GATED, bool GROUPED>
__global__ __launch_bounds__(64 * W) void mx_rows_kernel(const MxRowsArgs a) {
  constexpr int kOutB = GATED ? NB / 2 : NB, kCols = 16 * kOutB;
  static_assert(kOutB <= W, "an output piece a thread");
  __shared__ v4f part[W][NB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);

  // The tile: rows m0 .. of M (M counts from row `lo` on), columns n0 ...
  const uint8_t *A = a.A, *SA = a.SA, *B = a.B, *SB = a.SB, *bias = a.bias;
  int M = a.M, lo = 0, m0, n0;
  if constexpr (GROUPED) {
    const Found f = find_unit(a.offsets, a.groups, a.M, (int)blockIdx.x, kTM, a.tiles_n, lane);
    if (f.e < 0) return;
    M = f.hi - f.lo;
    lo = f.lo;
    const int tiles_m = (M + kTM - 1) / kTM;
    n0 = f.unit / tiles_m * kCols;
    m0 = (f.unit % tiles_m) * kTM;
    B += (size_t)f.e * (size_t)a.stride_b;
    SB += (size_t)f.e * (size_t)a.stride_sb;
    if (bias) bias += (size_t)f.e * (size_t)(GATED ? 2 * a.N : a.N) * 2;
  } else {
    m0 = (int)blockIdx.x % a.tiles_m * kTM;
    n0 = (int)blockIdx.x / a.tiles_m * kCols;
  }

  // Lane l's row of every block and its four blocks of 32 elements of a unit.
  const int r = lane & 15, g = lane >> 4;
  const int cols = min(a.N - n0, kCols);
  const uint32_t row_bytes = (uint32_t)a.K >> 1;
  const auto rb = rsrc_of(B + (size_t)n0 * a.ldb, (uint32_t)((GATED ? a.half : 0) + cols - 1) * (uint32_t)a.ldb + row_bytes);
  ScaleRows srb, sra;
  srb.init(SB + (size_t)n0 * a.kb, (uint32_t)((GATED ? a.half : 0) + cols), a.kb);
  uint32_t boff[NB], aoff;
  ScaleLane sb[NB], sa;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int c = (GATED ? b >> 1 : b) * 16 + r;
    const uint32_t row = (uint32_t)(c + (GATED && (b & 1) ? a.half : 0));
    boff[b] = c < cols ? row * (uint32_t)a.ldb + 16u * (uint32_t)g : kOOB;
    sb[b].init(srb, c < cols, row, a.kb);
  }
  __amdgpu_buffer_rsrc_t ra;
  if (GROUPED && a.rows) {
    ra = rsrc_of(A, a.src_rows > 0 ? (uint32_t)(a.src_rows - 1) * (uint32_t)a.lda + row_bytes : 0u);
    sra.init(SA, (uint32_t)a.src_rows, a.kb);
    const int src = m0 + r < M ? a.rows[lo + m0 + r] : -1;
    const bool in = src >= 0 && src < a.src_rows;
    aoff = in ? (uint32_t)src * (uint32_t)a.lda + 16u * (uint32_t)g : kOOB;
    sa.init(sra, in, in ? (uint32_t)src : 0u, a.kb);
  } else {
    const int rows = min(M - m0, kTM);
    ra = rsrc_of(A + (size_t)(lo + m0) * a.lda, (uint32_t)(rows - 1) * (uint32_t)a.lda + row_bytes);
    sra.init(SA + (size_t)(lo + m0) * a.kb, (uint32_t)rows, a.kb);
    aoff = r < rows ? (uint32_t)r * (uint32_t)a.lda + 16u * (uint32_t)g : kOOB;
    sa.init(sra, r < rows, (uint32_t)r, a.kb);
  }

  // This thread's piece of the output: lane l of wave ob holds row l % 16,
  // columns 4 (l / 16) .. + 3 of output block ob.
  const int m = m0 + r, c = 16 * wave + 4 * g, n = n0 + c;
  const bool mine = wave < kOutB && m < M && c < cols;
  const size_t row = (size_t)(lo + m);
  v2u bias0 = {}, bias1 = {}, res = {};
  if (mine) {
    if (bias) {
      bias0 = *(const v2u *)(bias + (size_t)n * 2);
      if constexpr (GATED) bias1 = *(const v2u *)(bias + (size_t)(a.half + n) * 2);
    }
    if (a.res) res = *(const v2u *)(a.res + (row * a.ldr + n) * 2);
  }

  v4f acc[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) acc[i] = v4f{};
  const int units = (a.K + 511) >> 9;
  const uint32_t pick = 0x0c0c0400u + 0x0101u * (uint32_t)g;
  // One unit at a time: the next one's loads wait for it, but the registers
  // that holding both would take are worth more as further waves.
  for (int u = wave; u < units; u += W) {
    v4u x[4][NB], y[4];
    ScaleWords wx[NB], wy;
    // (K % 32 == 0: a block is all inside K or all outside, where both operands
    // read zeros.  The weights' loads first: A's wait for its row's index.)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bool in = 512 * u + 128 * s + 32 * g < a.K;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        x[s][b] = __builtin_amdgcn_raw_buffer_load_b128(rb, in ? boff[b] : kOOB, (uint32_t)u * 256u + 64u * (uint32_t)s, 0);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) wx[b] = sb[b].load(srb, (uint32_t)u);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bool in = 512 * u + 128 * s + 32 * g < a.K;
      y[s] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? aoff : kOOB, (uint32_t)u * 256u + 64u * (uint32_t)s, 0);
    }
    wy = sa.load(sra, (uint32_t)u);
    __builtin_amdgcn_sched_barrier(0);  // (all on their way before the products)
    // Blocks of the row from this lane's first of the unit on, four apart (bytes
    // behind the row's last are the next row's: a NaN among them would meet the
    // zeros past K).
    const int left = (a.kb - 16 * u - g + 3) >> 2;
    const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : ~0u >> (32 - 8 * left);
    const uint32_t sy = sa.get(wy, pick, keep);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t sx = sb[b].get(wx[b], pick, keep);
      acc[b] = mfma<0>(x[0][b], y[0], acc[b], sx, sy);
      acc[b] = mfma<1>(x[1][b], y[1], acc[b], sx, sy);
      acc[b] = mfma<2>(x[2][b], y[2], acc[b], sx, sy);
      acc[b] = mfma<3>(x[3][b], y[3], acc[b], sx, sy);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) part[wave][b][lane] = acc[b];
  __syncthreads();
  if (!mine) return;

  auto sum = [&](int b, float (&v)[4]) {
    v4f t = part[0][b][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) t += part[w][b][lane];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = t[q];
  };
  auto add = [&](const v2u &w, float (&v)[4]) {
    float t[4];
    unpack2<DT>(w[0], t);
    unpack2<DT>(w[1], t + 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] += t[q];
  };
  float z[4], up[4];
  sum(GATED ? 2 * wave : wave, z);
  if constexpr (GATED) sum(2 * wave + 1, up);
  if (bias) {
    add(bias0, z);
    if constexpr (GATED) add(bias1, up);
  }
  if (a.pre) {
    uint8_t *p = a.pre + (row * a.ldp + n) * 2;
    store4<DT>(p, z);
    if constexpr (GATED) store4<DT>(p + (size_t)a.half * 2, up);
  }
  with_act<GATED>(a.act, [&](auto act) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      z[q] = act_fwd<decltype(act)::value>(z[q]);
      if constexpr (GATED) z[q] *= up[q];
    }
  });
  if (a.res) add(res, z);
  store4<DT>(a.C + (row * a.ldc + n) * 2, z);
}

template <int DT, int W, int NB, bool GATED>
hipError_t launch_one(const MxGemm &g) {
  MxRowsArgs a{};
  a.A = static_cast<const uint8_t *>(g.A);
  a.SA = static_cast<const uint8_t *>(g.SA);
  a.B = static_cast<const uint8_t *>(g.B);
  a.SB = static_cast<const uint8_t *>(g.SB);
  a.C = static_cast<uint8_t *>(g.C);
  a.bias = static_cast<const uint8_t *>(g.bias);
  a.res = static_cast<const uint8_t *>(g.residual);
  a.pre = static_cast<uint8_t *>(g.preact);
  a.M = (int)g.M;
  a.N = (int)(GATED ? g.N / 2 : g.N);
  a.K = (int)g.K;
  a.lda = (int)g.lda;
  a.ldb = (int)g.ldb;
  a.ldc = (int)g.ldc;
  a.ldr = (int)g.ldr;
  a.ldp = (int)g.ldp;
  a.kb = (int)(g.K / 32);
  a.act = g.act;
  a.half = GATED ? a.N : 0;
  a.offsets = g.offsets;
  a.rows = g.rows;
  a.groups = (int)g.groups;
  a.src_rows = (int)g.src_rows;
  a.stride_b = g.stride_b;
  a.stride_sb = g.stride_sb;
  constexpr int kCols = 16 * (GATED ? NB / 2 : NB);
  a.tiles_n = (a.N + kCols - 1) / kCols;
  a.tiles_m = (int)((g.M + kTM - 1) / kTM);
  const int64_t tm = g.groups ? g.M / kTM + std::min(g.groups, g.M) : a.tiles_m;
  const int64_t wgs = tm * a.tiles_n;
  if (wgs > (int64_t)(UINT32_MAX / (64 * W))) return hipErrorInvalidConfiguration;
  void *args[] = {&a};
  const void *fn = g.groups ? reinterpret_cast<const void *>(&mx_rows_kernel<DT, W, NB, GATED, true>)
                            : reinterpret_cast<const void *>(&mx_rows_kernel<DT, W, NB, GATED, false>);
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(64 * W), args, 0, g.stream);
}

// NB blocks of 16 weight rows a wave and W waves: eight waves where each of four would
// take more than one unit of K, and two blocks for four waves and so many weight rows
// that one a wave fills the chip more than once.  (K above 1024 with that many goes to
// 64 x 64 tiles.)  us between launches of a graph, weights from memory; one row, NB 1:
//   N      K     W 4    W 8
//   4096   1024  2.86   2.95
//   4096   2048  3.46   3.55
//   4096   4096  4.72   4.63
//   4096   8192  7.66   6.86
// and W 4:
//   rows  groups  N      K     NB 1   NB 2
//   1     -       16384  1024  4.58   4.77
//   1     -       65536  1024  9.40   9.95
//   16    -       16384  1024  5.45   5.16
//   16    -       65536  1024  12.9   10.9
//   74    64      2048   256   10.4   9.07
//   74    64      2048   1024  15.1   13.9
//   600   64      4096   1024  42.3   37.1
template <int DT, int W>
hipError_t launch_waves(const MxGemm &g) {
  if (is_gated(g.act)) return launch_one<DT, W, 2, true>(g);
  if constexpr (W == 4)
    if (g.N * (g.groups ? std::min(g.groups, g.M) : 1) > 32 * g.cus) return launch_one<DT, W, 2, false>(g);
  return launch_one<DT, W, 1, false>(g);
}

template <int DT>
hipError_t launch_dt(const MxGemm &g) {
  return g.K > 2048 ? launch_waves<DT, 8>(g) : launch_waves<DT, 4>(g);
}

}  // namespace

hipError_t launch_mx_rows(const MxGemm &g) { return g.dtype == 1 ? launch_dt<1>(g) : launch_dt<0>(g); }

}  // namespace ffn
}  // namespace tgemm
