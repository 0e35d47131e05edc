// Products of few rows with an epilogue, dense or grouped, for gfx950: single
// tokens and small batches against weights stored K-contiguous (N x K).
//
// What bounds such a product is reading the weight once.  A workgroup takes
// 16 NB rows of the weight (columns of C) and up to 16 rows of A, and its W
// waves divide K: wave w takes units of 64 K elements (a 128-byte line of
// each row) w, w + W, ...  Weights and rows of A go from memory straight into
// the registers of v_mfma_f32_16x16x32 (lane l holds row l % 16, eight K
// elements from 8 (l / 16)), no LDS between: each weight byte is used by one
// wave only.  A batch of units is loaded while the one before is multiplied,
// and the bias and the residual before either.  The waves' sums meet in LDS,
// are added in wave order (the result does not depend on timing) and pass
// through the epilogue.
//
// Measured: one row of 4096 x 4096 with bias, silu and residual 8.0 us (33.5
// MB, 4.2 TB/s); 37 tokens of 6 of 64 experts, 53 of them hit, 2048 x 2048
// gated: 85 to 92 us for 445 MB (4.8 to 5.2 TB/s, a copy's rate), 2048 x 1024 42
// to 45 us for 222 MB.
//
// More rows would mean reading A's rows in every workgroup from the L2: with
// 48 rows, 8192 columns, K = 4096 a form of this kernel with up to 64 rows took
// 22 us where the 64 x 64 tiles take 14, with 32 rows 13.4 as they do.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tgemm_ffn_math.hpp"

namespace tgemm {
namespace ffn {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 v8bf;
typedef __attribute__((ext_vector_type(8))) _Float16 v8h;

constexpr uint32_t kOOB = 0x80000000u;  // an offset past every resource

struct RowsArgs {
  const uint8_t *A, *B;
  uint8_t *C;
  const uint8_t *bias, *res;
  uint8_t *pre;
  int M, N, K;  // N: output columns
  int lda, ldb, ldc, ldr, ldp;
  int act, half;
  int tiles_m, tiles_n;  // dense
  // grouped
  const int32_t *offsets, *rows;
  int groups, src_rows;
  int64_t stride_b, stride_bias;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void *p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, 0x00020000);
}

template <int DT>
__device__ __forceinline__ v4f mfma(const v4u &x, const v4u &y, const v4f &c) {
  if constexpr (DT == 1)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, x), __builtin_bit_cast(v8h, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ void store4(uint8_t *p, const float (&v)[4]) {
  *(v2u *)p = v2u{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}

constexpr int kTM = 16;

template <int DT, int W, int NB, bool GATED, bool GROUPED>
__global__ __launch_bounds__(64 * W) void rows_kernel(const RowsArgs a) {
  constexpr int kOutB = GATED ? NB / 2 : NB, kCols = 16 * kOutB;
  static_assert(kOutB <= W, "an output piece a thread");
  // Units of a batch; two batches are in registers, one on its way while the
  // other is multiplied.
  constexpr int kU = NB == 1 ? 4 : 2;
  __shared__ v4f part[W][NB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);

  // The tile: rows m0 .. of M (M counts from row `lo` on), columns n0 ...
  const uint8_t *A = a.A, *B = a.B, *bias = a.bias;
  int M = a.M, lo = 0, m0, n0;
  if constexpr (GROUPED) {
    const Found f = find_unit(a.offsets, a.groups, a.M, (int)blockIdx.x, kTM, a.tiles_n, lane);
    if (f.e < 0) return;
    M = f.hi - f.lo;
    lo = f.lo;
    const int tiles_m = (M + kTM - 1) / kTM;
    n0 = f.unit / tiles_m * kCols;
    m0 = (f.unit % tiles_m) * kTM;
    B += (size_t)f.e * (size_t)a.stride_b * 2;
    if (bias) bias += (size_t)f.e * (size_t)a.stride_bias * 2;
  } else {
    m0 = (int)blockIdx.x % a.tiles_m * kTM;
    n0 = (int)blockIdx.x / a.tiles_m * kCols;
  }

  // Lane l's row of every block and its 16-byte chunk of a unit's first half.
  const int r = lane & 15, g = lane >> 4;
  const int cols = min(a.N - n0, kCols);
  const auto rb = rsrc_of(B + (size_t)n0 * a.ldb * 2,
                          ((uint32_t)((GATED ? a.half : 0) + cols - 1) * (uint32_t)a.ldb + (uint32_t)a.K) * 2u);
  uint32_t boff[NB], aoff;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int c = (GATED ? b >> 1 : b) * 16 + r;
    const int row = c + (GATED && (b & 1) ? a.half : 0);
    boff[b] = c < cols ? (uint32_t)row * (uint32_t)a.ldb * 2u + 16u * (uint32_t)g : kOOB;
  }
  __amdgpu_buffer_rsrc_t ra;
  if (GROUPED && a.rows) {
    ra = rsrc_of(A, a.src_rows > 0 ? ((uint32_t)(a.src_rows - 1) * (uint32_t)a.lda + (uint32_t)a.K) * 2u : 0u);
    const int src = m0 + r < M ? a.rows[lo + m0 + r] : -1;
    aoff = src >= 0 && src < a.src_rows ? (uint32_t)src * (uint32_t)a.lda * 2u + 16u * (uint32_t)g : kOOB;
  } else {
    ra = rsrc_of(A + (size_t)(lo + m0) * a.lda * 2,
                 ((uint32_t)(min(M - m0, kTM) - 1) * (uint32_t)a.lda + (uint32_t)a.K) * 2u);
    aoff = m0 + r < M ? (uint32_t)r * (uint32_t)a.lda * 2u + 16u * (uint32_t)g : kOOB;
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
  const int units = (a.K + 63) >> 6;
  struct Batch {
    v4u x[kU][2][NB], y[kU][2];
  };
  // (K % 8 == 0: a lane's chunk is all inside K or all outside, where both
  // operands read zeros; a unit past the last is all outside.  The weights'
  // loads first: A's wait for its row's index.)
  auto load = [&](Batch &f, int u0) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int u = u0 + W * i;
        const bool in = 64 * u + 32 * s + 8 * g < a.K;
#pragma unroll
        for (int b = 0; b < NB; ++b)
          f.x[i][s][b] = __builtin_amdgcn_raw_buffer_load_b128(rb, in ? boff[b] : kOOB, (uint32_t)u * 128u + 64u * (uint32_t)s, 0);
      }
#pragma unroll
    for (int i = 0; i < kU; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int u = u0 + W * i;
        const bool in = 64 * u + 32 * s + 8 * g < a.K;
        f.y[i][s] = __builtin_amdgcn_raw_buffer_load_b128(ra, in ? aoff : kOOB, (uint32_t)u * 128u + 64u * (uint32_t)s, 0);
      }
    __builtin_amdgcn_sched_barrier(0);  // (all on their way before the next products)
  };
  auto multiply = [&](const Batch &f) {
#pragma unroll
    for (int i = 0; i < kU; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = mfma<DT>(f.x[i][s][b], f.y[i][s], acc[b]);
    __builtin_amdgcn_sched_barrier(0);
  };
  Batch f0, f1;
  constexpr int kStep = W * kU;
  load(f0, wave);
  for (int u0 = wave; u0 < units; u0 += 2 * kStep) {
    load(f1, u0 + kStep);
    multiply(f0);
    if (u0 + kStep >= units) break;
    load(f0, u0 + 2 * kStep);
    multiply(f1);
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
hipError_t launch_one(const Gemm &g) {
  RowsArgs a{};
  a.A = static_cast<const uint8_t *>(g.A);
  a.B = static_cast<const uint8_t *>(g.B);
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
  a.act = g.act;
  a.half = GATED ? a.N : 0;
  a.offsets = g.offsets;
  a.rows = g.rows;
  a.groups = (int)g.groups;
  a.src_rows = (int)g.src_rows;
  a.stride_b = g.stride_b;
  a.stride_bias = g.stride_bias;
  constexpr int kCols = 16 * (GATED ? NB / 2 : NB);
  a.tiles_n = (a.N + kCols - 1) / kCols;
  a.tiles_m = (int)((g.M + kTM - 1) / kTM);
  const int64_t tm = g.groups ? g.M / kTM + std::min(g.groups, g.M) : a.tiles_m;
  const int64_t wgs = tm * a.tiles_n;
  if (wgs > (int64_t)(UINT32_MAX / (64 * W))) return hipErrorInvalidConfiguration;
  void *args[] = {&a};
  const void *fn = g.groups ? reinterpret_cast<const void *>(&rows_kernel<DT, W, NB, GATED, true>)
                            : reinterpret_cast<const void *>(&rows_kernel<DT, W, NB, GATED, false>);
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(64 * W), args, 0, g.stream);
}

// Weight rows that are read, if every row of A hits another group.
int64_t weight_rows(const Gemm &g) { return g.N * (g.groups ? std::min(g.groups, g.M) : 1); }

template <int DT, int W>
hipError_t launch_waves(const Gemm &g) {
  if (is_gated(g.act)) return launch_one<DT, W, 2, true>(g);
  // One block of 16 columns a workgroup while that leaves no more than two
  // workgroups a CU (2 of 16 experts of 2048 x 1536: 5.3 us, with two blocks
  // 5.9; 16 of 64 of 2048 x 1024: 17.2 and 13.5).
  return weight_rows(g) <= 32 * g.cus ? launch_one<DT, W, 1, false>(g) : launch_one<DT, W, 2, false>(g);
}

template <int DT>
hipError_t launch_dt(const Gemm &g) {
  // Eight waves a workgroup over a deep K of many weight rows, else four and
  // more workgroups a CU.  One row, us with 4 and 8 waves: 32768 x 4096 64.3 and
  // 56.3, 32768 x 2048 29.6 and 27.4, 32768 x 1024 15.4 and 15.9, 8192 x 4096
  // 16.0 and 17.0; 64 gated experts of 2048 x 2048 114 and 100.
  return g.K >= 2048 && weight_rows(g) > 32 * g.cus ? launch_waves<DT, 8>(g) : launch_waves<DT, 4>(g);
}

}  // namespace

hipError_t launch_rows(const Gemm &g) { return g.dtype == 1 ? launch_dt<1>(g) : launch_dt<0>(g); }

}  // namespace ffn
}  // namespace tgemm
