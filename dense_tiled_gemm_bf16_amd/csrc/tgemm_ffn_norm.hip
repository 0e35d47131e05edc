// Layer norm over rows and its gradients, for gfx950.
//
// y = (x - mean) rstd w + b.  With g = dy w and h = (x - mean) rstd:
// dx = rstd (g - mean(g) - h mean(g h)) + residual, dw = sum over rows of
// dy h, db = sum over rows of dy.  About 8 operations a value forward and 20
// backward for 4 to 10 bytes moved: memory bounds both.
//
// Statistics and sums are binary32.  The variance is summed over differences
// from the mean, from registers or a second read of the row (which the caches
// hold), so that a row far from zero keeps its digits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tgemm_ffn_math.hpp"

namespace tgemm {
namespace ffn {
namespace {

// Eight consecutive values of type DT (0 bf16, 1 fp16, 2 fp32): as stored, and
// as binary32.
template <int DT>
struct Eight {
  v4u w[DT == 2 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t *p) {
    w[0] = *(const v4u *)p;
    if constexpr (DT == 2) w[1] = *(const v4u *)(p + 16);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (DT == 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const v4f f = __builtin_bit_cast(v4f, w[i]);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[4 * i + q] = f[q];
      }
    } else {
      unpack8<DT>(w[0], v);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    if constexpr (DT == 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, v[i]);
    } else {
      w[0] = pack8<DT>(v);
    }
  }
  __device__ __forceinline__ void store(uint8_t *p) const {
    *(v4u *)p = w[0];
    if constexpr (DT == 2) *(v4u *)(p + 16) = w[1];
  }
};
constexpr int bytes_of(int dt) { return dt == 2 ? 4 : 2; }

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

struct NormArgs {
  const uint8_t *x, *w, *b;
  uint8_t *y;
  float *mean, *rstd;
  int M, N;
  int64_t ldx, ldy;  // bytes
  float eps, inv_n;
};

// One row a workgroup of T threads, P pieces of 8 values a thread in
// registers; P = 0: any length, three reads of the row.
template <int DT, int WDT, int T, int P>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_kernel(const NormArgs a) {
  constexpr int kB = bytes_of(DT), kW = bytes_of(WDT), kWaves = T / 64, kRows = T < 256 ? 256 / T : 1;
  __shared__ float part[2][kWaves];
  const int t = (int)threadIdx.x % T;
  const int row = (int)blockIdx.x * kRows + (int)threadIdx.x / T;
  if (kRows > 1 && row >= a.M) return;  // (a whole wave, where no barrier follows)
  auto total = [&](float v, int which) {
    v = wave_sum(v);
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) part[which][threadIdx.x >> 6] = v;
      __syncthreads();
      v = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) v += part[which][i];
    }
    return v;
  };
  const uint8_t *x = a.x + (size_t)row * a.ldx;
  uint8_t *y = a.y + (size_t)row * a.ldy;
  auto put = [&](int n, const float (&v)[8], float mu, float rs) {
    float w[8], b[8], o[8];
    Eight<WDT> e;
    if (a.w) {
      e.load(a.w + (size_t)n * kW);
      e.get(w);
    }
    if (a.b) {
      e.load(a.b + (size_t)n * kW);
      e.get(b);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      o[q] = (v[q] - mu) * rs;
      if (a.w) o[q] *= w[q];
      if (a.b) o[q] += b[q];
    }
    Eight<DT> r;
    r.set(o);
    r.store(y + (size_t)n * kB);
  };
  float mu, rs;
  if constexpr (P > 0) {
    float v[P][8], s = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int n = (p * T + t) * 8;
      Eight<DT> e{};
      if (n < a.N) e.load(x + (size_t)n * kB);
      e.get(v[p]);
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int q = 0; q < 8; ++q) s += v[p][q];
    mu = total(s, 0) * a.inv_n;
    float d = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
      if ((p * T + t) * 8 < a.N) {
#pragma unroll
        for (int q = 0; q < 8; ++q) d += (v[p][q] - mu) * (v[p][q] - mu);
      }
    rs = 1.0f / sqrtf(total(d, 1) * a.inv_n + a.eps);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int n = (p * T + t) * 8;
      if (n < a.N) put(n, v[p], mu, rs);
    }
  } else {
    float v[8], s = 0.0f, d = 0.0f;
    Eight<DT> e;
    for (int n = t * 8; n < a.N; n += T * 8) {
      e.load(x + (size_t)n * kB);
      e.get(v);
#pragma unroll
      for (int q = 0; q < 8; ++q) s += v[q];
    }
    mu = total(s, 0) * a.inv_n;
    for (int n = t * 8; n < a.N; n += T * 8) {
      e.load(x + (size_t)n * kB);
      e.get(v);
#pragma unroll
      for (int q = 0; q < 8; ++q) d += (v[q] - mu) * (v[q] - mu);
    }
    rs = 1.0f / sqrtf(total(d, 1) * a.inv_n + a.eps);
    for (int n = t * 8; n < a.N; n += T * 8) {
      e.load(x + (size_t)n * kB);
      e.get(v);
      put(n, v, mu, rs);
    }
  }
  if (t == 0) {
    if (a.mean) a.mean[row] = mu;
    if (a.rstd) a.rstd[row] = rs;
  }
}

template <int DT, int WDT>
hipError_t launch_norm_types(const Norm &g) {
  const int b = bytes_of(DT);
  NormArgs a{static_cast<const uint8_t *>(g.x), static_cast<const uint8_t *>(g.weight),
             static_cast<const uint8_t *>(g.bias), static_cast<uint8_t *>(g.y), g.mean, g.rstd, (int)g.M, (int)g.N,
             g.ldx * b, g.ldy * b, g.eps, (float)(1.0 / (double)g.N)};
  void *args[] = {&a};
  const void *fn;
  int threads = 256, rows = 1;
  if (g.N <= 512) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 64, 1>);
    rows = 4;
  } else if (g.N <= 1024) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 64, 2>);
    rows = 4;
  } else if (g.N <= 2048) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 256, 1>);
  } else if (g.N <= 4096) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 256, 2>);
  } else if (g.N <= 8192) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 256, 4>);
  } else if (g.N <= 16384) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 512, 4>);
    threads = 512;
  } else {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 1024, 0>);
    threads = 1024;
  }
  const int64_t wgs = (g.M + rows - 1) / rows;
  if (wgs > (int64_t)(UINT32_MAX / threads)) return hipErrorInvalidConfiguration;
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(threads), args, 0, g.stream);
}

// ---------------------------------------------------------------------------
// Gradients.
//
// Rows of any length in two steps: norm_rows_kernel, a row a workgroup, leaves
// mean(g) and mean(g h) in the workspace; norm_columns_kernel takes kRowsWg
// rows and 256 columns (as the epilogue's gradient), writes dx and adds up its
// columns of dy h and dy.  norm_sum_kernel adds those of all row blocks.
// ---------------------------------------------------------------------------
constexpr int kRowsWg = 64;

struct NormGradArgs {
  const uint8_t *dy, *x, *w, *res;
  const float *mean, *rstd;
  uint8_t *dx, *dw, *db;
  float *rowsums, *colsums;  // M x 2; blocks x 2 x N
  int M, N;
  int64_t ldd, ldx, ldr, ldo;  // bytes
  float inv_n;
  int tiles_n, blocks;
};

template <int DT, int WDT>
__global__ __launch_bounds__(256) void norm_rows_kernel(const NormGradArgs a) {
  constexpr int kB = bytes_of(DT), kW = bytes_of(WDT);
  __shared__ float part[2][4];
  const int row = (int)blockIdx.x;
  const float mu = a.mean[row], rs = a.rstd[row];
  float s0 = 0.0f, s1 = 0.0f;
  for (int n = (int)threadIdx.x * 8; n < a.N; n += 2048) {
    float d[8], x[8], w[8];
    Eight<DT> e;
    e.load(a.dy + (size_t)row * a.ldd + (size_t)n * kB);
    e.get(d);
    e.load(a.x + (size_t)row * a.ldx + (size_t)n * kB);
    e.get(x);
    if (a.w) {
      Eight<WDT> f;
      f.load(a.w + (size_t)n * kW);
      f.get(w);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float g = a.w ? d[q] * w[q] : d[q];
      s0 += g;
      s1 += g * ((x[q] - mu) * rs);
    }
  }
  s0 = wave_sum(s0);
  s1 = wave_sum(s1);
  if ((threadIdx.x & 63) == 0) {
    part[0][threadIdx.x >> 6] = s0;
    part[1][threadIdx.x >> 6] = s1;
  }
  __syncthreads();
  if (threadIdx.x < 2)
    a.rowsums[2 * (size_t)row + threadIdx.x] =
        ((part[threadIdx.x][0] + part[threadIdx.x][1]) + (part[threadIdx.x][2] + part[threadIdx.x][3])) * a.inv_n;
}

template <int DT, int WDT>
__global__ __launch_bounds__(256) void norm_columns_kernel(const NormGradArgs a) {
  constexpr int kB = bytes_of(DT), kW = bytes_of(WDT);
  __shared__ float sums[2][8][256];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int block = (int)blockIdx.x / a.tiles_n, ct = (int)blockIdx.x % a.tiles_n;
  const int r0 = block * kRowsWg, r1 = min(r0 + kRowsWg, a.M);
  const int n = ct * 256 + tx * 8;
  float sw[8] = {}, sb[8] = {};
  if (n < a.N) {
    float w[8];
    if (a.w) {
      Eight<WDT> f;
      f.load(a.w + (size_t)n * kW);
      f.get(w);
    }
#pragma unroll 2
    for (int r = r0 + ty; r < r1; r += 8) {
      float d[8], x[8], o[8];
      Eight<DT> e;
      e.load(a.dy + (size_t)r * a.ldd + (size_t)n * kB);
      e.get(d);
      e.load(a.x + (size_t)r * a.ldx + (size_t)n * kB);
      e.get(x);
      const float mu = a.mean[r], rs = a.rstd[r], c0 = a.rowsums[2 * (size_t)r], c1 = a.rowsums[2 * (size_t)r + 1];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float h = (x[q] - mu) * rs;
        sw[q] += d[q] * h;
        sb[q] += d[q];
        o[q] = rs * ((a.w ? d[q] * w[q] : d[q]) - c0 - h * c1);
      }
      if (a.res) {
        e.load(a.res + (size_t)r * a.ldr + (size_t)n * kB);
        e.get(x);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] += x[q];
      }
      e.set(o);
      e.store(a.dx + (size_t)r * a.ldo + (size_t)n * kB);
    }
  }
  if (!a.dw && !a.db) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    sums[0][ty][tx * 8 + q] = sw[q];
    sums[1][ty][tx * 8 + q] = sb[q];
  }
  __syncthreads();
  const int c = ct * 256 + (int)threadIdx.x;
  if (c >= a.N) return;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float v = 0.0f;
#pragma unroll
    for (int y = 0; y < 8; ++y) v += sums[p][y][threadIdx.x];
    a.colsums[((size_t)block * 2 + p) * a.N + c] = v;
  }
}

// 64 columns of both sums: sixteen waves take the blocks in turn.
template <int WDT>
__global__ __launch_bounds__(1024) void norm_sum_kernel(const NormGradArgs a) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int p = (int)blockIdx.y, n = (int)blockIdx.x * 64 + lane;
  uint8_t *out = p ? a.db : a.dw;
  if (!out) return;
  float v = 0.0f;
  if (n < a.N) {
#pragma unroll 4
    for (int b = wave; b < a.blocks; b += 16) v += a.colsums[((size_t)b * 2 + p) * a.N + n];
  }
  sums[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && n < a.N) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sums[i][lane];
    if constexpr (WDT == 2)
      *(float *)(out + (size_t)n * 4) = t;
    else
      *(uint16_t *)(out + (size_t)n * 2) = (uint16_t)(pack2<WDT>(t, 0.0f) & 0xffffu);
  }
}

template <int DT, int WDT>
hipError_t launch_norm_grad_types(const NormGrad &g) {
  const int b = bytes_of(DT);
  NormGradArgs a{};
  a.dy = static_cast<const uint8_t *>(g.dy);
  a.x = static_cast<const uint8_t *>(g.x);
  a.w = static_cast<const uint8_t *>(g.weight);
  a.res = static_cast<const uint8_t *>(g.residual);
  a.mean = g.mean;
  a.rstd = g.rstd;
  a.dx = static_cast<uint8_t *>(g.dx);
  a.dw = static_cast<uint8_t *>(g.dweight);
  a.db = static_cast<uint8_t *>(g.dbias);
  a.M = (int)g.M;
  a.N = (int)g.N;
  a.ldd = g.ldd * b;
  a.ldx = g.ldx * b;
  a.ldr = g.ldr * b;
  a.ldo = g.ldo * b;
  a.inv_n = (float)(1.0 / (double)g.N);
  a.tiles_n = (a.N + 255) / 256;
  a.blocks = (int)((g.M + kRowsWg - 1) / kRowsWg);
  a.rowsums = g.ws;
  a.colsums = g.ws + (g.M + 1) / 2 * 4;
  void *args[] = {&a};
  hipError_t e = hipSuccess;
  if (g.M > 0) {
    const int64_t wgs = (int64_t)a.blocks * a.tiles_n;
    if (g.M > (int64_t)(UINT32_MAX / 256) || wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
    e = hipLaunchKernel(reinterpret_cast<const void *>(&norm_rows_kernel<DT, WDT>), dim3((unsigned)g.M), dim3(256), args, 0,
                        g.stream);
    if (e == hipSuccess)
      e = hipLaunchKernel(reinterpret_cast<const void *>(&norm_columns_kernel<DT, WDT>), dim3((unsigned)wgs), dim3(256),
                          args, 0, g.stream);
  }
  if (e == hipSuccess && (g.dweight || g.dbias))
    e = hipLaunchKernel(reinterpret_cast<const void *>(&norm_sum_kernel<WDT>), dim3((unsigned)((a.N + 63) / 64), 2),
                        dim3(1024), args, 0, g.stream);
  return e;
}

}  // namespace

uint64_t norm_grad_ws_floats(int64_t M, int64_t N) {
  return (uint64_t)((M + 1) / 2 * 4) + (uint64_t)((M + kRowsWg - 1) / kRowsWg) * 2u * (uint64_t)N;
}

hipError_t launch_norm(const Norm &g) {
  if (g.dtype == 2) return launch_norm_types<2, 2>(g);
  if (g.dtype == 1) return g.wdtype == 2 ? launch_norm_types<1, 2>(g) : launch_norm_types<1, 1>(g);
  return g.wdtype == 2 ? launch_norm_types<0, 2>(g) : launch_norm_types<0, 0>(g);
}

hipError_t launch_norm_grad(const NormGrad &g) {
  if (g.dtype == 2) return launch_norm_grad_types<2, 2>(g);
  if (g.dtype == 1) return g.wdtype == 2 ? launch_norm_grad_types<1, 2>(g) : launch_norm_grad_types<1, 1>(g);
  return g.wdtype == 2 ? launch_norm_grad_types<0, 2>(g) : launch_norm_grad_types<0, 0>(g);
}

}  // namespace ffn
}  // namespace tgemm
