// Layer norm over rows and its gradients, for gfx950.
//
// y = (x - mean) rstd w + b.  With g = dy w and h = (x - mean) rstd:
// dx = rstd (g - mean(g) - h mean(g h)) + residual, dw = sum over rows of
// dy h, db = sum over rows of dy.  About 8 operations a value forward and 20
// backward for 4 to 10 bytes moved: memory bounds both.
//
// Statistics and sums are binary32.  The variance is summed over differences
// from the mean, from registers or a second read of the row (which the caches
// hold), so that a row far from zero keeps its digits.  A thread of a row kernel
// adds at most 32 values one after the other; where rows may be longer its sums
// are compensated (LongSum).
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

// Sum over the wave, in every lane: rows of 16 lanes by shifts, then the rows'
// totals handed on, the wave's in lane 63.  (By lane exchanges through LDS, six
// one after the other, a row's two sums took 0.4 us.)
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](auto ctrl) {
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  add(Int<0x111>());
  add(Int<0x112>());
  add(Int<0x114>());
  add(Int<0x118>());
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xa, 0xf, false));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xc, 0xf, false));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// A sum of any length: pieces of eight values, added up in pairs, sixteen pieces one
// after the other, and those sums compensated (Kahan's: `lost` is what the last
// addition rounded away).  One running sum over a row of 2^31 values, 2^21 additions
// a thread, lost 0.8% of the mean: once it is large every addition rounds the same
// way.  (Gradients of 8 x 65536 bf16: one running sum 18.2 us, this way 18.7, every
// piece compensated 19.9; 2048 x 20000 forward 42.5 and, this way, 43.3.)
constexpr int kLongTurns = 16;
__device__ __forceinline__ float sum8(const float (&v)[8]) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}
struct LongSum {
  float s = 0.0f, lost = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float y = v - lost, t = s + y;
    lost = (t - s) - y;
    if (!(lost == lost)) lost = 0.0f;  // (an infinity stays one)
    s = t;
  }
};

struct NormArgs {
  const uint8_t *x, *w, *b;
  uint8_t *y;
  float *mean, *rstd;
  int M, N;
  int64_t ldx, ldy;  // bytes
  float eps, inv_n;
};

// One row a workgroup of T threads (or a wave, T = 64, which needs no barrier),
// P pieces of 8 values a thread in registers; P = 0: any length, three reads of
// the row, the last two from the caches.  Reading x and writing y once bound it:
// 8192 x 4096 bf16 29 us from memory (134 MB, 4.6 TB/s), 4093 x 5000 fp16 19,
// 8192 x 4096 binary32 48 (268 MB, 5.6 TB/s, one call after another); 8 x 4096 2.7
// between launches of a graph, the latency of a load and two sums across the row.
// T x P, us for 2^25 bf16 values:
//   N = 512     64 x 1   23.5   256 x 1  50.8
//   N = 1024    64 x 2   22.3   256 x 1  32.5
//   N = 2048    256 x 1  23.2   64 x 4   23.2   256 x 2  23.5
//   N = 4096    256 x 2  22.0   512 x 1  23.6
//   N = 5000    256 x 3  23.1   512 x 2  24.6   256 x 4  23.1
//   N = 6144    256 x 3  23.0   512 x 2  22.8
//   N = 8192    512 x 2  22.4   256 x 4  23.5   512 x 4  22.3
//   N = 16384   512 x 4  24.2   1024 x 2 24.5   any length 29.4
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
    float v[8];
    LongSum s, d;
    Eight<DT> e;
    for (uint32_t n = t * 8; n < (uint32_t)a.N;) {
      float sum = 0.0f;
      const uint32_t end = min(n + kLongTurns * T * 8, (uint32_t)a.N);  // (steps past the end may pass 2^31)
      for (; n < end; n += T * 8) {
        e.load(x + (size_t)n * kB);
        e.get(v);
        sum += sum8(v);
      }
      s.add(sum);
    }
    mu = total(s.s, 0) * a.inv_n;
    for (uint32_t n = t * 8; n < (uint32_t)a.N;) {
      float sum = 0.0f;
      const uint32_t end = min(n + kLongTurns * T * 8, (uint32_t)a.N);
      for (; n < end; n += T * 8) {
        e.load(x + (size_t)n * kB);
        e.get(v);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = (v[q] - mu) * (v[q] - mu);
        sum += sum8(v);
      }
      d.add(sum);
    }
    rs = 1.0f / sqrtf(total(d.s, 1) * a.inv_n + a.eps);
    for (uint32_t n = t * 8; n < (uint32_t)a.N; n += T * 8) {
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
  } else if (g.N <= 6144) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 256, 3>);
  } else if (g.N <= 8192) {
    fn = reinterpret_cast<const void *>(&norm_kernel<DT, WDT, 512, 2>);
    threads = 512;
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
// Rows of up to 8192 values in one pass (norm_grad_kernel): T threads hold a row
// of x, dy and the residual in registers between its two sums and dx, and add
// up dy h and dy of their own columns over all the rows that their workgroup
// takes.  The workgroups, one or two a CU, take sets of rows in turn; the sums of
// the row groups of a workgroup meet in LDS, those of the workgroups in the
// workspace, where norm_sum_kernel adds them in order (atomics would add them in
// another each time).  A thread's sums go there every kSumTurns turns, so that no
// running sum gets long: in one over 32768 turns (134 million rows of 8 values)
// dweight lost 3e-4 of its sum of magnitudes.  The next rows are loaded before the
// sums of the present ones are waited for.  Four arrays of one read or write bound
// it: 8192 x 4096 bf16 with the residual 45 us behind the forward pass (268 MB, 6.0
// TB/s: part of x is still in the caches), its column sums 4.7; binary32 without a
// residual 80 us with them (403 MB, 5.0 TB/s), though its loads do not run ahead.
// T x P, us for 2^25 bf16 values without a residual, the sums with them, for one
// and two workgroups a CU, before the sums went to the workspace in runs (the
// chosen ones since then, in turn: 39.6, 37.8, 39.0, 38.6, 41.2):
//   N = 512    64 x 1   44.2 40.2   256 x 1  148  94.7
//   N = 1024   64 x 2   40.7 45.7   256 x 1  84.2 58.4
//   N = 2048   256 x 1  50.8 42.4   512 x 1  83.9 56.7   256 x 2  57.9 61.3
//   N = 4096   256 x 2  46.3 50.7   512 x 1  51.9 45.3
//   N = 8192   512 x 2  49.6 55.0
//
// Longer rows in two steps: norm_rows_kernel, a row a workgroup, leaves
// mean(g) and mean(g h) in the workspace; norm_columns_kernel takes kRowsWg
// rows and 256 columns (as the epilogue's gradient), writes dx and adds up its
// columns.  (8192 x 4096 bf16 with the residual this way 23 + 57 us, in one pass
// 45; but 2048 x 12288 48 and 69, whose one pass would spill.)
// ---------------------------------------------------------------------------
constexpr int kGradWgs = 256;
constexpr int kRowsWg = 64;
constexpr int kSumTurns = 512;

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

template <int DT, int WDT, int T, int P>
__global__ __launch_bounds__(512) void norm_grad_kernel(const NormGradArgs a) {
  constexpr int kB = bytes_of(DT), kW = bytes_of(WDT), kGroups = 512 / T, kWaves = T / 64;
  constexpr bool kAhead = DT != 2;  // (registers for two sets of rows)
  __shared__ float part[2][kGroups][2][kWaves];
  __shared__ float sums[2 * P * 8 * T];
  const int t = (int)threadIdx.x % T, group = (int)threadIdx.x / T;
  struct Row {
    Eight<DT> x[P], d[P], r[P];
    float mu, rs;
  };
  auto load = [&](Row &v, int row) {
    const bool in = row < a.M;
    v.mu = in ? a.mean[row] : 0.0f;
    v.rs = in ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int n = (p * T + t) * 8;
      v.x[p] = v.d[p] = v.r[p] = Eight<DT>{};
      if (in && n < a.N) {
        v.x[p].load(a.x + (size_t)row * a.ldx + (size_t)n * kB);
        v.d[p].load(a.dy + (size_t)row * a.ldd + (size_t)n * kB);
        if (a.res) v.r[p].load(a.res + (size_t)row * a.ldr + (size_t)n * kB);
      }
    }
  };
  Eight<WDT> w[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int n = (p * T + t) * 8;
    w[p] = Eight<WDT>{};
    if (a.w && n < a.N) w[p].load(a.w + (size_t)n * kW);
  }
  float sw[P][8] = {}, sb[P][8] = {};
  const int step = a.blocks * kGroups, first = (int)blockIdx.x * kGroups;
  Row cur;
  load(cur, first + group);
  int which = 0;
  bool again = false;
  // (row0 is the workgroup's: every thread takes as many turns.)
  for (int row0 = first; row0 < a.M; again = true) {
    const int end = (int)min((uint32_t)row0 + (uint32_t)kSumTurns * (uint32_t)step, (uint32_t)a.M);
    for (; row0 < end; row0 += step, which ^= 1) {
      const int row = row0 + group;
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float d[8], x[8], wv[8];
        cur.x[p].get(x);
        cur.d[p].get(d);
        w[p].get(wv);
        const bool in = (p * T + t) * 8 < a.N;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float h = in ? (x[q] - cur.mu) * cur.rs : 0.0f, g = a.w ? d[q] * wv[q] : d[q];
          s0 += g;
          s1 += g * h;
          sw[p][q] += d[q] * h;
          sb[p][q] += d[q];
        }
      }
      Row next;
      if constexpr (kAhead) load(next, row + step);
      s0 = wave_sum(s0);
      s1 = wave_sum(s1);
      if constexpr (kWaves > 1) {
        if ((threadIdx.x & 63) == 0) {
          part[which][group][0][t >> 6] = s0;
          part[which][group][1][t >> 6] = s1;
        }
        __syncthreads();  // (the buffers alternate: the next turn's writes need no barrier of their own)
        s0 = s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
          s0 += part[which][group][0][i];
          s1 += part[which][group][1][i];
        }
      }
      const float c0 = s0 * a.inv_n, c1 = s1 * a.inv_n;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int n = (p * T + t) * 8;
        float d[8], x[8], wv[8], r[8], o[8];
        cur.d[p].get(d);
        cur.x[p].get(x);
        w[p].get(wv);
        cur.r[p].get(r);
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = cur.rs * ((a.w ? d[q] * wv[q] : d[q]) - c0 - (x[q] - cur.mu) * cur.rs * c1) + r[q];
        if (row < a.M && n < a.N) {
          Eight<DT> e;
          e.set(o);
          e.store(a.dx + (size_t)row * a.ldo + (size_t)n * kB);
        }
      }
      if constexpr (kAhead)
        cur = next;
      else
        load(cur, row + step);
    }
    if (!a.dw && !a.db) continue;
    // The row groups' sums one after the other, into the first's registers.
#pragma unroll 1
    for (int g = 1; g < kGroups; ++g) {
      __syncthreads();
      if (group == g) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            sums[(p * 8 + q) * T + t] = sw[p][q];
            sums[((P + p) * 8 + q) * T + t] = sb[p][q];
          }
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            sw[p][q] += sums[(p * 8 + q) * T + t];
            sb[p][q] += sums[((P + p) * 8 + q) * T + t];
          }
      }
    }
    // Into the workspace, or (from the second time on) to what is there.
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int n = (p * T + t) * 8;
      if (group == 0 && n < a.N) {
        float *c = a.colsums + (size_t)blockIdx.x * 2 * a.N + n;
        auto put = [&](float *at, const float *v) {
          v4f s = {v[0], v[1], v[2], v[3]};
          if (again) s += *(const v4f *)at;
          *(v4f *)at = s;
        };
        put(c, sw[p]);
        put(c + 4, sw[p] + 4);
        put(c + a.N, sb[p]);
        put(c + a.N + 4, sb[p] + 4);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sw[p][q] = sb[p][q] = 0.0f;
    }
  }
}

template <int DT, int WDT>
__global__ __launch_bounds__(256) void norm_rows_kernel(const NormGradArgs a) {
  constexpr int kB = bytes_of(DT), kW = bytes_of(WDT);
  __shared__ float part[2][4];
  const int row = (int)blockIdx.x;
  const float mu = a.mean[row], rs = a.rstd[row];
  LongSum g0, g1;
  for (int n = (int)threadIdx.x * 8; n < a.N;) {
    float s0 = 0.0f, s1 = 0.0f;
    const int end = min(n + kLongTurns * 2048, a.N);  // (the workspace's limit keeps N below 2^30)
    for (; n < end; n += 2048) {
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
        if (a.w) d[q] *= w[q];
        x[q] = d[q] * ((x[q] - mu) * rs);
      }
      s0 += sum8(d);
      s1 += sum8(x);
    }
    g0.add(s0);
    g1.add(s1);
  }
  const float s0 = wave_sum(g0.s), s1 = wave_sum(g1.s);
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

// 64 columns of both sums at a time: sixteen waves take the blocks in turn.  A dispatch
// holds kSumWgs workgroups of 1024 threads; rows of more than 2^28 values take several turns.
constexpr int kSumWgs = (1 << 22) - 1;
template <int WDT>
__global__ __launch_bounds__(1024) void norm_sum_kernel(const NormGradArgs a) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int p = (int)blockIdx.y;
  uint8_t *out = p ? a.db : a.dw;
  if (!out) return;
  for (int64_t n0 = (int64_t)blockIdx.x * 64; n0 < a.N; n0 += (int64_t)gridDim.x * 64) {
    const int64_t n = n0 + lane;
    float v = 0.0f;
    if (n < a.N) {
      for (int b = wave; b < a.blocks;) {  // (32 of them at a time, as above)
        const int end = min(b + 512, a.blocks);
        float part = 0.0f;
#pragma unroll 4
        for (; b < end; b += 16) part += a.colsums[((size_t)b * 2 + p) * a.N + n];
        v += part;
      }
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
    __syncthreads();
  }
}

constexpr int64_t kFusedMost = 8192;  // values of a row
// Blocks of column sums in the workspace.
int grad_blocks(int64_t M, int64_t N) {
  if (N > kFusedMost) return (int)((M + kRowsWg - 1) / kRowsWg);
  const int groups = N <= 1024 ? 8 : N <= 4096 ? 2 : 1;  // rows of a workgroup at a time
  const bool two = N <= 512 || (N > 1024 && N <= 2048);  // (one piece a thread: registers for two a CU)
  return (int)std::min<int64_t>((M + groups - 1) / groups, two ? 2 * kGradWgs : kGradWgs);
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
  a.blocks = grad_blocks(g.M, g.N);
  a.rowsums = g.ws;
  a.colsums = g.ws + (g.N > kFusedMost ? (g.M + 1) / 2 * 4 : 0);
  void *args[] = {&a};
  hipError_t e = hipSuccess;
  if (g.M > 0 && g.N <= kFusedMost) {
    const void *fn = g.N <= 512    ? reinterpret_cast<const void *>(&norm_grad_kernel<DT, WDT, 64, 1>)
                     : g.N <= 1024 ? reinterpret_cast<const void *>(&norm_grad_kernel<DT, WDT, 64, 2>)
                     : g.N <= 2048 ? reinterpret_cast<const void *>(&norm_grad_kernel<DT, WDT, 256, 1>)
                     : g.N <= 4096 ? reinterpret_cast<const void *>(&norm_grad_kernel<DT, WDT, 256, 2>)
                                   : reinterpret_cast<const void *>(&norm_grad_kernel<DT, WDT, 512, 2>);
    e = hipLaunchKernel(fn, dim3((unsigned)a.blocks), dim3(512), args, 0, g.stream);
  } else if (g.M > 0) {
    const int64_t wgs = (int64_t)a.blocks * a.tiles_n;
    if (g.M > (int64_t)(UINT32_MAX / 256) || wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
    e = hipLaunchKernel(reinterpret_cast<const void *>(&norm_rows_kernel<DT, WDT>), dim3((unsigned)g.M), dim3(256), args, 0,
                        g.stream);
    if (e == hipSuccess)
      e = hipLaunchKernel(reinterpret_cast<const void *>(&norm_columns_kernel<DT, WDT>), dim3((unsigned)wgs), dim3(256),
                          args, 0, g.stream);
  }
  if (e == hipSuccess && (g.dweight || g.dbias))
    e = hipLaunchKernel(reinterpret_cast<const void *>(&norm_sum_kernel<WDT>),
                        dim3((unsigned)std::min((a.N + 63) / 64, kSumWgs), 2), dim3(1024), args, 0, g.stream);
  return e;
}

}  // namespace

uint64_t norm_grad_ws_floats(int64_t M, int64_t N) {
  return (N > kFusedMost ? (uint64_t)((M + 1) / 2 * 4) : 0u) + (uint64_t)grad_blocks(M, N) * 2u * (uint64_t)N;
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
