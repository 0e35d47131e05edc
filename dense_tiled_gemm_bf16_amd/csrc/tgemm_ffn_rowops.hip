// The feed-forward layers' passes over rows, for gfx950: the backward pass of
// the epilogue with its column sums, and the moves of rows between tokens and
// experts.  Each reads its inputs once and writes its outputs once, 16 bytes a
// lane; memory bounds them all.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm_ffn_math.hpp"

namespace tgemm {
namespace ffn {
namespace {

// ---------------------------------------------------------------------------
// dZ = dC * act'(Z); gated, Z = [G | U]: dG = dC U act'(G), dU = dC act(G).
// dbias = column sums of dZ before its rounding.
//
// A workgroup takes kGradRows rows of one group and 256 output columns: 32
// threads of 8 columns side by side, 8 rows at a time.  Its column sums go to
// a workspace row of their own, and a second kernel adds a group's rows in
// order, so that the sums do not depend on timing (atomics would).  dZ is
// rounded once, to the type that the products behind it take, after its columns
// are summed.  4096 x 4096 of
// gelu_tanh: 22.3 us for 100 MB (4.5 TB/s; a copy reaches 5.2), its sums 4.9 us.
// ---------------------------------------------------------------------------
struct GradArgs {
  const uint8_t *dout, *pre;
  uint8_t *dz;
  float *ws;
  const int32_t *offsets;
  int M, N, out_n;  // N: columns of dz; out_n: of dout
  int ldd, ldp, ldz;
  int act, groups, tiles_n;
};

template <int DT, bool GATED, bool GROUPED>
__global__ __launch_bounds__(256) void act_grad_kernel(const GradArgs a) {
  constexpr int kParts = GATED ? 2 : 1;
  __shared__ float sums[kParts][8][256];
  const int lane = threadIdx.x & 63, tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int chunk = (int)blockIdx.x / a.tiles_n, ct = (int)blockIdx.x % a.tiles_n;
  int r0, r1;
  if constexpr (GROUPED) {
    const Found f = find_unit(a.offsets, a.groups, a.M, chunk, kGradRows, 1, lane);
    if (f.e < 0) return;
    r0 = f.lo + f.unit * kGradRows;
    r1 = min(r0 + kGradRows, f.hi);
  } else {
    r0 = chunk * kGradRows;
    r1 = min(r0 + kGradRows, a.M);
  }
  const int n = ct * 256 + tx * 8;
  const bool in = n < a.out_n;
  float s[kParts][8] = {};
  if (in) {
    with_act<GATED>(a.act, [&](auto act_) {
      constexpr int ACT = decltype(act_)::value;
#pragma unroll 2
      for (int r = r0 + ty; r < r1; r += 8) {
        float d[8], g[8], u[8], f, df;
        unpack8<DT>(*(const v4u *)(a.dout + ((size_t)r * a.ldd + n) * 2), d);
        if constexpr (ACT != kNone) {
          const uint8_t *p = a.pre + ((size_t)r * a.ldp + n) * 2;
          unpack8<DT>(*(const v4u *)p, g);
          if constexpr (GATED) unpack8<DT>(*(const v4u *)(p + (size_t)a.out_n * 2), u);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if constexpr (ACT == kNone) {
            g[q] = d[q];
          } else {
            act_both<ACT>(g[q], f, df);
            if constexpr (GATED) {
              g[q] = d[q] * u[q] * df;
              u[q] = d[q] * f;
              s[1][q] += u[q];
            } else {
              g[q] = d[q] * df;
            }
          }
          s[0][q] += g[q];
        }
        if (a.dz) {
          uint8_t *p = a.dz + ((size_t)r * a.ldz + n) * 2;
          *(v4u *)p = pack8<DT>(g);
          if constexpr (GATED) *(v4u *)(p + (size_t)a.out_n * 2) = pack8<DT>(u);
        }
      }
    });
  }
  if (!a.ws) return;
#pragma unroll
  for (int p = 0; p < kParts; ++p)
#pragma unroll
    for (int q = 0; q < 8; ++q) sums[p][ty][tx * 8 + q] = s[p][q];
  __syncthreads();
  const int c = ct * 256 + (int)threadIdx.x;
  if (c >= a.out_n) return;
#pragma unroll
  for (int p = 0; p < kParts; ++p) {
    float v = 0.0f;
#pragma unroll
    for (int y = 0; y < 8; ++y) v += sums[p][y][threadIdx.x];
    a.ws[(size_t)chunk * a.N + p * a.out_n + c] = v;
  }
}

struct BiasArgs {
  const float *ws;
  uint8_t *dbias;
  const int32_t *offsets;
  int M, N, groups, tiles_n, chunks;  // chunks: rows of ws
};

// 64 columns of one group's sums: four waves take its workspace rows in turn.
template <int DT, bool GROUPED>
__global__ __launch_bounds__(256) void bias_sum_kernel(const BiasArgs a) {
  __shared__ float sums[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = (int)blockIdx.x / a.tiles_n, n = ((int)blockIdx.x % a.tiles_n) * 64 + lane;
  int first = 0, count;
  if constexpr (GROUPED) {
    first = total_units(a.offsets, e, a.M, kGradRows, 1, lane);
    const Range r = group_rows(a.offsets, e, a.M);
    count = (r.hi - r.lo + kGradRows - 1) / kGradRows;
    // (Offsets that are no offsets may count more blocks than there are.)
    if (first < 0 || first > a.chunks) first = a.chunks;
    count = min(count, a.chunks - first);
  } else {
    count = a.chunks;
  }
  float v = 0.0f;
  if (n < a.N) {
#pragma unroll 4
    for (int c = wave; c < count; c += 4) v += a.ws[(size_t)(first + c) * a.N + n];
  }
  sums[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && n < a.N) {
    const float t = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
    *(uint16_t *)(a.dbias + ((size_t)e * a.N + n) * 2) = (uint16_t)(pack2<DT>(t, 0.0f) & 0xffffu);
  }
}

template <int DT>
hipError_t launch_grad_dt(const ActGrad &g) {
  const bool gated = is_gated(g.act);
  GradArgs a{static_cast<const uint8_t *>(g.dout), static_cast<const uint8_t *>(g.preact),
             static_cast<uint8_t *>(g.dz), g.dbias ? g.ws : nullptr, g.offsets, (int)g.M, (int)g.N,
             (int)(gated ? g.N / 2 : g.N), (int)g.ldd, (int)g.ldp, (int)g.ldz, g.act, (int)g.groups, 0};
  a.tiles_n = (a.out_n + 255) / 256;
  const int64_t chunks = g.groups ? act_grad_chunks(g.M, g.groups) : (g.M + kGradRows - 1) / kGradRows;
  const int64_t wgs = chunks * a.tiles_n;
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  hipError_t e = hipSuccess;
  if (g.dz || g.dbias) {
    void *args[] = {&a};
    const void *fn = g.groups ? (gated ? reinterpret_cast<const void *>(&act_grad_kernel<DT, true, true>)
                                       : reinterpret_cast<const void *>(&act_grad_kernel<DT, false, true>))
                              : (gated ? reinterpret_cast<const void *>(&act_grad_kernel<DT, true, false>)
                                       : reinterpret_cast<const void *>(&act_grad_kernel<DT, false, false>));
    if (wgs > 0) e = hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(256), args, 0, g.stream);
  }
  if (e != hipSuccess || !g.dbias) return e;
  BiasArgs b{g.ws, static_cast<uint8_t *>(g.dbias), g.offsets, (int)g.M, (int)g.N, (int)g.groups,
             (int)((g.N + 63) / 64), (int)chunks};
  const int64_t sums = (g.groups ? g.groups : 1) * b.tiles_n;
  if (sums > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  void *args[] = {&b};
  const void *fn = g.groups ? reinterpret_cast<const void *>(&bias_sum_kernel<DT, true>)
                            : reinterpret_cast<const void *>(&bias_sum_kernel<DT, false>);
  return hipLaunchKernel(fn, dim3((unsigned)sums), dim3(256), args, 0, g.stream);
}

// ---------------------------------------------------------------------------
// The K split's second part: the planes of 32-bit sums added in their order
// (no atomics: the same bits each time), then the epilogue.  A thread takes 8
// output columns of a row, 4 planes' loads in flight; the planes come from the
// caches that the split left them in.  Its launch and the planes' way through
// memory are about 2.5 us of the 13.8 of 512 x 512 x 8192 in 4 splits.
// ---------------------------------------------------------------------------
struct JoinArgs {
  const float *ws;
  const uint8_t *bias, *res;
  uint8_t *pre, *C;
  int M, N, out_n, splits;  // N: columns of a plane
  int ldr, ldp, ldc, act;
};

template <int DT, bool GATED>
__global__ __launch_bounds__(256) void join_kernel(const JoinArgs a) {
  const int per = a.out_n >> 3;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)a.M * per) return;
  const int m = (int)(i / per), n = (int)(i - (int64_t)m * per) * 8;
  const size_t plane = (size_t)a.M * a.N;
  auto sum8 = [&](int col, float (&v)[8]) {
    const float *p = a.ws + (size_t)m * a.N + col;
    v4f lo = *(const v4f *)p, hi = *(const v4f *)(p + 4);
#pragma unroll 4
    for (int s = 1; s < a.splits; ++s) {
      lo += *(const v4f *)(p + s * plane);
      hi += *(const v4f *)(p + s * plane + 4);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = lo[q];
      v[4 + q] = hi[q];
    }
  };
  auto add8 = [&](const uint8_t *p, float (&v)[8]) {
    float t[8];
    unpack8<DT>(*(const v4u *)p, t);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] += t[q];
  };
  float z[8], u[8];
  sum8(n, z);
  if constexpr (GATED) sum8(a.out_n + n, u);
  if (a.bias) {
    add8(a.bias + (size_t)n * 2, z);
    if constexpr (GATED) add8(a.bias + (size_t)(a.out_n + n) * 2, u);
  }
  if (a.pre) {
    uint8_t *p = a.pre + ((size_t)m * a.ldp + n) * 2;
    *(v4u *)p = pack8<DT>(z);
    if constexpr (GATED) *(v4u *)(p + (size_t)a.out_n * 2) = pack8<DT>(u);
  }
  with_act<GATED>(a.act, [&](auto act) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      z[q] = act_fwd<decltype(act)::value>(z[q]);
      if constexpr (GATED) z[q] *= u[q];
    }
  });
  if (a.res) add8(a.res + ((size_t)m * a.ldr + n) * 2, z);
  *(v4u *)(a.C + ((size_t)m * a.ldc + n) * 2) = pack8<DT>(z);
}

// ---------------------------------------------------------------------------
// Rows to experts and back.  A wave takes one row (or 512 columns of one):
// its index is the same for all lanes.  Rows of 2048 columns: 8192 gathered
// from 4096 13.0 us (50 MB through memory and 17 again from the caches, 5.2
// TB/s); 8192 tokens of 4 experts combined 28 us (168 MB, 6.0 TB/s, part of it
// from the caches); the gradients of 4096 tokens of 2 experts 15.6 us (101 MB).
// ---------------------------------------------------------------------------
struct GatherArgs {
  const uint8_t *x;
  uint8_t *out;
  const int32_t *rows;
  int R, D, src_rows, ldx, ldo;
};

__global__ __launch_bounds__(256) void gather_kernel(const GatherArgs a) {
  const int lane = threadIdx.x & 63;
  const int r = __builtin_amdgcn_readfirstlane((int)blockIdx.x * 4 + ((int)threadIdx.x >> 6));
  if (r >= a.R) return;
  const int src = a.rows[r];
  if (src < 0 || src >= a.src_rows) return;
  const uint8_t *from = a.x + (size_t)src * a.ldx * 2;
  uint8_t *to = a.out + (size_t)r * a.ldo * 2;
#pragma unroll 4
  for (int n = lane * 8; n < a.D; n += 512) *(v4u *)(to + (size_t)n * 2) = *(const v4u *)(from + (size_t)n * 2);
}

struct CombineArgs {
  const uint8_t *h, *res;
  uint8_t *out;
  const int32_t *slots;
  const float *weights;
  int T, D, R, k, ldh, ldr, ldo, segs;
};

// out[t] = sum over j = 0, 1, ... of weights[t][j] h[slots[t][j]], + residual,
// summed in binary32 and rounded once.  Four rows are loaded ahead.
template <int DT>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t = __builtin_amdgcn_readfirstlane((int)(w / a.segs));
  if (t >= a.T) return;
  const int n = (int)(w - (int64_t)t * a.segs) * 512 + lane * 8;
  if (n >= a.D) return;
  float acc[8] = {};
  if (a.res) unpack8<DT>(*(const v4u *)(a.res + ((size_t)t * a.ldr + n) * 2), acc);
  float sum[8] = {};
  for (int j0 = 0; j0 < a.k; j0 += 4) {
    v4u v[4] = {};
    float wt[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = j0 + i < a.k ? a.slots[(size_t)t * a.k + j0 + i] : -1;
      const bool ok = s >= 0 && s < a.R;
      // (A choice without a row adds nothing, whatever its weight.)
      wt[i] = !ok ? 0.0f : a.weights ? a.weights[(size_t)t * a.k + j0 + i] : 1.0f;
      if (ok) v[i] = *(const v4u *)(a.h + ((size_t)s * a.ldh + n) * 2);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
      unpack8<DT>(v[i], x);
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] = fmaf(wt[i], x[q], sum[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] += sum[q];
  *(v4u *)(a.out + ((size_t)t * a.ldo + n) * 2) = pack8<DT>(acc);
}

struct CombineGradArgs {
  const uint8_t *dout, *h;
  uint8_t *dh;
  const int32_t *slots;
  const float *weights;
  float *dweights;
  int T, D, R, k, ldd, ldh, ldg;
};

// One wave a choice: dh[slot] = weight dout[t], dweight = dout[t] . h[slot].
// dh is rounded once, to the type that the two products behind it take; the dot
// product stays in binary32.  (Choices that share a row write over one another:
// a plan's do not.)
template <int DT>
__global__ __launch_bounds__(256) void combine_grad_kernel(const CombineGradArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= (int64_t)a.T * a.k) return;
  const int c = __builtin_amdgcn_readfirstlane((int)w);
  const int s = a.slots[c], t = c / a.k;
  if (s < 0 || s >= a.R) {
    if (lane == 0) a.dweights[c] = 0.0f;
    return;
  }
  const float wt = a.weights[c];
  const uint8_t *d = a.dout + (size_t)t * a.ldd * 2, *h = a.h + (size_t)s * a.ldh * 2;
  uint8_t *to = a.dh + (size_t)s * a.ldg * 2;
  float dot = 0.0f;
#pragma unroll 4
  for (int n = lane * 8; n < a.D; n += 512) {
    float dv[8], hv[8];
    unpack8<DT>(*(const v4u *)(d + (size_t)n * 2), dv);
    unpack8<DT>(*(const v4u *)(h + (size_t)n * 2), hv);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      dot = fmaf(dv[q], hv[q], dot);
      dv[q] *= wt;
    }
    *(v4u *)(to + (size_t)n * 2) = pack8<DT>(dv);
  }
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) dot += __shfl_xor(dot, m, 64);
  if (lane == 0) a.dweights[c] = dot;
}

hipError_t launch_waves(const void *fn, int64_t waves, void *args, hipStream_t stream) {
  const int64_t wgs = (waves + 3) / 4;
  if (wgs == 0) return hipSuccess;
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  void *argv[] = {args};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(256), argv, 0, stream);
}

}  // namespace

hipError_t launch_act_grad(const ActGrad &g) { return g.dtype == 1 ? launch_grad_dt<1>(g) : launch_grad_dt<0>(g); }

hipError_t launch_join(const Gemm &g) {
  const bool gated = is_gated(g.act);
  JoinArgs a{g.ws, static_cast<const uint8_t *>(g.bias), static_cast<const uint8_t *>(g.residual),
             static_cast<uint8_t *>(g.preact), static_cast<uint8_t *>(g.C), (int)g.M, (int)g.N,
             (int)(gated ? g.N / 2 : g.N), g.splits, (int)g.ldr, (int)g.ldp, (int)g.ldc, g.act};
  const int64_t wgs = ((int64_t)a.M * (a.out_n / 8) + 255) / 256;
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  const void *fn = g.dtype == 1 ? (gated ? reinterpret_cast<const void *>(&join_kernel<1, true>)
                                         : reinterpret_cast<const void *>(&join_kernel<1, false>))
                                : (gated ? reinterpret_cast<const void *>(&join_kernel<0, true>)
                                         : reinterpret_cast<const void *>(&join_kernel<0, false>));
  void *args[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(256), args, 0, g.stream);
}

hipError_t launch_gather(const Gather &g) {
  GatherArgs a{static_cast<const uint8_t *>(g.x), static_cast<uint8_t *>(g.out), g.rows, (int)g.R, (int)g.D,
               (int)g.src_rows, (int)g.ldx, (int)g.ldo};
  return launch_waves(reinterpret_cast<const void *>(&gather_kernel), g.R, &a, g.stream);
}

hipError_t launch_combine(const Combine &c) {
  CombineArgs a{static_cast<const uint8_t *>(c.h), static_cast<const uint8_t *>(c.residual),
                static_cast<uint8_t *>(c.out), c.slots, c.weights, (int)c.T, (int)c.D, (int)c.R, c.k, (int)c.ldh,
                (int)c.ldr, (int)c.ldo, (int)((c.D + 511) / 512)};
  const void *fn = c.dtype == 1 ? reinterpret_cast<const void *>(&combine_kernel<1>)
                                : reinterpret_cast<const void *>(&combine_kernel<0>);
  return launch_waves(fn, c.T * a.segs, &a, c.stream);
}

hipError_t launch_combine_grad(const CombineGrad &c) {
  CombineGradArgs a{static_cast<const uint8_t *>(c.dout), static_cast<const uint8_t *>(c.h),
                    static_cast<uint8_t *>(c.dh), c.slots, c.weights, c.dweights, (int)c.T, (int)c.D, (int)c.R, c.k,
                    (int)c.ldd, (int)c.ldh, (int)c.ldg};
  const void *fn = c.dtype == 1 ? reinterpret_cast<const void *>(&combine_grad_kernel<1>)
                                : reinterpret_cast<const void *>(&combine_grad_kernel<0>);
  return launch_waves(fn, c.T * c.k, &a, c.stream);
}

}  // namespace ffn
}  // namespace tgemm
