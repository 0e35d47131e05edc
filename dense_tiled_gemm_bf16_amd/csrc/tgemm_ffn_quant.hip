// Quantisation to MXFP4 and back, for gfx950.
//
// A block of 32 consecutive values shares the scale 2^e, the least power of
// two with max|x| <= 6 * 2^e; an element is x * 2^-e rounded to nearest even
// among 0, 0.5, 1, 1.5, 2, 3, 4, 6.  With the maximum's bits as a whole number
// b, e + 127 = (b + 0x3fffff >> 23) - 2, at least 0: the addition carries into
// the exponent exactly where the mantissa is above 1.5 (6 = 1.5 * 2^2).  The
// scaling is an exact multiplication and the rounding the hardware's
// conversion.  Memory bounds all of it: 2 or 4 bytes a value in, 17/32 out.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm_ffn_math.hpp"

namespace tgemm {
namespace ffn {
namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
  const int e = (int)((top + 0x3fffffu) >> 23) - 2;
  return top >= kInfBits ? 255u : (uint32_t)max(e, 0);
}
// 2^-e of a scale byte (0 of the NaN: its elements are zeros).
__device__ __forceinline__ float inverse_of(uint32_t byte) {
  return byte == 255u ? 0.0f : __builtin_bit_cast(float, (254u - byte) << 23);
}
// Eight values times 2^-e as elements; v finite, or inv 0.
__device__ __forceinline__ uint32_t elements8(const float (&v)[8], float inv) {
  uint32_t w = 0;
  if (inv == 0.0f) return 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * inv, v[1] * inv, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * inv, v[3] * inv, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * inv, v[5] * inv, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * inv, v[7] * inv, 1.0f, 3);
  return w;
}
__device__ __forceinline__ uint32_t top_of(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < 8; ++q) m = max(m, __builtin_bit_cast(uint32_t, v[q]) & 0x7fffffffu);
  return m;
}

template <int DT>
__device__ __forceinline__ void load8(const uint8_t *p, float (&v)[8]) {
  if constexpr (DT == 2) {
    const v4f lo = *(const v4f *)p, hi = *(const v4f *)(p + 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = lo[q];
      v[4 + q] = hi[q];
    }
  } else {
    unpack8<DT>(*(const v4u *)p, v);
  }
}

struct QuantArgs {
  const uint8_t *x;
  uint8_t *q, *s, *qt, *st;
  int M, N;
  int64_t ldx;  // bytes
  int64_t ldq, ldqt;
  int tiles_n;
};

// Rows alone: a lane takes 8 values, four lanes a block; a workgroup 2048
// values of a row.
template <int DT>
__global__ __launch_bounds__(256) void quant_rows_kernel(const QuantArgs a) {
  constexpr int kB = DT == 2 ? 4 : 2;
  const int row = (int)(blockIdx.x / (unsigned)a.tiles_n);
  const int n = ((int)(blockIdx.x % (unsigned)a.tiles_n) * 256 + (int)threadIdx.x) * 8;
  if (n >= a.N) return;  // (N % 32 == 0: the four lanes of a block go together)
  float v[8];
  load8<DT>(a.x + (size_t)row * a.ldx + (size_t)n * kB, v);
  uint32_t m = top_of(v);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
  const uint32_t e = scale_of(m);
  *(uint32_t *)(a.q + (size_t)row * a.ldq + (n >> 1)) = elements8(v, inverse_of(e));
  if ((threadIdx.x & 3) == 0) a.s[(size_t)row * (a.N >> 5) + (n >> 5)] = (uint8_t)e;
}

// Columns, and rows with them: a workgroup takes 128 rows x 64 columns through
// LDS.  A thread then takes 32 rows of one column (and writes their 16 bytes);
// for the rows, 32 columns of one row.
template <int DT, bool ROWS>
__global__ __launch_bounds__(256) void quant_columns_kernel(const QuantArgs a) {
  constexpr int kB = DT == 2 ? 4 : 2, kTM = 128, kTN = 64, kPitch = kTN + 1;
  __shared__ float tile[kTM * kPitch];
  const int m0 = (int)(blockIdx.x / (unsigned)a.tiles_n) * kTM, n0 = (int)(blockIdx.x % (unsigned)a.tiles_n) * kTN;
#pragma unroll
  for (int i = 0; i < kTM * kTN / 8 / 256; ++i) {
    const int at = i * 256 + (int)threadIdx.x, r = at / (kTN / 8), c = at % (kTN / 8) * 8;
    float v[8] = {};
    if (m0 + r < a.M && n0 + c < a.N) load8<DT>(a.x + (size_t)(m0 + r) * a.ldx + (size_t)(n0 + c) * kB, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) tile[r * kPitch + c + q] = v[q];
  }
  __syncthreads();
  const int blocks = (a.M + 31) >> 5;  // of a column
  {
    const int c = (int)threadIdx.x & 63, b = (int)threadIdx.x >> 6;
    if (n0 + c < a.N && (m0 >> 5) + b < blocks) {
      float v[4][8];
      uint32_t top = 0;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[h][q] = tile[(32 * b + 8 * h + q) * kPitch + c];
        top = max(top, top_of(v[h]));
      }
      const uint32_t e = scale_of(top);
      const float inv = inverse_of(e);
      v4u w;
#pragma unroll
      for (int h = 0; h < 4; ++h) w[h] = elements8(v[h], inv);
      *(v4u *)(a.qt + (size_t)(n0 + c) * a.ldqt + (m0 >> 1) + 16 * b) = w;
      a.st[(size_t)(n0 + c) * blocks + (m0 >> 5) + b] = (uint8_t)e;
    }
  }
  if constexpr (ROWS) {
    const int r = (int)threadIdx.x >> 1, b = (int)threadIdx.x & 1;
    if (m0 + r < a.M && n0 + 32 * b < a.N) {
      float v[4][8];
      uint32_t top = 0;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[h][q] = tile[r * kPitch + 32 * b + 8 * h + q];
        top = max(top, top_of(v[h]));
      }
      const uint32_t e = scale_of(top);
      const float inv = inverse_of(e);
      v4u w;
#pragma unroll
      for (int h = 0; h < 4; ++h) w[h] = elements8(v[h], inv);
      *(v4u *)(a.q + (size_t)(m0 + r) * a.ldq + (n0 >> 1) + 16 * b) = w;
      a.s[(size_t)(m0 + r) * (a.N >> 5) + (n0 >> 5) + b] = (uint8_t)e;
    }
  }
}

template <int DT>
hipError_t launch_quant_dt(const Quant &g) {
  QuantArgs a{static_cast<const uint8_t *>(g.x), g.q, g.scales, g.qt, g.scalest, (int)g.M, (int)g.N,
              g.ldx * (DT == 2 ? 4 : 2), g.ldq, g.ldqt, 0};
  void *args[] = {&a};
  const void *fn;
  int64_t wgs;
  if (g.qt) {
    a.tiles_n = (int)((g.N + 63) / 64);
    wgs = (g.M + 127) / 128 * a.tiles_n;
    fn = g.q ? reinterpret_cast<const void *>(&quant_columns_kernel<DT, true>)
             : reinterpret_cast<const void *>(&quant_columns_kernel<DT, false>);
  } else {
    a.tiles_n = (int)((g.N + 2047) / 2048);
    wgs = g.M * a.tiles_n;
    fn = reinterpret_cast<const void *>(&quant_rows_kernel<DT>);
  }
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(256), args, 0, g.stream);
}

struct DequantArgs {
  const uint8_t *q, *s;
  uint8_t *out;
  int M, N;
  int64_t ldq, ldo;  // bytes
  int tiles_n;
};

// A lane takes 8 values (4 bytes).
template <int DT>
__global__ __launch_bounds__(256) void dequant_kernel(const DequantArgs a) {
  constexpr int kB = DT == 2 ? 4 : 2;
  const int row = (int)(blockIdx.x / (unsigned)a.tiles_n);
  const int n = ((int)(blockIdx.x % (unsigned)a.tiles_n) * 256 + (int)threadIdx.x) * 8;
  if (n >= a.N) return;
  const uint32_t w = *(const uint32_t *)(a.q + (size_t)row * a.ldq + (n >> 1));
  const uint32_t byte = a.s[(size_t)row * (a.N >> 5) + (n >> 5)];
  // 2^e in two factors: e = -127 is below the normal numbers.
  const float up = __builtin_bit_cast(float, byte == 255u ? 0x7fc00000u : (byte > 0 ? byte : 1u) << 23);
  const float scale = byte == 0 ? 0.5f : 1.0f;
  float v[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t c = (w >> (4 * q)) & 15u, m = c & 7u;
    // Exponent bits 1-2 and mantissa bit 0 as binary32's: (m + 252) / 2 powers;
    // code 1 is 0.5, which that would make 0.75.
    const uint32_t bits = m < 2u ? (m ? 0x3f000000u : 0u) : (m + 252u) << 22;
    v[q] = __builtin_bit_cast(float, bits | ((c & 8u) << 28)) * scale * up;
  }
  uint8_t *p = a.out + (size_t)row * a.ldo + (size_t)n * kB;
  if constexpr (DT == 2) {
    *(v4f *)p = v4f{v[0], v[1], v[2], v[3]};
    *(v4f *)(p + 16) = v4f{v[4], v[5], v[6], v[7]};
  } else {
    *(v4u *)p = pack8<DT>(v);
  }
}

template <int DT>
hipError_t launch_dequant_dt(const Dequant &g) {
  DequantArgs a{g.q, g.scales, static_cast<uint8_t *>(g.out), (int)g.M, (int)g.N, g.ldq, g.ldo * (DT == 2 ? 4 : 2),
                (int)((g.N + 2047) / 2048)};
  const int64_t wgs = g.M * a.tiles_n;
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  void *args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void *>(&dequant_kernel<DT>), dim3((unsigned)wgs), dim3(256), args, 0,
                         g.stream);
}

}  // namespace

hipError_t launch_quant_mxfp4(const Quant &g) {
  return g.dtype == 2 ? launch_quant_dt<2>(g) : g.dtype == 1 ? launch_quant_dt<1>(g) : launch_quant_dt<0>(g);
}
hipError_t launch_dequant_mxfp4(const Dequant &g) {
  return g.dtype == 2 ? launch_dequant_dt<2>(g) : g.dtype == 1 ? launch_dequant_dt<1>(g) : launch_dequant_dt<0>(g);
}

}  // namespace ffn
}  // namespace tgemm
