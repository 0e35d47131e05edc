// Quantisation to MXFP4 and back, for gfx950.
//
// A block of 32 consecutive values shares the scale 2^e, the least power of
// two with max|x| <= 6 * 2^e; an element is x * 2^-e rounded to nearest even
// among 0, 0.5, 1, 1.5, 2, 3, 4, 6.  With the maximum's binary32 bits as a whole
// number b, e + 127 = (b + 0x3fffff >> 23) - 2, at least 0: the addition carries
// into the exponent exactly where the mantissa is above 1.5 (6 = 1.5 * 2^2).
// Magnitudes are compared as whole numbers too, 16-bit ones two at a time, which
// finds infinities and NaN on the way; the conversion scales, rounds and
// takes 16-bit values as they are.  Memory bounds all of it: 2 or 4 bytes a value
// in, 17/32 out.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm_ffn_math.hpp"

namespace tgemm {
namespace ffn {
namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// The scale byte of a block whose largest magnitude has these binary32 bits.
__device__ __forceinline__ uint32_t scale_of(uint32_t top) {
  const int e = (int)((top + 0x3fffffu) >> 23) - 2;
  return top >= kInfBits ? 255u : (uint32_t)max(e, 0);
}
// 2^e of a scale byte.
__device__ __forceinline__ float power_of(uint32_t byte) {
  return __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);
}

// Values as they lie in memory: kPer of them a dword.
template <int DT>
struct Raw {
  static constexpr int kPer = DT == 2 ? 1 : 2;
  // Largest magnitudes so far of a dword's values, each by itself.
  __device__ static __forceinline__ uint32_t top(uint32_t m, uint32_t w) {
    if constexpr (DT == 2) {
      return max(m, w & 0x7fffffffu);
    } else {
      typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
      const u16x2 a = __builtin_bit_cast(u16x2, m), b = __builtin_bit_cast(u16x2, w & 0x7fff7fffu);
      return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
    }
  }
  // The larger one's binary32 bits.
  __device__ static __forceinline__ uint32_t bits(uint32_t m) {
    if constexpr (DT == 2) return m;
    const uint32_t t = max(m >> 16, m & 0xffffu);
    return __builtin_bit_cast(uint32_t, to_f32<DT>(t));
  }
  // Elements of two values (a dword, or the two dwords w and v) into byte B of q.
  template <int B>
  __device__ static __forceinline__ uint32_t convert(uint32_t q, uint32_t w, uint32_t v, float scale) {
    if constexpr (DT == 2)
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __builtin_bit_cast(float, w), __builtin_bit_cast(float, v), scale, B);
    else if constexpr (DT == 1)
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(v2h, w), scale, B);
    else
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(v2bf, w), scale, B);
  }
  // Elements of eight consecutive values (8 / kPer dwords); none of a block whose scale is NaN.
  __device__ static __forceinline__ uint32_t eight(const uint32_t *w, uint32_t byte) {
    const float scale = power_of(byte);
    constexpr int S = DT == 2 ? 2 : 1;
    uint32_t q = convert<0>(0, w[0], w[S - 1], scale);
    q = convert<1>(q, w[S], w[2 * S - 1], scale);
    q = convert<2>(q, w[2 * S], w[3 * S - 1], scale);
    q = convert<3>(q, w[3 * S], w[4 * S - 1], scale);
    return byte == 255u ? 0u : q;
  }
};

// Eight values from memory.
template <int DT>
struct Eight {
  uint32_t w[8 / Raw<DT>::kPer];
  __device__ __forceinline__ void load(const uint8_t *p) {
#pragma unroll
    for (int i = 0; i < (DT == 2 ? 2 : 1); ++i) {
      const v4u v = *(const v4u *)(p + 16 * i);
#pragma unroll
      for (int q = 0; q < 4; ++q) w[4 * i + q] = v[q];
    }
  }
  // The scale byte of the block that four lanes hold together.
  __device__ __forceinline__ uint32_t scale() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8 / Raw<DT>::kPer; ++i) m = Raw<DT>::top(m, w[i]);
    m = Raw<DT>::top(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, true));  // lanes 1 0 3 2
    m = Raw<DT>::top(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, true));  // lanes 2 3 0 1
    return scale_of(Raw<DT>::bits(m));
  }
};

struct QuantArgs {
  const uint8_t *x;
  uint8_t *q, *s, *qt, *st;
  int M, N;
  int64_t ldx;  // bytes
  int64_t ldq, ldqt;
  int tiles_n;
};

// Rows alone: a lane takes 8 values, four lanes a block; a workgroup 2048
// values of a row.  8192 x 4096 bf16 17 us (85 MB, 5.0 TB/s); 1 x 4096 1.6.
template <int DT>
__global__ __launch_bounds__(256) void quant_rows_kernel(const QuantArgs a) {
  constexpr int kB = DT == 2 ? 4 : 2;
  const int row = (int)(blockIdx.x / (unsigned)a.tiles_n);
  const int n = ((int)(blockIdx.x % (unsigned)a.tiles_n) * 256 + (int)threadIdx.x) * 8;
  if (n >= a.N) return;  // (N % 32 == 0: the four lanes of a block go together)
  Eight<DT> v;
  v.load(a.x + (size_t)row * a.ldx + (size_t)n * kB);
  const uint32_t e = v.scale();
  *(uint32_t *)(a.q + (size_t)row * a.ldq + (n >> 1)) = Raw<DT>::eight(v.w, e);
  if ((threadIdx.x & 3) == 0) a.s[(size_t)row * (a.N >> 5) + (n >> 5)] = (uint8_t)e;
}

// Columns, and rows with them: a workgroup takes 128 rows x 256 bytes of each
// (128 16-bit columns, 64 of binary32).  A thread loads 8 pieces of 16 bytes of 8
// rows (4 of 32 bytes), from which four lanes make up a row's block on the spot;
// the tile goes to LDS as it lies, and a thread then takes a dword of 32 rows: a
// block of two columns, or of one.  Lanes 4 c .. 4 c + 3 take the four row blocks
// of dword c, whose 64 bytes of a column they write side by side; the blocks lie
// 16 dwords further apart than their rows, so that these reads spread over all banks.
// An XCD takes tiles side by side, two across and on down the rows: outputs that
// share a cache line meet in its L2.  Both ways, 3999 x 4992 binary32 24 us (101 MB,
// 4.2 TB/s; tiles half as wide 37, twice as wide the same), 4001 x 4096 bf16 12 (50 MB);
// a 64-byte piece of a column is what is written at once, half a cache line.
// The stores into the tile do meet on banks: in binary32 a lane's 16 bytes lie 32
// from the next one's, so that each store uses half of the banks (of the LDS's busy
// cycles 50%; 33% with 16-bit values).  What that costs has not been measured.
template <int DT, bool ROWS>
__global__ __launch_bounds__(256) void quant_columns_kernel(const QuantArgs a) {
  constexpr int kB = DT == 2 ? 4 : 2, kPer = Raw<DT>::kPer, kTM = 128, kTN = 64 * kPer;
  constexpr int kLanes = kTN / 8;              // threads across a row: 16 bytes each, 32 of binary32
  constexpr int kRows = 256 / kLanes, kPasses = kTM / kRows, kBlock = 32 * 64 + 16;
  __shared__ __attribute__((aligned(16))) uint32_t tile[4 * kBlock];
  const int tiles_m = (a.M + kTM - 1) / kTM, total = tiles_m * a.tiles_n;
  const int wg = (int)blockIdx.x, xcd = wg & 7, base = total >> 3, rem = total & 7;
  const int v0 = xcd * base + min(xcd, rem) + (wg >> 3);
  const int strip = v0 / (2 * tiles_m), across = min(a.tiles_n - 2 * strip, 2), in = v0 - strip * 2 * tiles_m;
  const int m0 = in / across * kTM, n0 = (2 * strip + in % across) * kTN;
  const int r0 = (int)threadIdx.x / kLanes, c0 = (int)threadIdx.x % kLanes;
  Eight<DT> v[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int m = m0 + i * kRows + r0, n = n0 + 8 * c0;
    v[i] = Eight<DT>{};
    if (m < a.M && n < a.N) v[i].load(a.x + (size_t)m * a.ldx + (size_t)n * kB);
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + r0;
#pragma unroll
    for (int h = 0; h < 2 / kPer; ++h) {
      *(v4u *)&tile[(r >> 5) * kBlock + (r & 31) * 64 + (8 / kPer) * c0 + 4 * h] = v4u{v[i].w[4 * h], v[i].w[4 * h + 1], v[i].w[4 * h + 2], v[i].w[4 * h + 3]};
    }
    if constexpr (ROWS) {
      const int m = m0 + r, n = n0 + 8 * c0;
      const uint32_t e = v[i].scale();
      if (m < a.M && n < a.N) {
        *(uint32_t *)(a.q + (size_t)m * a.ldq + (n >> 1)) = Raw<DT>::eight(v[i].w, e);
        if ((threadIdx.x & 3) == 0) a.s[(size_t)m * (a.N >> 5) + (n >> 5)] = (uint8_t)e;
      }
    }
  }
  __syncthreads();
  const int blocks = (a.M + 31) >> 5;  // of a column
  const int c = (int)threadIdx.x >> 2, b = (int)threadIdx.x & 3;
  if ((m0 >> 5) + b >= blocks || n0 + kPer * c >= a.N) return;
  uint32_t w[32], m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    w[i] = tile[b * kBlock + i * 64 + c];
    m = Raw<DT>::top(m, w[i]);
  }
#pragma unroll
  for (int h = 0; h < kPer; ++h) {
    const uint32_t e = scale_of(Raw<DT>::bits(kPer == 1 ? m : h ? m & 0xffff0000u : m & 0xffffu));
    v4u q;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      uint32_t x[8 / kPer];
#pragma unroll
      for (int i = 0; i < 8 / kPer; ++i) {
        if constexpr (kPer == 1)
          x[i] = w[8 * o + i];
        else  // (the values of two rows side by side)
          x[i] = __builtin_amdgcn_perm(w[8 * o + 2 * i + 1], w[8 * o + 2 * i], h ? 0x07060302u : 0x05040100u);
      }
      q[o] = Raw<DT>::eight(x, e);
    }
    const size_t n = (size_t)(n0 + kPer * c + h);
    *(v4u *)(a.qt + n * a.ldqt + (m0 >> 1) + 16 * b) = q;
    a.st[n * blocks + (m0 >> 5) + b] = (uint8_t)e;
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
    constexpr int kTN = 64 * Raw<DT>::kPer;
    a.tiles_n = (int)((g.N + kTN - 1) / kTN);
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

// A lane takes 8 values (4 bytes).  8192 x 4096 to bf16 16 us (85 MB, 5.3 TB/s).
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
