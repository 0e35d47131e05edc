// The plain products' kernels for gfx950: instances of the kernel template of
// tgemm_kernel.hpp, the K split's reduction and the choice of tile shape.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "tgemm_internal.hpp"
#include "tgemm_kernel.hpp"
#include "tgemm_shapes.hpp"

namespace tgemm {
namespace {

// One workgroup per CU: either shape's ring takes 128 KiB of the 160 KiB
// LDS, and a 256-row tile's accumulators fill a SIMD's registers.
template <class T, int TM, int TN, bool SPLIT = false>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_kernel(const Args a) {
#if defined(__HIP_DEVICE_COMPILE__)  // the body is device code only; the host pass needs the symbol
  // A separate array per slot (not one indexed array) so the compiler can
  // tell the slot being loaded from the slot being read and does not insert
  // a vmcnt wait in front of every LDS read.
  __shared__ __attribute__((aligned(1024))) uint8_t sA0[TM * T::kPitch];
  __shared__ __attribute__((aligned(1024))) uint8_t sA1[TM * T::kPitch];
  __shared__ __attribute__((aligned(1024))) uint8_t sB0[TN * T::kPitch];
  __shared__ __attribute__((aligned(1024))) uint8_t sB1[TN * T::kPitch];
  Slots slots;
  slots.a[0] = (LDS_AS uint8_t *)sA0;
  slots.a[1] = (LDS_AS uint8_t *)sA1;
  slots.b[0] = (LDS_AS uint8_t *)sB0;
  slots.b[1] = (LDS_AS uint8_t *)sB1;
  if constexpr (kSlots<T, TM, TN> == 4) {
    __shared__ __attribute__((aligned(1024))) uint8_t sA2[TM * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sA3[TM * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sB2[TN * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sB3[TN * kRowBytes];
    slots.a[2] = (LDS_AS uint8_t *)sA2;
    slots.a[3] = (LDS_AS uint8_t *)sA3;
    slots.b[2] = (LDS_AS uint8_t *)sB2;
    slots.b[3] = (LDS_AS uint8_t *)sB3;
  }
  slots.junk = nullptr;
  if constexpr (Kernel<T, TM, TN, SPLIT>::kPfDist > 0) {
    __shared__ __attribute__((aligned(256))) uint8_t junk[4 * 256];
    slots.junk = (LDS_AS uint8_t *)junk;
  }
  slots.stage = nullptr;
  if constexpr (Kernel<T, TM, TN, SPLIT>::kStaged) {
    __shared__ __attribute__((aligned(1024))) uint8_t st[Kernel<T, TM, TN, SPLIT>::kStageBytes];
    slots.stage = (LDS_AS uint8_t *)st;
  }
  Kernel<T, TM, TN, SPLIT> k(a, slots);
  k.run();
#endif
}

template <class T, int TM, int TN, bool SPLIT = false>
hipError_t launch_shape(const Problem &p, Args a) {
  a.tiles_m = (int)((p.M + TM - 1) / TM);
  a.tiles_n = (int)((p.N + TN - 1) / TN);
  // A dispatch holds fewer than 2^32 work-items per dimension.
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  const int64_t wgs = tiles * (SPLIT ? a.splits : 1);
  if (wgs > (int64_t)(UINT32_MAX / kThreads)) return hipErrorInvalidConfiguration;
  // hipLaunchKernel returns this launch's own status (hipGetLastError could
  // report an earlier, unrelated failure of the calling thread).
  void *args[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void *>(&gemm_kernel<T, TM, TN, SPLIT>), dim3((unsigned)wgs),
                         dim3(kThreads), args, 0, p.stream);
}

// K split, second pass: C[m][n] = the sum over s = 0, 1, ... splits - 1, in
// that order, of plane s [m][n], rounded to nearest-even bf16 (DT = kBf16)
// or fp16.  One thread per 8 consecutive columns of a row (N % 8 == 0):
// two 16-byte loads per plane, one 16-byte store.
struct ReduceArgs {
  const float *ws;
  uint8_t *C;
  int splits, M, N, ldc;
};

template <int DT>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const ReduceArgs r) {
  const int per_row = r.N >> 3;
  const int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (g >= (int64_t)r.M * per_row) return;
  const int m = (int)(g / per_row);
  const int n = (int)(g - (int64_t)m * per_row) * 8;
  const size_t plane = (size_t)r.M * (size_t)r.N;
  const float *p = r.ws + (size_t)m * r.N + n;
  f32x4 lo = *(const f32x4 *)p, hi = *(const f32x4 *)(p + 4);
  for (int s = 1; s < r.splits; ++s) {
    lo += *(const f32x4 *)(p + s * plane);
    hi += *(const f32x4 *)(p + s * plane + 4);
  }
  u32x4 out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x4 &v = h ? hi : lo;
    const f32x2 x = {v[0], v[1]}, y = {v[2], v[3]};
    if constexpr (DT == kF16) {
      out[2 * h] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16x2));
      out[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, f16x2));
    } else {
      out[2 * h] = __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
      out[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2));
    }
  }
  store_c(r.C + ((size_t)m * r.ldc + n) * 2, out);
}

template <int DT>
hipError_t launch_reduce(const Problem &p, const Args &a) {
  ReduceArgs r{a.ws, a.C, a.splits, a.M, a.N, a.ldc};
  const int64_t blocks = ((int64_t)p.M * (p.N / 8) + 255) / 256;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  void *args[] = {&r};
  return hipLaunchKernel(reinterpret_cast<const void *>(&splitk_reduce_kernel<DT>), dim3((unsigned)blocks),
                         dim3(256), args, 0, p.stream);
}

// The K-split pair of one layout: partial sums, then the reduction.
template <int DT, bool AK, bool BK>
hipError_t launch_split_layout(const Problem &p, const Args &a, int tm, int tn) {
  using T = Traits<DT, AK, BK>;
  hipError_t e = hipErrorInvalidValue;
  if (tm == 128 && tn == 128) e = launch_shape<T, 128, 128, true>(p, a);
  else if (tm == 64 && tn == 64) e = launch_shape<T, 64, 64, true>(p, a);
  if (e != hipSuccess) return e;
  return launch_reduce<DT>(p, a);
}

template <int DT>
hipError_t launch_split_dt(const Problem &p, const Args &a, int tm, int tn) {
  const bool ak = !p.trans_a, bk = p.trans_b;
  if (ak && bk) return launch_split_layout<DT, true, true>(p, a, tm, tn);
  if (ak) return launch_split_layout<DT, true, false>(p, a, tm, tn);
  if (bk) return launch_split_layout<DT, false, true>(p, a, tm, tn);
  return launch_split_layout<DT, false, false>(p, a, tm, tn);
}

// The 16-bit kernels of one operand layout, by tile shape (256 x 192 only
// where B is K-contiguous: a K-major B slot must be 256 or 128 wide).
template <int DT, bool AK, bool BK>
hipError_t launch_layout(const Problem &p, const Args &a, int tm, int tn) {
  using T = Traits<DT, AK, BK>;
  if (tm == 256 && tn == 256) return launch_shape<T, 256, 256>(p, a);
  if constexpr (BK)
    if (tm == 256 && tn == 192) return launch_shape<T, 256, 192>(p, a);
  if (tm == 128 && tn == 128) return launch_shape<T, 128, 128>(p, a);
  if (tm == 64 && tn == 64) return launch_shape<T, 64, 64>(p, a);
  return hipErrorInvalidValue;
}

template <int DT>
hipError_t launch_dt(const Problem &p, const Args &a, int tm, int tn) {
  const bool ak = !p.trans_a, bk = p.trans_b;
  if (ak && bk) return launch_layout<DT, true, true>(p, a, tm, tn);
  if (ak) return launch_layout<DT, true, false>(p, a, tm, tn);
  if (bk) return launch_layout<DT, false, true>(p, a, tm, tn);
  return launch_layout<DT, false, false>(p, a, tm, tn);
}

// Whether to split K, and into how many pieces of which tile shape.  Only
// the 128 x 128 and 64 x 64 tiles have split kernels; with another tile
// forced there is no split (the front end refuses explicit splits then).
// Explicit splits are taken as given (the caller's workspace holds them).
// Automatic ones (p.splits == 0) only where the plain grid leaves at least
// half the CUs idle and K has at least 48 slices (3072 elements): then
// 64 x 64 tiles and at most 4 splits, no more than fill the CUs once, at
// least 16 slices each, and no more than the workspace holds.  Measured
// under graph replay (bf16 NT, us per call, plain -> split): 512 x 512 x 4096
// 10.95 -> 9.68 (3 splits 9.3, 6 splits 12.7), 512 x 512 x 8192 22.5 -> 13.1,
// 256 x 256 x 4096 10.8 -> 7.7; but 768 x 512 x 2048 (32 slices) 6.7 -> 8.4
// with 2 splits: the partial sums' round trip and the second kernel cost
// about 2-3 us, which short K ranges do not repay.  Returns false for no
// split (tm, tn untouched).
bool choose_split(const Problem &p, int ksteps, int &tm, int &tn, int &splits) {
  const bool forced = p.tile_m != 0;
  if (forced && !((p.tile_m == 128 && p.tile_n == 128) || (p.tile_m == 64 && p.tile_n == 64))) return false;
  const uint64_t plane = (uint64_t)p.M * (uint64_t)p.N * 4u;
  const int64_t fit = plane > 0 ? (int64_t)(p.ws_bytes / plane) : 0;
  if (p.splits >= 2) {
    splits = (int)std::min<int64_t>({(int64_t)p.splits, (int64_t)kMaxSplits, (int64_t)ksteps, fit});
    if (splits < 2) return false;
    tm = forced ? p.tile_m : 64;
    tn = forced ? p.tile_n : 64;
    return true;
  }
  const Shape plain = p.trans_b ? pick_shape(kShapesBK, p.M, p.N, p.cus) : pick_shape(kShapesBN, p.M, p.N, p.cus);
  const int64_t plain_tiles = ((p.M + plain.tm - 1) / plain.tm) * ((p.N + plain.tn - 1) / plain.tn);
  if (plain_tiles * 2 > p.cus || ksteps < 48) return false;
  const int stm = forced ? p.tile_m : 64, stn = forced ? p.tile_n : 64;
  const int64_t tiles = ((p.M + stm - 1) / stm) * ((p.N + stn - 1) / stn);
  const int64_t want = std::min<int64_t>({(int64_t)p.cus / tiles, (int64_t)kAutoMaxSplits, (int64_t)ksteps / 16, fit});
  if (want < 2) return false;
  splits = (int)want;
  tm = stm;
  tn = stn;
  return true;
}

}  // namespace

hipError_t launch(const Problem &p) {
  Args a;
  a.A = static_cast<const uint8_t *>(p.A);
  a.B = static_cast<const uint8_t *>(p.B);
  a.SA = static_cast<const uint8_t *>(p.scale_A);
  a.SB = static_cast<const uint8_t *>(p.scale_B);
  a.C = static_cast<uint8_t *>(p.C);
  a.M = (int)p.M;
  a.N = (int)p.N;
  a.K = (int)p.K;
  a.lda = (int)p.lda;
  a.ldb = (int)p.ldb;
  a.ldc = (int)p.ldc;
  a.ws = nullptr;
  a.splits = 1;
  a.kq = 0;
  const int slice = p.dt == Dt::kMxfp8 ? 128 : 64;
  a.ksteps = (int)((p.K + slice - 1) / slice);
  a.kb = (int)((p.K + 127) / 128);
  if (p.dt == Dt::kMxfp4) {
    // Rows of bytes (two elements each), 128-byte slices, a scale per 32.
    a.K = (int)(p.K / 2);
    a.ksteps = (a.K + kRowBytes - 1) / kRowBytes;
    a.kb = (int)((p.K + 31) / 32);
  }
  const bool fp6 = p.dt == Dt::kMxfp6E2M3 || p.dt == Dt::kMxfp6E3M2;
  if (fp6) {
    // Rows of bytes (four elements in three), a scale per 32; the K loop
    // counts 64-element steps (48 bytes; K % 64 == 0).
    a.K = (int)(p.K / 4 * 3);
    a.ksteps = (int)(p.K / 64);
    a.kb = (int)((p.K + 31) / 32);
  }
  const bool scaled = p.dt == Dt::kMxfp8 || p.dt == Dt::kMxfp4 || fp6;
  // MXFP8 with no ragged slice (128 elements each) takes the kernel whose
  // loads check no columns (2% fewer cycles).
  const bool whole = p.K > 0 && p.K % 128 == 0;
  int tm = p.tile_m, tn = p.tile_n;
  if ((p.dt == Dt::kBf16 || p.dt == Dt::kF16) && p.splits != 1 && p.ws != nullptr) {
    int splits = 0;
    if (choose_split(p, a.ksteps, tm, tn, splits)) {
      // Whole slices per split, and no split left empty.
      a.kq = (a.ksteps + splits - 1) / splits;
      a.splits = (a.ksteps + a.kq - 1) / a.kq;
      a.ws = static_cast<float *>(p.ws);
      return p.dt == Dt::kBf16 ? launch_split_dt<kBf16>(p, a, tm, tn) : launch_split_dt<kF16>(p, a, tm, tn);
    }
  }
  if (tm == 0) {
    const Shape s = scaled             ? Shape{256, 256, 1.0}
                    : p.trans_b        ? pick_shape(kShapesBK, p.M, p.N, p.cus)
                                       : pick_shape(kShapesBN, p.M, p.N, p.cus);
    tm = s.tm;
    tn = s.tn;
  }
  switch (p.dt) {
    case Dt::kBf16:
      return launch_dt<kBf16>(p, a, tm, tn);
    case Dt::kF16:
      return launch_dt<kF16>(p, a, tm, tn);
    case Dt::kMxfp8:
      if (tm == 256 && tn == 256 && !p.trans_a && p.trans_b)
        return whole ? launch_shape<Traits<kFp8, true, true, true>, 256, 256>(p, a)
                     : launch_shape<Traits<kFp8, true, true>, 256, 256>(p, a);
      break;
    case Dt::kMxfp4:
      if (tm == 256 && tn == 256 && !p.trans_a && p.trans_b)
        return p.K > 0 && p.K % 256 == 0 && (((uintptr_t)a.SA | (uintptr_t)a.SB) & 3) == 0
                   ? launch_shape<Traits<kFp4, true, true, true>, 256, 256>(p, a)
                   : launch_shape<Traits<kFp4, true, true>, 256, 256>(p, a);
      break;
    case Dt::kMxfp6E2M3:
      if (tm == 256 && tn == 256 && !p.trans_a && p.trans_b)
        return launch_shape<Traits<kFp6E2M3, true, true>, 256, 256>(p, a);
      break;
    case Dt::kMxfp6E3M2:
      if (tm == 256 && tn == 256 && !p.trans_a && p.trans_b)
        return launch_shape<Traits<kFp6E3M2, true, true>, 256, 256>(p, a);
      break;
  }
  return hipErrorInvalidValue;
}

bool shape_supported(const Problem &p, int tile_m, int tile_n) {
  if (p.dt != Dt::kBf16 && p.dt != Dt::kF16) return tile_m == 256 && tile_n == 256;
  if (p.splits >= 2) return (tile_m == 128 && tile_n == 128) || (tile_m == 64 && tile_n == 64);
  return (tile_m == 256 && tile_n == 256) || (tile_m == 128 && tile_n == 128) || (tile_m == 64 && tile_n == 64) ||
         (tile_m == 256 && tile_n == 192 && p.trans_b);
}

}  // namespace tgemm
