// Device helpers of the feed-forward kernels: activations with their
// derivatives in binary32, 16-bit vectors, and the walk over row groups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm_ffn_internal.hpp"

namespace tgemm {
namespace ffn {
namespace {

typedef __attribute__((ext_vector_type(4))) float v4f;
typedef __attribute__((ext_vector_type(4))) uint32_t v4u;
typedef __attribute__((ext_vector_type(2))) uint32_t v2u;
typedef __attribute__((ext_vector_type(2))) float v2f;
typedef __attribute__((ext_vector_type(2))) __bf16 v2bf;
typedef __attribute__((ext_vector_type(2))) _Float16 v2h;

// The element types of 16-bit tensors: 0 bf16, 1 fp16.
template <int DT>
__device__ __forceinline__ float to_f32(uint32_t bits16) {
  if constexpr (DT == 1)
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
  else
    return __builtin_bit_cast(float, bits16 << 16);
}
template <int DT>
__device__ __forceinline__ void unpack2(uint32_t w, float *v) {
  v[0] = to_f32<DT>(w & 0xffffu);
  v[1] = to_f32<DT>(w >> 16);
}
// Two values rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const v2f v = {a, b};
  if constexpr (DT == 1)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2h));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));
}
template <int DT>
__device__ __forceinline__ void unpack8(const v4u &w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2<DT>(w[i], v + 2 * i);
}
template <int DT>
__device__ __forceinline__ v4u pack8(const float (&v)[8]) {
  v4u w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
  return w;
}

// exp(x): its argument is rounded to binary32, so that the relative error grows
// with it: |x| 2^-24, 2^-17.6 where the result leaves binary32's range.
__device__ __forceinline__ float exp_(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f); }

// Upper tail of the normal distribution over its density's shape: for x >= 0,
// (1 - Phi(x)) exp(x^2 / 2) = t p(t) with t = 1 / (1 + x / 5); p is this
// project's own least-maximum fit of the left side's values on [0, 14],
// within 1.7e-6 of them, relatively, in binary32 (past 14 the tail is below
// 1e-44).
__device__ __forceinline__ float tail_shape(float x) {
  const float t = __builtin_amdgcn_rcpf(1.0f + 0.2f * x);
  float p = 0.27909741570705704f;
  p = fmaf(p, t, -0.3868376091974559f);
  p = fmaf(p, t, 0.44695617060760665f);
  p = fmaf(p, t, -0.12319883483718998f);
  p = fmaf(p, t, 0.13254210635479885f);
  p = fmaf(p, t, 0.0710911050271966f);
  p = fmaf(p, t, 0.08035027360384696f);
  return p * t;
}

__device__ __forceinline__ float sigmoid_(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_(-z)); }

// Scales of exponents are folded into their polynomials: each instruction a value
// is 0.9 us of a 4096 x 4096 output's epilogue.
// exp(-z^2 / 2), within z^2 2^-24 of it, relatively (two roundings of z^2 / 2).
__device__ __forceinline__ float bell(float z) { return __builtin_amdgcn_exp2f(z * -0.72134752044448170368f * z); }
// sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3); zz = z^2.
__device__ __forceinline__ float tanh_gate(float z, float zz) {
  constexpr float c = (float)(-1.59576912160573071176 * 1.44269504088896340736);
  constexpr float c3 = (float)(-1.59576912160573071176 * 1.44269504088896340736 * 0.044715);
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * fmaf(c3, zz, c)));
}

// act(z) of the activation ACT (the gated ones': of their gate).
template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == kRelu) {
    return z < 0.0f ? 0.0f : z;  // (NaN stays)
  } else if constexpr (ACT == kGelu || ACT == kGeglu) {
    const float q = bell(z) * tail_shape(fabsf(z));
    return z * (z < 0.0f ? q : 1.0f - q);
  } else if constexpr (ACT == kGeluTanh) {
    // z (1 + tanh u) / 2 = z sigmoid(2 u).
    return z * tanh_gate(z, z * z);
  } else if constexpr (ACT == kSilu || ACT == kSwiglu) {
    return z * sigmoid_(z);
  } else {
    return z;
  }
}

// act(z) and act'(z).
template <int ACT>
__device__ __forceinline__ void act_both(float z, float &f, float &d) {
  if constexpr (ACT == kRelu) {
    f = act_fwd<kRelu>(z);
    d = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  } else if constexpr (ACT == kGelu || ACT == kGeglu) {
    const float e = bell(z);
    const float q = e * tail_shape(fabsf(z));
    const float cdf = z < 0.0f ? q : 1.0f - q;
    f = z * cdf;
    d = fmaf(z * 0.3989422804014327f, e, cdf);
  } else if constexpr (ACT == kGeluTanh) {
    const float zz = z * z;
    const float s = tanh_gate(z, zz);
    f = z * s;
    // (Past |z| = 100 the derivative is 0 or 1; z^2 could overflow.)
    d = fmaf(f * (1.0f - s), 1.5957691216057308f * fmaf(0.134145f, fminf(zz, 1e4f), 1.0f), s);
  } else if constexpr (ACT == kSilu || ACT == kSwiglu) {
    const float s = sigmoid_(z);
    f = z * s;
    d = fmaf(f, 1.0f - s, s);
  } else {
    f = z;
    d = 1.0f;
  }
}

// Calls f(std::integral_constant<int, act>) for the (wave-uniform) act; the
// gated ones or the others.
template <int V>
struct Int {
  static constexpr int value = V;
};
template <bool GATED, class F>
__device__ __forceinline__ void with_act(int act, F f) {
  if constexpr (GATED) {
    if (act == kSwiglu) f(Int<kSwiglu>());
    else f(Int<kGeglu>());
  } else {
    switch (act) {
      case kRelu: f(Int<kRelu>()); break;
      case kGelu: f(Int<kGelu>()); break;
      case kGeluTanh: f(Int<kGeluTanh>()); break;
      case kSilu: f(Int<kSilu>()); break;
      default: f(Int<kNone>()); break;
    }
  }
}

// Row groups: group e holds rows [offsets[e], offsets[e + 1]) of R.  The
// offsets come from device memory, so they are clamped: whatever they hold,
// no row outside [0, R) is touched, and no more than `most` blocks are
// counted in all.
struct Range {
  int lo, hi;
};
__device__ __forceinline__ Range group_rows(const int32_t *offsets, int e, int R) {
  const int lo = min(max(offsets[e], 0), R);
  return {lo, max(lo, min(offsets[e + 1], R))};
}

// Block `index` of the groups' rows, cut into blocks of `size` rows group by
// group, each block standing for `times` units: which group, its rows, the
// unit inside the group.  Every wave works it out for itself, 64 groups at a
// time.  total: units in all (index >= total: no such block, and e = -1).
struct Found {
  int e, lo, hi;
  int unit;    // index inside the group
  int before;  // units of the groups before
};
// Sums of lanes 0 .. l: inside rows of 16 lanes by row shifts (lanes shifted
// in read 0), then the rows' totals handed on (row_bcast 15 to rows 1 and 3,
// row_bcast 31 to rows 2 and 3).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}
// Lane l's group e0 + l (empty past the last).
__device__ __forceinline__ Range lane_rows(const int32_t *offsets, int groups, int R, int e) {
  if (e >= groups) return {0, 0};
  return group_rows(offsets, e, R);
}
// units(rows): of a group of so many rows (0 of none).
template <class F>
__device__ __forceinline__ int sum_units(const int32_t *offsets, int groups, int R, int lane, F units) {
  int sum = 0;
  for (int e0 = 0; e0 < groups; e0 += 64) {
    const Range r = lane_rows(offsets, groups, R, e0 + lane);
    sum += units(r.hi - r.lo);
  }
  return __builtin_amdgcn_readlane(wave_scan(sum), 63);
}
template <class F>
__device__ __forceinline__ Found find_in(const int32_t *offsets, int groups, int R, int index, int lane, F units) {
  int base = 0;
  for (int e0 = 0; e0 < groups; e0 += 64) {
    const Range r = lane_rows(offsets, groups, R, e0 + lane);
    const int n = units(r.hi - r.lo);
    const int upto = wave_scan(n);
    const uint64_t past = __ballot(index < base + upto);
    if (past) {
      const int l = (int)__builtin_ctzll(past);
      const int before = base + __builtin_amdgcn_readlane(upto - n, l);
      // (Only offsets that are no offsets can leave the unit outside the group.)
      if (index < before || e0 + l >= groups) return {-1, 0, 0, 0, 0};
      return {e0 + l, __builtin_amdgcn_readlane(r.lo, l), __builtin_amdgcn_readlane(r.hi, l), index - before, before};
    }
    base += __builtin_amdgcn_readlane(upto, 63);
  }
  return {-1, 0, 0, 0, base};
}

// Blocks of `size` rows, each `times` units.
__device__ __forceinline__ int total_units(const int32_t *offsets, int groups, int R, int size, int times, int lane) {
  return sum_units(offsets, groups, R, lane, [&](int n) { return (n + size - 1) / size * times; });
}
__device__ __forceinline__ Found find_unit(const int32_t *offsets, int groups, int R, int index, int size, int times,
                                           int lane) {
  return find_in(offsets, groups, R, index, lane, [&](int n) { return (n + size - 1) / size * times; });
}

}  // namespace
}  // namespace ffn
}  // namespace tgemm
