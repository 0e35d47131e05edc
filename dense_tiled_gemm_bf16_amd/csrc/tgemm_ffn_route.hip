// Routing to experts for gfx950: the choice of experts with its gradient, and
// the plan that sorts the choices by expert.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tgemm_ffn_math.hpp"

namespace tgemm {
namespace ffn {
namespace {

constexpr float kInf = __builtin_inff();
enum Score : int { kSoftmax = 0, kSigmoid = 1 };

// Logits of type DT (2: binary32) as binary32; NaN reads as -inf (masked).
template <int DT>
__device__ __forceinline__ float load_logit(const void *p, size_t i) {
  float x;
  if constexpr (DT == 2)
    x = ((const float *)p)[i];
  else
    x = to_f32<DT>(((const uint16_t *)p)[i]);
  return x == x ? x : -kInf;
}

// The row's V logits of lane l (experts l, l + L, ...; -inf past the last),
// loaded without a branch between them so that all are in flight at once.
template <int DT, int L, int V>
__device__ __forceinline__ void load_row(const void *p, size_t row, int E, int l, float (&x)[V]) {
  using Raw = typename std::conditional<DT == 2, float, uint16_t>::type;
  Raw raw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) raw[v] = ((const Raw *)p)[row + min(v * L + l, E - 1)];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f;
    if constexpr (DT == 2)
      f = raw[v];
    else
      f = to_f32<DT>(raw[v]);
    x[v] = v * L + l < E && f == f ? f : -kInf;
  }
}

// exp(x - m) for x <= m, of the largest of a row; 1 where both are infinite.
__device__ __forceinline__ float exp_below(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// Lane l's value from the lane D further on in its row of 16 (cyclic).
template <int D>
__device__ __forceinline__ int row_turn(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + D, 0xf, 0xf, false);
}
// All lanes of L (16 or 64) combined, in every lane; op commutes, so that all
// lanes get the same bits.
template <int L, class V, class Op>
__device__ __forceinline__ V all_l(V v, Op op) {
  static_assert(sizeof(V) == 4 && (L == 16 || L == 64), "one register, whole rows");
  v = op(v, __builtin_bit_cast(V, row_turn<8>(__builtin_bit_cast(int, v))));
  v = op(v, __builtin_bit_cast(V, row_turn<4>(__builtin_bit_cast(int, v))));
  v = op(v, __builtin_bit_cast(V, row_turn<2>(__builtin_bit_cast(int, v))));
  v = op(v, __builtin_bit_cast(V, row_turn<1>(__builtin_bit_cast(int, v))));
  if constexpr (L == 64) {
    v = op(v, __shfl_xor(v, 16, 64));
    v = op(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float max_l(float v) {
  return all_l<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float sum_l(float v) {
  return all_l<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ uint32_t umax_l(uint32_t v) {
  return all_l<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// ---------------------------------------------------------------------------
// The choice.  A token takes L lanes of a wave, lane l the experts l, l + L,
// ...: V of them, held in registers.
//
// The keys are compared as 64-bit arithmetic gives them, but nearly always
// 32 bits settle that, so the work is done on whole numbers that hold a
// rounded key above the expert's index (31 bits in all; higher is better, so
// the index is kept as its distance from the last): the next best below
// `cur` is cur + max(v - cur) in wrapping unsigned arithmetic, which takes
// one subtraction and half a three-way maximum a value, with nothing to
// remove, and four row turns to join 16 lanes.  What the rounded keys leave
// open -- two keys in a row closer than their errors, or two groups at the
// cut -- sends the token through exact_choice.
//  * 16-bit logits without a bias: the logit's own 16 bits in order; exact.
//  * otherwise a key's place between the row's largest and least (at most
//    kWindow below) in 31 - index bits; without a bias the logit itself,
//    whose places are in order (only equal ones are open); with one the
//    score + bias in 32 bits, off by at most kKeyError times max(1, |key|):
//    2^-21 for a sigmoid (its exponential, sum and reciprocal, slopes below
//    1, and the bias's sum: 5 half steps), 2^-19 for a softmax (also the
//    row's sum of up to 1024: 30 half steps).
// Measured at 32768 tokens, 256 binary32 logits, 8 groups, 8 choices of
// biased sigmoids: 57 us with every key in 64 bits.
// ---------------------------------------------------------------------------
struct TopkArgs {
  const void *logits;
  const float *bias;
  float *weights;
  int32_t *ids;
  int T, E, ld, k, groups, used, per, renorm;
  int shift;           // 2^shift lanes of a token share a group's scan
  uint32_t per_magic;  // expert -> group: __umulhi(e, per_magic)
  float scale;
};

__device__ __forceinline__ int group_of(const TopkArgs &a, int e) {
  return (int)(a.per == 1 ? (uint32_t)e : __umulhi((uint32_t)e, a.per_magic));
}

// Place of expert e in a token's LDS row (its 32 runs start on other banks).
__device__ __forceinline__ constexpr int skewed(int e) { return e + (e >> 5); }

// Two largest of the keys of each group, by 2^shift lanes a group: lane l
// works for group l >> shift.  Valid where that is below a.groups.
template <int L, class Key>
__device__ __forceinline__ Key group_score(const TopkArgs &a, const Key *keys, int l, int shift) {
  const Key none = -(Key)kInf;
  Key best = none, second = none;
  const int share = 1 << shift, g = min(l >> shift, a.groups - 1), i0 = l & (share - 1);
  for (int i = i0; i < a.per; i += 8 * share) {
    Key s[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) s[u] = keys[skewed(g * a.per + min(i + u * share, a.per - 1))];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const Key w = i + u * share < a.per ? s[u] : none;
      second = w < best ? (w > second ? w : second) : best;
      best = w > best ? w : best;
    }
  }
  for (int d = 1; d < share; d <<= 1) {
    const Key ob = __shfl_xor(best, d, L), os = __shfl_xor(second, d, L);
    const Key low = ob < best ? ob : best;
    best = ob > best ? ob : best;
    second = os > second ? os : second;
    second = low > second ? low : second;
  }
  return second == none ? best : best + second;
}

// Orders LDS traffic between a wave's lanes for the compiler (the hardware
// keeps a wave's LDS operations in order).
__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }

// The k choices with every key in 64 bits; lane j returns the j-th (-1: none).
// All L lanes of a token come here together; keys: the token's LDS row.
template <int L, int V, int SCORE, bool BIAS>
__device__ __forceinline__ int exact_choice(const TopkArgs &a, const float (&x)[V], float m, double *keys, int l) {
  double key[V];
  const double none = -(double)kInf;
  double z = 0.0;
  const bool scores = BIAS || a.groups > 1;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!scores) {
      key[v] = 0.0;
    } else if constexpr (SCORE == kSoftmax) {
      key[v] = x[v] == -kInf ? 0.0 : x[v] == m ? 1.0 : exp((double)x[v] - (double)m);
      z += key[v];
    } else {
      key[v] = 1.0 / (1.0 + exp(-(double)x[v]));
    }
  }
  if constexpr (SCORE == kSoftmax)
#pragma unroll
    for (int d = 1; d < L; d <<= 1) z += __shfl_xor(z, d, L);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    if constexpr (SCORE == kSoftmax)
      if (scores) key[v] /= z;
    if constexpr (BIAS)
      if (e < a.E) key[v] += (double)a.bias[e];
    if (x[v] == -kInf || !(key[v] == key[v])) key[v] = none;
  }
  if (a.groups > 1) {
    lds_order();
#pragma unroll
    for (int v = 0; v < V; ++v) keys[skewed(v * L + l)] = key[v];
    lds_order();
    const double score = group_score<L>(a, keys, l, 0);
    int above = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(score, g, L);
      above += o > score || (o == score && g < l);
    }
    const uint64_t all = __ballot(l < a.groups && above < a.used);
    const uint64_t mask = L == 64 ? all : (all >> ((threadIdx.x & 63) / L * L)) & ((1ull << (L & 63)) - 1);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!((mask >> (group_of(a, v * L + l) & 63)) & 1)) key[v] = none;
  }
  // Without a bias the score only grows with the logit: ties of scores that
  // 64 bits no longer tell apart go by the logit.
  if constexpr (!BIAS)
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key[v] == none ? none : (double)x[v];
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    double best = none;
    int at = 0x7fffffff;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v * L + l;
      }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) {
      const double ob = __shfl_xor(best, d, L);
      const int oa = __shfl_xor(at, d, L);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (l == j) mine = at == 0x7fffffff ? -1 : at;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at == v * L + l) key[v] = none;
  }
  return mine;
}

template <int DT, int L, int V, int SCORE, bool BIAS>
__global__ __launch_bounds__(256) void topk_kernel(const TopkArgs a) {
  constexpr int kTok = 256 / L, kE = L * V;
  constexpr int kIdx = kE <= 256 ? 8 : kE <= 512 ? 9 : 10;  // bits of an index
  constexpr uint32_t kLow = (1u << kIdx) - 1;
  constexpr bool kRaw16 = DT != 2 && !BIAS;
  constexpr float kWindow = BIAS ? 4.0f : 32.0f;
  // Of a key, relative to max(1, |key|).
  constexpr float kKeyError = SCORE == kSoftmax ? 0x1p-19f : 0x1p-21f;
  constexpr float kPlaces = (float)((1 << (31 - kIdx)) - 64);
  __shared__ double lds[kTok][skewed(kE - 1) + 1];
  const int l = threadIdx.x & (L - 1), tok = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * kTok + tok;
  const bool live = t < a.T;  // (the lanes of a dead token go along)
  const size_t row = (size_t)(live ? t : 0) * a.ld;

  float x[V], bias[BIAS ? V : 1];
  if constexpr (BIAS)
#pragma unroll
    for (int v = 0; v < V; ++v) bias[v] = a.bias[min(v * L + l, a.E - 1)];
  load_row<DT, L>(a.logits, row, a.E, l, x);
  // The row's largest logit and the softmax's sum, when something needs them.
  const bool scores = BIAS || a.groups > 1;
  const bool whole = SCORE == kSoftmax && (scores || !a.renorm);
  float m = -kInf, z = 1.0f;
  if (whole) {
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
    m = max_l<L>(m);
  }
  float key[V];  // scores + bias (-inf: cannot be chosen)
  if (whole) {
    z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] = x[v] == -kInf ? 0.0f : exp_below(x[v], m);
      z += key[v];
    }
    z = sum_l<L>(z);
  }
  if (scores) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (SCORE == kSoftmax)
        key[v] *= 1.0f / z;
      else
        key[v] = sigmoid_(x[v]);
      if constexpr (BIAS) key[v] += bias[v];
      if (x[v] == -kInf || !(key[v] == key[v])) key[v] = -kInf;
    }
  }
  bool open = false;  // the token needs exact_choice

  // Groups: x is masked where its group is dropped.
  float y[V];
#pragma unroll
  for (int v = 0; v < V; ++v) y[v] = BIAS ? key[v] : x[v];
  if (a.groups > 1) {
    float *keys = (float *)lds[tok];
#pragma unroll
    for (int v = 0; v < V; ++v) keys[skewed(v * L + l)] = key[v];
    lds_order();
    const float score = group_score<L>(a, keys, l, a.shift);
    const int g0 = l >> a.shift;
    int above = 0;
    for (int g = 0; g < a.groups; g += 8) {
      float o[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) o[u] = __shfl(score, ((g + u) << a.shift) & (L - 1), L);
#pragma unroll
      for (int u = 0; u < 8; ++u) above += g + u < a.groups && (o[u] > score || (o[u] == score && g + u < g0));
    }
    const bool is = g0 < a.groups, keep = is && above < a.used;
    // The worst that stays against the best that goes.
    const float worst = -max_l<L>(keep ? -score : -kInf), best = max_l<L>(is && !keep ? score : -kInf);
    float most = 1.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) most = fmaxf(most, key[v] == -kInf ? 0.0f : fabsf(key[v]));
    const float err = 2.0f * kKeyError * max_l<L>(most) * 1.01f;
    open = best != -kInf && !(worst - best > 2.0f * err);
    const uint64_t all = __ballot(keep && l == g0 << a.shift);
    const uint64_t mask = L == 64 ? all : (all >> ((threadIdx.x & 63) / L * L)) & ((1ull << (L & 63)) - 1);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!((mask >> ((group_of(a, v * L + l) << a.shift) & 63)) & 1)) y[v] = -kInf;
  }

  // Keys over indices.
  uint32_t q[V];
  uint32_t gap = 1u << kIdx;  // two keys in a row this far apart are in order
  if constexpr (kRaw16) {
    gap = 0;  // equal logits are ties: the index settles them
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float w = y[v] + 0.0f;  // (-0 ties with 0)
      const uint32_t f = __builtin_bit_cast(uint32_t, w);
      // A bf16 or fp16 value in order: its binary32 bits, 16 of them (fp16:
      // 19 hold its sign, exponent and fraction).
      constexpr int kDrop = DT == 0 ? 16 : 13;
      const uint32_t o = ((int32_t)f < 0 ? ~f : f | 0x80000000u) >> kDrop;
      q[v] = y[v] == -kInf ? 0u : ((o + 1) << kIdx) | (kLow - (uint32_t)(v * L + l));
    }
  } else {
    float hi = -kInf, lo = kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hi = fmaxf(hi, y[v]);
      lo = y[v] == -kInf ? lo : fminf(lo, y[v]);
    }
    hi = max_l<L>(hi);
    lo = fmaxf(-max_l<L>(-lo), hi - kWindow);
    const float span = hi - lo;
    const float per = span > 0.0f ? kPlaces / span : 0.0f;
    // (An infinite or empty span has no places: what is chosen is then open.)
    open = open || (hi != -kInf && !(span > 0.0f && span <= kWindow));
    if constexpr (BIAS) {
      // (4: the place's own two roundings and its and this line's cut.)
      const float err = kKeyError * fmaxf(1.0f, fmaxf(fabsf(hi), fabsf(lo)));
      gap = ((uint32_t)fminf(2.0f * err * per, 1e6f) + 4u) << kIdx;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t place = (uint32_t)(fmaxf(y[v] - lo, 0.0f) * per);
      q[v] = y[v] == -kInf ? 0u : ((place + 1) << kIdx) | (kLow - (uint32_t)(v * L + l));
    }
  }
  int mine = -1;
  uint32_t cur = 0x7fffffffu;
  for (int j = 0; j <= a.k; ++j) {
    uint32_t next = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t d = q[v] - cur;
      next = d > next ? d : next;
    }
    next = umax_l<L>(next) + cur;
    next = cur == 0 ? 0 : next;  // none are left
    if (j > 0 && next != 0) open = open || (cur | kLow) - (next | kLow) < gap;
    if (l == j && j < a.k) mine = next == 0 ? -1 : (int)(kLow - (next & kLow));
    cur = next;
  }
  if (!kRaw16 || a.groups > 1)
    if (open) mine = exact_choice<L, V, SCORE, BIAS>(a, x, m, lds[tok], l);

  // Lane j: its choice's score and weight.
  float s = 0.0f, w;
  const float xs = mine >= 0 ? load_logit<DT>(a.logits, row + mine) : -kInf;
  if constexpr (SCORE == kSoftmax) {
    const float mm = a.renorm ? max_l<L>(xs) : m;
    s = mine >= 0 ? exp_below(xs, mm) : 0.0f;
    w = a.renorm ? s / (sum_l<L>(s) + 1e-20f) : s / z;
  } else {
    s = mine >= 0 ? 1.0f / (1.0f + expf(-xs)) : 0.0f;
    w = a.renorm ? s / (sum_l<L>(s) + 1e-20f) : s;
  }
  if (live && l < a.k) {
    a.weights[(size_t)t * a.k + l] = mine >= 0 ? w * a.scale : 0.0f;
    a.ids[(size_t)t * a.k + l] = mine;
  }
}

template <int DT, int L, int V>
hipError_t launch_topk_lv(const Topk &t) {
  TopkArgs a{t.logits, t.bias, t.weights, t.ids, (int)t.T, (int)t.E, (int)t.ld, t.k, t.groups, t.used,
             (int)(t.E / t.groups), t.renorm, 0, 0, t.scale};
  while ((t.groups << (a.shift + 1)) <= L) ++a.shift;
  // ceil(2^32 / per): exact quotients for experts below 2^16 (not for per = 1).
  a.per_magic = a.per > 1 ? (uint32_t)((0x100000000ull + (uint64_t)a.per - 1) / (uint64_t)a.per) : 0u;
  const bool bias = t.bias != nullptr;
  const int64_t wgs = (t.T + 256 / L - 1) / (256 / L);
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  const void *fn =
      t.score == kSoftmax ? (bias ? reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSoftmax, true>)
                                   : reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSoftmax, false>))
                          : (bias ? reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSigmoid, true>)
                                   : reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSigmoid, false>));
  void *args[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(256), args, 0, t.stream);
}

template <int DT>
hipError_t launch_topk_dt(const Topk &t) {
  // 16 lanes a token while they hold the experts, the choices and the groups.
  if (t.E <= 256 && t.k <= 16 && t.groups <= 16) {
    if (t.E <= 64) return launch_topk_lv<DT, 16, 4>(t);
    if (t.E <= 128) return launch_topk_lv<DT, 16, 8>(t);
    return launch_topk_lv<DT, 16, 16>(t);
  }
  if (t.E <= 512) return launch_topk_lv<DT, 64, 8>(t);
  return launch_topk_lv<DT, 64, 16>(t);
}

// ---------------------------------------------------------------------------
// Gradient.  With p the softmax or sigmoid of the row and g the weights'
// gradients (times scale), S the chosen scores' sum:
//   softmax, renormalised:  dx_j = v_j (g_j - sum v g), v the softmax over the chosen
//   softmax:                dx_e = p_e ([e chosen] g_e - sum over the chosen p g)
//   sigmoid, renormalised:  dx_j = (1 - s_j) v_j (g_j - sum v g), v = s / S
//   sigmoid:                dx_j = g_j s_j (1 - s_j)
// and 0 for experts not chosen, except the second.  Lane j works out choice
// j; the choices meet the row in LDS.
// ---------------------------------------------------------------------------
struct TopkGradArgs {
  const void *logits;
  const int32_t *ids;
  const float *dw;
  void *out;
  int T, E, ld, ldo, k, renorm;
  float scale;
};

template <int DT, int L, int V, int SCORE>
__global__ __launch_bounds__(256) void topk_grad_kernel(const TopkGradArgs a) {
  constexpr int kTok = 256 / L;
  __shared__ float add[kTok][L * V];
  const int l = threadIdx.x & (L - 1), tok = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * kTok + tok;
  const bool live = t < a.T;
  const size_t tt = (size_t)(live ? t : 0), row = tt * a.ld;
#pragma unroll
  for (int v = 0; v < V; ++v) add[tok][v * L + l] = 0.0f;
  int id = -1;
  float g = 0.0f;
  if (l < a.k) {
    id = a.ids[tt * a.k + l];
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0) g = a.dw[tt * a.k + l] * a.scale;
  }
  const float xs = id >= 0 ? load_logit<DT>(a.logits, row + id) : -kInf;
  const bool dense = SCORE == kSoftmax && !a.renorm;
  float d = 0.0f, base = 0.0f, m = -kInf, z = 1.0f;
  float x[V];
  if (dense) {
    load_row<DT, L>(a.logits, row, a.E, l, x);
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
    m = max_l<L>(m);
    z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = x[v] == -kInf ? 0.0f : exp_below(x[v], m);
      z += x[v];
    }
    z = sum_l<L>(z);
    if (z == 0.0f) z = 1.0f;  // every logit masked
    const float p = id >= 0 && xs != -kInf ? exp_below(xs, m) / z : 0.0f;
    d = p * g;
    base = sum_l<L>(d);
  } else if constexpr (SCORE == kSoftmax) {
    m = max_l<L>(xs);
    const float s = id >= 0 && xs != -kInf ? exp_below(xs, m) : 0.0f;
    const float v = s / (sum_l<L>(s) + 1e-20f);
    d = v * (g - sum_l<L>(v * g));
  } else {
    const float s = id >= 0 ? 1.0f / (1.0f + expf(-xs)) : 0.0f;
    // 1 - s without its cancellation.
    const float c = id >= 0 ? 1.0f / (1.0f + expf(xs)) : 0.0f;
    if (a.renorm) {
      const float v = s / (sum_l<L>(s) + 1e-20f);
      d = c * v * (g - sum_l<L>(v * g));
    } else {
      d = g * s * c;
    }
  }
  __syncthreads();
  if (id >= 0) add[tok][id] = d;
  __syncthreads();
  if (!live) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    if (e >= a.E) continue;
    float o = add[tok][e];
    if (dense) o -= x[v] / z * base;
    const size_t at = tt * a.ldo + e;
    if constexpr (DT == 2)
      ((float *)a.out)[at] = o;
    else
      ((uint16_t *)a.out)[at] = (uint16_t)(pack2<DT>(o, 0.0f) & 0xffffu);
  }
}

template <int DT, int L, int V>
hipError_t launch_grad_lv(const TopkGrad &t) {
  TopkGradArgs a{t.logits, t.ids, t.dweights, t.dlogits, (int)t.T, (int)t.E, (int)t.ld, (int)t.ldo, t.k, t.renorm,
                 t.scale};
  const int64_t wgs = (t.T + 256 / L - 1) / (256 / L);
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  const void *fn = t.score == kSoftmax ? reinterpret_cast<const void *>(&topk_grad_kernel<DT, L, V, kSoftmax>)
                                       : reinterpret_cast<const void *>(&topk_grad_kernel<DT, L, V, kSigmoid>);
  void *args[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(256), args, 0, t.stream);
}

template <int DT>
hipError_t launch_grad_dt(const TopkGrad &t) {
  if (t.E <= 256 && t.k <= 16) {
    if (t.E <= 64) return launch_grad_lv<DT, 16, 4>(t);
    if (t.E <= 128) return launch_grad_lv<DT, 16, 8>(t);
    return launch_grad_lv<DT, 16, 16>(t);
  }
  if (t.E <= 512) return launch_grad_lv<DT, 64, 8>(t);
  return launch_grad_lv<DT, 64, 16>(t);
}

// ---------------------------------------------------------------------------
// Plan: a stable counting sort of the T k choices by expert.  A workgroup
// takes kPlanChunk choices in order, wave w a run of them.  Whole numbers
// only, so the order of the counting does not matter; the placing goes in
// order: a choice's row is its expert's first row + the choices of the
// expert in chunks before + in waves before + in the wave before it.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64, kPlanPer = kPlanChunk / kPlanWaves;

struct PlanArgs {
  const int32_t *ids;
  int32_t *offsets, *rows, *slots, *hist;
  int n, E, k, chunks;
};

__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(const PlanArgs a) {
  __shared__ int32_t counts[kPlanThreads];
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) counts[e] = 0;
  __syncthreads();
  const int first = (int)blockIdx.x * kPlanChunk;
#pragma unroll
  for (int i = 0; i < kPlanChunk / kPlanThreads; ++i) {
    const int c = first + i * kPlanThreads + (int)threadIdx.x;
    const int id = c < a.n ? a.ids[c] : -1;
    if (id >= 0 && id < a.E) atomicAdd(&counts[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) a.hist[(size_t)blockIdx.x * a.E + e] = counts[e];
}

// One thread an expert (E <= kPlanThreads) for the offsets.
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(const PlanArgs a) {
  __shared__ int32_t cnt[kPlanWaves * kPlanThreads];  // [wave][expert], then rows
  __shared__ int32_t scan[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = (int)blockIdx.x * kPlanChunk;
  for (int i = tid; i < kPlanWaves * a.E; i += kPlanThreads) cnt[i] = 0;
  __syncthreads();
  int id[kPlanPer / 64];
#pragma unroll
  for (int i = 0; i < kPlanPer / 64; ++i) {
    const int c = first + wave * kPlanPer + i * 64 + lane;
    id[i] = c < a.n ? a.ids[c] : -1;
    if (id[i] < 0 || id[i] >= a.E) id[i] = -1;
    if (id[i] >= 0) atomicAdd(&cnt[wave * a.E + id[i]], 1);
  }
  __syncthreads();
  // Totals of this thread's expert: in the chunks before, and in all.
  int before = 0, total = 0;
  if (tid < a.E) {
    if (a.chunks > 1) {
#pragma unroll 8
      for (int c = 0; c < a.chunks; ++c) {
        const int h = a.hist[(size_t)c * a.E + tid];
        total += h;
        before += c < (int)blockIdx.x ? h : 0;
      }
    } else {
      for (int w = 0; w < kPlanWaves; ++w) total += cnt[w * a.E + tid];
    }
  }
  int upto = wave_scan(total, lane);
  if (lane == 63) scan[wave] = upto;
  __syncthreads();
  int all = 0;
  for (int w = 0; w < kPlanWaves; ++w) {
    if (w < wave) upto += scan[w];
    all += scan[w];
  }
  if (tid < a.E) {
    int at = upto - total;
    if (blockIdx.x == 0) {
      a.offsets[tid] = at;
      if (tid == a.E - 1) a.offsets[a.E] = upto;
    }
    at += before;
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = cnt[w * a.E + tid];
      cnt[w * a.E + tid] = at;
      at += c;
    }
  }
  __syncthreads();
  int bits = 0;
  while ((1 << bits) < a.E) ++bits;
#pragma unroll
  for (int i = 0; i < kPlanPer / 64; ++i) {
    const int c = first + wave * kPlanPer + i * 64 + lane;
    // The lanes with this lane's expert.
    uint64_t same = __ballot(id[i] >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((id[i] >> b) & 1);
      same &= (id[i] >> b) & 1 ? set : ~set;
    }
    int at = -1;
    if (id[i] >= 0) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      int32_t *p = &cnt[wave * a.E + id[i]];
      at = *p + rank;
      // (A wave's LDS operations stay in order: its lanes have read.)
      asm volatile("" ::: "memory");
      if (rank == 0) *p = at + __popcll(same);
      asm volatile("" ::: "memory");
      a.rows[at] = c / a.k;
    }
    if (c < a.n) {
      a.slots[c] = at;
      // Rows behind the last: no token.
      if (c >= all) a.rows[c] = -1;
    }
  }
}

}  // namespace

hipError_t launch_topk(const Topk &t) {
  if (t.dtype == 0) return launch_topk_dt<0>(t);
  if (t.dtype == 1) return launch_topk_dt<1>(t);
  return launch_topk_dt<2>(t);
}

hipError_t launch_topk_grad(const TopkGrad &t) {
  if (t.dtype == 0) return launch_grad_dt<0>(t);
  if (t.dtype == 1) return launch_grad_dt<1>(t);
  return launch_grad_dt<2>(t);
}

hipError_t launch_plan(const Plan &p) {
  PlanArgs a{p.ids, p.offsets, p.rows, p.slots, p.ws, (int)(p.T * p.k), (int)p.E, p.k, 1};
  a.chunks = (a.n + kPlanChunk - 1) / kPlanChunk;
  if (a.chunks < 1) a.chunks = 1;
  void *args[] = {&a};
  if (a.chunks > 1) {
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&plan_count_kernel), dim3((unsigned)a.chunks),
                                         dim3(kPlanThreads), args, 0, p.stream);
    if (e != hipSuccess) return e;
  }
  return hipLaunchKernel(reinterpret_cast<const void *>(&plan_place_kernel), dim3((unsigned)a.chunks),
                         dim3(kPlanThreads), args, 0, p.stream);
}

}  // namespace ffn
}  // namespace tgemm
