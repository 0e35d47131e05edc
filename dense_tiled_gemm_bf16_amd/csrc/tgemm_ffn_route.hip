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
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + D, 0xf, 0xf, true);
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
// the index is kept as its distance from the last).  The next best below
// `cur` is cur + max(v - cur) in wrapping unsigned arithmetic, which takes
// one subtraction and half a three-way maximum a value, with nothing to
// remove, and four row turns to join 16 lanes.  What the rounded keys leave
// open -- two keys in a row closer than their errors, or two groups at the
// cut -- sends the token through exact_choice.
//  * Without a bias the order is the logits': 16-bit ones hold their own bits
//    in order and leave nothing open; binary32 ones their place in the 32
//    below the row's largest, in 31 - index bits, where only equal places
//    are open.
//  * With one, a key's place between the least bias and the largest + 1:
//    place = score * per + (bias - least) * per.  The score is off by at
//    most kScoreError (sigmoid: exponential, sum and reciprocal, slopes below
//    a quarter for the first: 4 half steps; softmax: also the row's sum of up
//    to 1024, 40 half steps, where a bias is added to it), the second term by a place and the sum by half
//    a one; the place is cut to a whole number.
// Each value costs instructions in every token, and they bound the kernel: at
// 32768 tokens, 256 binary32 logits, 8 groups, 8 choices of biased sigmoids,
// all keys in 64 bits took 57 us, rounded keys with a lane-by-lane scan of
// the groups in LDS 34 us (1640 VALU instructions a wave of 4 tokens), groups
// as runs of registers 25 us (1235; 33.6 MB of logits, 1.4 TB/s).  8 tokens
// take 4.8 us, the way through one wave.  More than 256 experts take a whole
// wave a token: 8192 tokens of 384 in 8 groups 18.5 us, of 256 11.7.
// ---------------------------------------------------------------------------
struct TopkArgs {
  const void *logits;
  const float *bias;
  float *weights;
  int32_t *ids;
  int T, E, ld, k, groups, used, per, renorm;
  int picks;           // best keys to look at: k + 2, or k + 1
  int shift;           // 2^shift lanes of a token share a group's scan
  uint32_t ends;       // bit v: a group ends with the v-th experts of all lanes (0: groups are no such runs)
  uint32_t per_magic;  // expert -> group: __umulhi(e, per_magic)
  float scale;
};

__device__ __forceinline__ int group_of(const TopkArgs &a, int e) {
  return (int)(a.per == 1 ? (uint32_t)e : __umulhi((uint32_t)e, a.per_magic));
}

// Place of expert e in a token's LDS row (its 32 runs start on other banks).
__device__ __forceinline__ constexpr int skewed(int e) { return e + (e >> 5); }

// Score of group l (lanes past the last group: of the last) from its keys.
template <int L>
__device__ __forceinline__ double group_score(const TopkArgs &a, const double *keys, int l) {
  const double none = -(double)kInf;
  double best = none, second = none;
  const int g = min(l, a.groups - 1);
#pragma unroll 8
  for (int i = 0; i < a.per; ++i) {
    const double s = keys[skewed(g * a.per + i)];
    second = s < best ? (s > second ? s : second) : best;
    best = s > best ? s : best;
  }
  return second == none ? best : best + second;
}

// Two largest of the distinct whole numbers (0: none) of each group, by
// 2^shift lanes a group: lane l works for group l >> shift.  Valid where that
// is below a.groups.
template <int L>
__device__ __forceinline__ void group_top2(const TopkArgs &a, const uint32_t *keys, int l, int shift, uint32_t &best,
                                           uint32_t &second) {
  best = second = 0;
  const int share = 1 << shift, g = min(l >> shift, a.groups - 1), i0 = l & (share - 1);
  for (int i = i0; i < a.per; i += 8 * share) {
    uint32_t s[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) s[u] = keys[skewed(g * a.per + min(i + u * share, a.per - 1))];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t w = i + u * share < a.per ? s[u] : 0u;
      second = max(second, min(best, w));
      best = max(best, w);
    }
  }
  for (int d = 1; d < share; d <<= 1) {
    const uint32_t ob = __shfl_xor(best, d, L), os = __shfl_xor(second, d, L);
    second = max(max(second, os), min(best, ob));
    best = max(best, ob);
  }
}

// How many of the row's other 15 lanes hold more (distinct numbers).
template <int D = 1>
__device__ __forceinline__ int ranks_above(uint32_t v) {
  const int more = (uint32_t)row_turn<D>((int)v) > v;
  if constexpr (D == 15)
    return more;
  else
    return more + ranks_above<D + 1>(v);
}

// Orders LDS traffic between a wave's lanes for the compiler (the hardware
// keeps a wave's LDS operations in order).
__device__ __forceinline__ void lds_order() { asm volatile("" ::: "memory"); }

// Expert e's key in 64 bits from its logit x (m, z: the row's largest and the
// softmax's sum); -inf if it cannot be chosen.
template <int SCORE, bool BIAS>
__device__ __forceinline__ double exact_key(const TopkArgs &a, float x, int e, float m, double z) {
  double s;
  if constexpr (SCORE == kSoftmax)
    s = (x == m ? 1.0 : exp((double)x - (double)m)) / z;
  else
    s = 1.0 / (1.0 + exp(-(double)x));
  if constexpr (BIAS) s += (double)a.bias[e];
  return x == -kInf || !(s == s) ? -(double)kInf : s;
}
template <int L, int V>
__device__ __forceinline__ double exact_sum(const float (&x)[V], int rest, float m) {
  double z = 0.0;
#pragma unroll 2
  for (int v = 0; v < V; ++v)
    z += v * L < rest && x[v] > -kInf ? x[v] == m ? 1.0 : exp((double)x[v] - (double)m) : 0.0;
#pragma unroll
  for (int d = 1; d < L; d <<= 1) z += __shfl_xor(z, d, L);
  return z;
}

// The k choices with every key in 64 bits; lane j returns the j-th (-1: none).
// All L lanes of a token come here together; keys: the token's LDS row.  Few
// tokens do, so it keeps its keys in LDS and its loops rolled: what it does
// not hold in registers the kernel's usual path can.
template <int DT, int L, int SCORE, bool BIAS>
__device__ __forceinline__ int exact_choice(const TopkArgs &a, size_t row, float m, double z, double *keys, int l) {
  const double none = -(double)kInf;
  lds_order();
#pragma unroll 4
  for (int e = l; e < a.E; e += L) {
    const float x = load_logit<DT>(a.logits, row + e);
    // (Without a bias and groups the order is the logits'.)
    keys[skewed(e)] = BIAS || a.groups > 1 ? exact_key<SCORE, BIAS>(a, x, e, m, z) : (double)x;
  }
  if (a.groups > 1) {
    lds_order();
    const double score = group_score<L>(a, keys, l);
    lds_order();
    int above = 0;
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      const double o = __shfl(score, g, L);
      above += o > score || (o == score && g < l);
    }
    const uint64_t all = __ballot(l < a.groups && above < a.used);
    const uint64_t mask = L == 64 ? all : (all >> ((threadIdx.x & 63) / L * L)) & ((1ull << (L & 63)) - 1);
#pragma unroll 4
    for (int e = l; e < a.E; e += L) {
      const bool in = (mask >> (group_of(a, e) & 63)) & 1;
      if (!in)
        keys[skewed(e)] = none;
      else if constexpr (!BIAS)
        keys[skewed(e)] = load_logit<DT>(a.logits, row + e);
    }
  }
  int mine = -1;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = none;
    int at = 0x7fffffff;
#pragma unroll 8
    for (int e = l; e < a.E; e += L) {
      const double s = keys[skewed(e)];
      if (s > best) {
        best = s;
        at = e;
      }
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
    if (at != 0x7fffffff && at % L == l) keys[skewed(at)] = none;
  }
  lds_order();
  return mine;
}

// GROUPS: none, runs of whole v (a group is per / L experts of every lane), or
// any (asked at run time; for these a token takes the whole wave).
enum Grouping : int { kNoGroups = 0, kRuns = 1, kAnyGroups = 2 };
template <int DT, int L, int V, int SCORE, bool BIAS, int GROUPS>
__global__ __launch_bounds__(256, 4) void topk_kernel(const TopkArgs a) {
  static_assert(GROUPS != kAnyGroups || L == 64, "a lane for each of 64 groups");
  constexpr int kTok = 256 / L, kE = L * V;
  constexpr int kIdx = kE <= 256 ? 8 : kE <= 512 ? 9 : 10;  // bits of an index
  constexpr uint32_t kLow = (1u << kIdx) - 1, kOne = 1u << kIdx;
  constexpr bool kRaw16 = DT != 2 && !BIAS;
  constexpr float kPlaces = (float)((1 << (31 - kIdx)) - 64);
  constexpr bool kOverSum = SCORE == kSoftmax && BIAS;  // scores are divided by the row's sum
  constexpr float kScoreError = kOverSum ? 0x1p-18f : 0x1p-22f;
  using Raw = typename std::conditional<DT == 2, uint32_t, uint16_t>::type;
  __shared__ double lds[kTok][skewed(kE - 1) + 1];
  const int l = threadIdx.x & (L - 1), tok = threadIdx.x / L;
  // The tokens of this workgroup through a resource at the first: a row's
  // loads past the last expert read the next row's, past the end zeros.
  const int64_t first = (int64_t)blockIdx.x * kTok;
  const int64_t left = ((int64_t)a.T - 1 - first) * a.ld + a.E;
  const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)((const uint8_t *)a.logits + first * a.ld * sizeof(Raw)), 0,
                                                    (uint32_t)min(left * (int64_t)sizeof(Raw), (int64_t)0x7fffffff), 0x00020000);

  // Per expert: `code`, its index as the low bits of a key; `shift`, its place
  // with a score of 0 (its bias; from 1 on), or so far below 0 if it is none or
  // its bias bars it that a score of up to 1 leaves it there.
  const bool grouped = GROUPS == kRuns || (GROUPS == kAnyGroups && a.groups > 1);
  const bool scores = BIAS || grouped;
  uint32_t code[V];
  float per = kPlaces, shift[V];
  bool window = true;
#pragma unroll
  for (int v = 0; v < V; ++v) code[v] = kLow - (uint32_t)(v * L + l);
  if constexpr (BIAS) {
    float hi = -kInf, lo = kInf;
#pragma unroll
    for (int v = 0; v < V; ++v) shift[v] = a.bias[min(v * L + l, a.E - 1)];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool in = v * L + l < a.E && shift[v] > -kInf;  // (no NaN either)
      shift[v] = in ? shift[v] : -kInf;
      hi = fmaxf(hi, shift[v]);
      lo = fminf(lo, in ? shift[v] : kInf);
    }
    hi = max_l<L>(hi);
    lo = -max_l<L>(-lo);
    const float span = hi - lo + 1.0f;
    window = span < 0x1p20f;  // else (an infinite bias too) every token is open
    per = window ? kPlaces / span : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) shift[v] = shift[v] == -kInf ? -0x1p30f : window ? fmaf(shift[v] - lo, per, 1.0f) : 1.0f;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) shift[v] = v * L + l < a.E ? 1.0f : -0x1p30f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) asm volatile("" : "+v"(shift[v]));  // (kept, not worked out again)
  // Two keys in a row further apart than this are in order; sums of two
  // places of groups likewise.
  const uint32_t gap = BIAS ? (((uint32_t)(2.0f * kScoreError * per) + 7u) << kIdx) : kOne;
  const uint32_t group_gap = (uint32_t)(4.0f * kScoreError * per) + 16u;

  const int64_t t = first + tok;
  const bool live = t < a.T;  // (the lanes of a dead token go along)
  const uint32_t off = ((uint32_t)(live ? tok : 0) * (uint32_t)a.ld + (uint32_t)l) * (uint32_t)sizeof(Raw);
  Raw raw[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t o = off + (uint32_t)(v * L * (int)sizeof(Raw));
    if constexpr (DT == 2)
      raw[v] = __builtin_amdgcn_raw_buffer_load_b32(rs, o, 0, 0);
    else
      raw[v] = __builtin_amdgcn_raw_buffer_load_b16(rs, o, 0, 0);
  }
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] = DT == 2 ? __builtin_bit_cast(float, (uint32_t)raw[v]) : to_f32<DT>(raw[v]);
  // Scores, and for a softmax the row's largest logit and sum.
  const int rest = a.E - l;  // expert v L + l is one if v L < rest
  float m = -kInf, z = 1.0f, s[V];
  if (SCORE == kSoftmax && (scores || !a.renorm)) {
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, v * L < rest ? x[v] : -kInf);
    m = max_l<L>(m);
    z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // (Experts whose bias bars them stay in the sum.  Past the last expert
      // x is another row's or a gap's, and its exponential has no bound: no
      // score there, or it would outweigh any shift.)
      const float w = x[v] == m ? 1.0f : exp_(x[v] - m);
      const bool is = v * L < rest && x[v] > -kInf;
      z += is ? w : 0.0f;
      s[v] = is ? w : __builtin_nanf("");
    }
    z = sum_l<L>(z);
  } else if (SCORE == kSigmoid && scores) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = sigmoid_(x[v]);
  }
  bool open = !window;

  // Keys over indices; first by score where groups or a bias go by it.
  // Place 0 (a key below kOne) is for what cannot be chosen.
  uint32_t q[V];
  if (scores) {
    // (Groups without a bias go by the scores times the row's sum, which use all
    // the places, so few tokens are left open: 8192 tokens of 256 binary32 logits in
    // 8 groups 25.0 -> 10.5 us, 331 of 480 25.8 -> 6.4.)
    const float per_s = kOverSum ? per / z : per;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      // (A masked logit's score is NaN, and the maximum then 0.  0 x makes
      // it one for the sigmoid of -inf; +inf is held back from that.)
      float at = shift[v];
      if constexpr (SCORE == kSigmoid) at = fmaf(fminf(x[v], 0x1p100f), 0.0f, at);
      const uint32_t place = (uint32_t)fmaxf(fmaf(s[v], per_s, at), 0.0f);
      q[v] = (place << kIdx) + code[v];
    }
  }
  uint32_t keep = ~0u, keep2 = ~0u;  // bit g: group g stays (keep2: from 32 on)
  if (grouped) {
    uint32_t score = 0;     // of group l >> gs: the sum of its two places
    uint32_t odd = kOne;    // below kOne: a group has just one expert left
    const int gs = GROUPS == kRuns ? 0 : a.shift, g0 = l >> gs;
    const bool is = g0 < a.groups;
    if constexpr (GROUPS == kRuns) {
      // Groups are whole runs of v: two largest in each lane, then over
      // the lanes.  Bit v of ends: a group ends with v.
      uint32_t b1 = 0, b2 = 0;
      int g = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        b2 = max(b2, min(b1, q[v]));
        b1 = max(b1, q[v]);
        if ((a.ends >> v) & 1) {
          const uint32_t top = umax_l<L>(b1), next = umax_l<L>(b1 == top ? b2 : b1);
          score = l == g ? (top >> kIdx) + (next >> kIdx) : score;
          odd = min(odd, top < kOne ? kOne : next);
          ++g;
          b1 = b2 = 0;
        }
      }
    } else {
      uint32_t *keys = (uint32_t *)lds[tok];
      lds_order();
#pragma unroll
      for (int v = 0; v < V; ++v) keys[skewed(v * L + l)] = q[v];
      lds_order();
      uint32_t top, next;
      group_top2<L>(a, keys, l, a.shift, top, next);
      score = (top >> kIdx) + (next >> kIdx);
      odd = ~umax_l<L>(is && top >= kOne ? ~next : 0u);
      lds_order();
    }
    // Groups before this one in the order: of distinct numbers in 16 lanes
    // of their own, by turning the row; else one by one.
    int above = 0;
    if constexpr (GROUPS == kRuns && L == 16) {
      above = ranks_above(is ? (score << 4) + (15u - (uint32_t)l) : 0u);
    } else {
      for (int g = 0; g < a.groups; g += 8) {
        uint32_t o[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) o[u] = __shfl(score, ((g + u) << gs) & (L - 1), L);
#pragma unroll
        for (int u = 0; u < 8; ++u) above += g + u < a.groups && (o[u] > score || (o[u] == score && g + u < g0));
      }
    }
    const bool stays = is && above < a.used;
    // The worst that stays against the best that goes; a group with one
    // expert left has no sum of two places.
    const uint32_t worst = ~umax_l<L>(stays ? ~score : 0u), best = umax_l<L>(is && !stays ? score : 0u);
    open = open || (odd < kOne && a.per > 1) || (a.used < a.groups && worst - best < group_gap);
    const uint64_t all = __ballot(stays && l == g0 << gs);
    const uint64_t mask = L == 64 ? all : (all >> ((threadIdx.x & 63) / L * L)) & ((1ull << (L & 63)) - 1);
    keep = (uint32_t)mask;
    keep2 = (uint32_t)(mask >> 32);
  }
  if constexpr (!BIAS) {
    // By the logits.
    if constexpr (kRaw16) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // A bf16 or fp16 value in order: its binary32 bits, 16 of them
        // (fp16: 19 hold its sign, exponent and fraction); -0 ties with 0.
        constexpr int kDrop = DT == 0 ? 16 : 13;
        const uint32_t f = __builtin_bit_cast(uint32_t, x[v] + 0.0f);
        const uint32_t o = (f ^ (uint32_t)((int32_t)f >> 31 | (int32_t)0x80000000)) >> kDrop;
        q[v] = (v * L < rest && x[v] > -kInf ? (o + 1) << kIdx : 0u) + code[v];
      }
    } else {
      float hi = -kInf;
#pragma unroll
      for (int v = 0; v < V; ++v) hi = fmaxf(hi, v * L < rest ? x[v] : -kInf);
      hi = max_l<L>(hi);
      open = open || hi == kInf;
      const float lo = hi == kInf || hi == -kInf ? 0.0f : hi - 32.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t place = (uint32_t)fminf(fmaxf((x[v] - lo) * (kPlaces / 32.0f), 0.0f), kPlaces);
        q[v] = (v * L < rest && x[v] > -kInf ? (place + 1) << kIdx : 0u) + code[v];
      }
    }
  }
  if (grouped) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int g = GROUPS == kRuns ? __popc(a.ends & ((1u << v) - 1)) : group_of(a, v * L + l) << a.shift;
      const uint32_t word = L == 64 && g >= 32 ? keep2 : keep;
      q[v] = (word >> (g & 31)) & 1 ? q[v] : code[v];
    }
  }
  // The k best and the one or two behind them, in falling order (all V L
  // numbers are distinct, and there are more of them); mine: the l-th;
  // step: the least step down between the first k + 1, last: the one
  // after.
  uint32_t mine32 = 0, cur = 0x7fffffffu, step = ~0u, last = ~0u;
  for (int j = 0; j < a.picks; ++j) {
    uint32_t next = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) next = max(next, q[v] - cur);
    next = umax_l<L>(next) + cur;
    step = j > 0 ? min(step, last) : step;
    last = j > 0 ? cur - next : ~0u;
    mine32 = l == j ? next : mine32;
    cur = next;
  }
  int mine = mine32 < kOne ? -1 : (int)(kLow - (mine32 & kLow));
  const size_t row = (size_t)(live ? t : 0) * a.ld;
  if (!kRaw16 || grouped) {
    // (A step of whole places differs from that of keys by less than one.)
    const uint32_t least_step = kRaw16 ? 0u : gap + kOne;
    const bool close = step < least_step, near = last < least_step;
    // The k + 1 best are settled among themselves (a lane each) unless the
    // next is close to them too; without lanes for that all keys are.
    open = open || (near && (close || a.picks < a.k + 2)) || (close && a.picks < a.k + 2);
    if (open || close) {
      const double zd = SCORE == kSoftmax && scores ? exact_sum<L>(x, rest, m) : 1.0;
      if (open) {
        mine = exact_choice<DT, L, SCORE, BIAS>(a, row, m, zd, lds[tok], l);
      } else {
        const float xm = mine >= 0 && l <= a.k ? load_logit<DT>(a.logits, row + mine) : -kInf;
        const double key = xm == -kInf ? -(double)kInf : BIAS ? exact_key<SCORE, BIAS>(a, xm, mine, m, zd) : (double)xm;
        int above = 0;
        for (int j = 0; j <= a.k; ++j) {
          const double o = __shfl(key, j, L);
          const int at = __shfl(mine, j, L);
          above += o > key || (o == key && at < mine);
        }
        // (Missing choices, all -1, stay behind the others.)
        int *order = (int *)lds[tok];
        lds_order();
        if (l <= a.k) order[l] = -1;
        lds_order();
        if (l <= a.k && mine >= 0) order[above] = mine;
        lds_order();
        mine = l <= a.k ? order[l] : -1;
        lds_order();
      }
    }
  }
  if (l >= a.k) mine = -1;

  // Lane j: its choice's score and weight.
  float sc = 0.0f, w;
  const float xs = mine >= 0 ? load_logit<DT>(a.logits, row + mine) : -kInf;
  if constexpr (SCORE == kSoftmax) {
    const float mm = a.renorm ? max_l<L>(xs) : m;
    sc = mine >= 0 ? exp_below(xs, mm) : 0.0f;
    w = a.renorm ? sc / (sum_l<L>(sc) + 1e-20f) : sc / z;
  } else {
    sc = mine >= 0 ? 1.0f / (1.0f + expf(-xs)) : 0.0f;
    w = a.renorm ? sc / (sum_l<L>(sc) + 1e-20f) : sc;
  }
  if (live && l < a.k) {
    a.weights[(size_t)t * a.k + l] = mine >= 0 ? w * a.scale : 0.0f;
    a.ids[(size_t)t * a.k + l] = mine;
  }
}

template <int DT, int L, int V, int GROUPS>
hipError_t launch_topk_lv(const Topk &t) {
  TopkArgs a{t.logits, t.bias, t.weights, t.ids, (int)t.T, (int)t.E, (int)t.ld, t.k, t.groups, t.used,
             (int)(t.E / t.groups), t.renorm, t.k + 1, 0, 0, 0, t.scale};
  // (Where lanes are left for the k + 1 best, and keys are rounded.)
  if (t.k + 1 <= L && (t.dtype == 2 || t.bias)) a.picks = t.k + 2;
  while ((t.groups << (a.shift + 1)) <= L) ++a.shift;
  if (GROUPS == kRuns)
    for (int v = a.per / L - 1; v < V; v += a.per / L) a.ends |= 1u << v;
  const int64_t tokens = 256 / L;
  // ceil(2^32 / per): exact quotients for experts below 2^16 (not for per = 1).
  a.per_magic = a.per > 1 ? (uint32_t)((0x100000000ull + (uint64_t)a.per - 1) / (uint64_t)a.per) : 0u;
  const bool bias = t.bias != nullptr;
  const int64_t wgs = (t.T + tokens - 1) / tokens;
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  const void *fn =
      t.score == kSoftmax ? (bias ? reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSoftmax, true, GROUPS>)
                                  : reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSoftmax, false, GROUPS>))
                          : (bias ? reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSigmoid, true, GROUPS>)
                                  : reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSigmoid, false, GROUPS>));
  void *args[] = {&a};
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(256), args, 0, t.stream);
}

template <int DT>
hipError_t launch_topk_dt(const Topk &t) {
  // 16 lanes a token while they hold the experts, the choices and the groups.
  if (t.E <= 256 && t.k <= 16 && t.groups == 1) {
    if (t.E <= 64) return launch_topk_lv<DT, 16, 4, kNoGroups>(t);
    if (t.E <= 128) return launch_topk_lv<DT, 16, 8, kNoGroups>(t);
    return launch_topk_lv<DT, 16, 16, kNoGroups>(t);
  }
  if (t.E <= 256 && t.k <= 16 && t.groups <= 16 && t.E / t.groups % 16 == 0) {
    if (t.E <= 64) return launch_topk_lv<DT, 16, 4, kRuns>(t);
    if (t.E <= 128) return launch_topk_lv<DT, 16, 8, kRuns>(t);
    return launch_topk_lv<DT, 16, 16, kRuns>(t);
  }
  if (t.E <= 256) return launch_topk_lv<DT, 64, 4, kAnyGroups>(t);
  if (t.E <= 512) return launch_topk_lv<DT, 64, 8, kAnyGroups>(t);
  return launch_topk_lv<DT, 64, 16, kAnyGroups>(t);
}

// ---------------------------------------------------------------------------
// Gradient.  With p the softmax or sigmoid of the row and g the weights'
// gradients (times scale), S the chosen scores' sum:
//   softmax, renormalised:  dx_j = v_j (g_j - sum v g), v the softmax over the chosen
//   softmax:                dx_e = p_e ([e chosen] g_e - sum over the chosen p g)
//   sigmoid, renormalised:  dx_j = (1 - s_j) v_j (g_j - sum v g), v = s / S
//   sigmoid:                dx_j = g_j s_j (1 - s_j)
// and 0 for experts not chosen, except the second.  Lane j works out choice
// j; the choices meet the row in LDS.  Latency bounds it below tens of
// thousands of tokens: 16381 x 97 bf16, 6 choices, renormalised: 5.5 us (6.8 MB,
// 1.2 TB/s; a kernel of this size ends in 4 us at best), 4096 x 16: 4.7 us.
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
// Its steps wait for one another, and that bounds it: one chunk 4.4 us (up to
// 4096 choices, one launch), 64 chunks of 256 experts 4.0 + 8.1 us (count, then
// place; 4.2 MB in all).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64, kPlanPer = kPlanChunk / kPlanWaves;

struct PlanArgs {
  const int32_t *ids;
  int32_t *offsets, *rows, *slots, *hist;
  int n, E, k, chunks;
  int padded;  // E rounded up to a power of two
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
  __shared__ int32_t scan[kPlanWaves], sums[2][kPlanThreads];
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
  // Totals of this thread's expert: in the chunks before, and in all.  The
  // chunks' counts come from memory, so as many threads as there are share an
  // expert's: thread (part, expert) takes chunks part, part + parts, ...
  // (64 chunks of 256 experts: one thread an expert 9.3 us, four 8.4 us.)
  int before = 0, total = 0;
  if (a.chunks > 1) {
    const int e = tid % a.padded, part = tid / a.padded, parts = kPlanThreads / a.padded;
    if (e < a.E) {
#pragma unroll 8
      for (int c = part; c < a.chunks; c += parts) {
        const int h = a.hist[(size_t)c * a.E + e];
        total += h;
        before += c < (int)blockIdx.x ? h : 0;
      }
    }
    if (parts > 1) {
      sums[0][tid] = total;
      sums[1][tid] = before;
      __syncthreads();
      if (tid < a.padded)
        for (int p = 1; p < parts; ++p) {
          total += sums[0][p * a.padded + tid];
          before += sums[1][p * a.padded + tid];
        }
      else
        total = 0;
    }
  } else if (tid < a.E) {
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) total += cnt[w * a.E + tid];
  }
  int upto = wave_scan(total);
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
    int c[kPlanWaves];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) c[w] = cnt[w * a.E + tid];
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) {
      cnt[w * a.E + tid] = at;
      at += c[w];
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
  PlanArgs a{p.ids, p.offsets, p.rows, p.slots, p.ws, (int)(p.T * p.k), (int)p.E, p.k, 1, 1};
  while (a.padded < a.E) a.padded *= 2;
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
