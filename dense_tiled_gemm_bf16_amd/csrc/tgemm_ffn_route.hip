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

// exp(x - m) for x <= m, of the largest of a row; 1 where both are infinite.
__device__ __forceinline__ float exp_below(float x, float m) { return x == m ? 1.0f : expf(x - m); }

template <int L>
__device__ __forceinline__ float max_l(float v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, L));
  return v;
}
template <int L, class V>
__device__ __forceinline__ V sum_l(V v) {
#pragma unroll
  for (int d = 1; d < L; d <<= 1) v += __shfl_xor(v, d, L);
  return v;
}

// A token takes L lanes of a wave, lane l the experts l, l + L, ...: V of
// them, held in registers.
struct TopkArgs {
  const void *logits;
  const float *bias;
  float *weights;
  int32_t *ids;
  int T, E, ld, k, groups, used, per, renorm;
  uint32_t per_magic;  // expert -> group: __umulhi(e, per_magic)
  float scale;
};

// KEYED: keys are scores + bias in 64 bits, within the best groups; else the
// logits themselves (both scores grow with the logit).
template <int DT, int L, int V, int SCORE, bool KEYED>
__global__ __launch_bounds__(256) void topk_kernel(const TopkArgs a) {
  using Key = typename std::conditional<KEYED, double, float>::type;
  constexpr int kTok = 256 / L;
  __shared__ Key keys[KEYED ? kTok : 1][KEYED ? L * V : 1];
  const int l = threadIdx.x & (L - 1), tok = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * kTok + tok;
  const bool live = t < a.T;  // (the lanes of a dead token go along)
  const size_t row = (size_t)(live ? t : 0) * a.ld;

  Key key[V];
  float x[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = v * L + l;
    x[v] = e < a.E ? load_logit<DT>(a.logits, row + e) : -kInf;
  }
  // Softmax over the row: its largest and the sum (when a score needs them).
  float m = -kInf, z = 1.0f;
  double zd = 1.0;
  const bool whole = SCORE == kSoftmax && (KEYED || !a.renorm);
  if (whole) {
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
    m = max_l<L>(m);
    if constexpr (KEYED) {
      zd = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const double s = x[v] == -kInf ? 0.0 : x[v] == m ? 1.0 : exp((double)x[v] - (double)m);
        key[v] = s;
        zd += s;
      }
      zd = sum_l<L>(zd);
      z = (float)zd;
    } else {
      z = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) z += x[v] == -kInf ? 0.0f : exp_below(x[v], m);
      z = sum_l<L>(z);
    }
  }
  if constexpr (KEYED) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + l;
      double s;
      if constexpr (SCORE == kSoftmax)
        s = key[v] / zd;
      else
        s = 1.0 / (1.0 + exp(-(double)x[v]));
      if (a.bias && e < a.E) s += (double)a.bias[e];
      key[v] = x[v] == -kInf || !(s == s) ? -(double)kInf : s;
    }
    if (a.groups > 1) {
#pragma unroll
      for (int v = 0; v < V; ++v) keys[tok][v * L + l] = key[v];
      __syncthreads();
      // Lane g: the two largest keys of group g.
      double best = -(double)kInf, second = -(double)kInf;
      if (l < a.groups) {
        for (int i = 0; i < a.per; ++i) {
          const double s = keys[tok][l * a.per + i];
          second = fmax(second, fmin(s, best));
          best = fmax(best, s);
        }
      }
      const double score = second == -(double)kInf ? best : best + second;
      int above = 0;
      for (int g = 0; g < a.groups; ++g) {
        const double o = __shfl(score, g, L);
        above += o > score || (o == score && g < l);
      }
      // Bit g of the token's mask: group g stays.
      const uint64_t all = __ballot(l < a.groups && above < a.used);
      const uint64_t mask = L == 64 ? all : (all >> ((threadIdx.x & 63) / L * L)) & ((1ull << (L & 63)) - 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t e = (uint32_t)(v * L + l);
        const int g = (int)(a.per == 1 ? e : __umulhi(e, a.per_magic));
        if (!((mask >> (g & 63)) & 1)) key[v] = -(double)kInf;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = x[v];
  }

  // k times the largest key, ties to the lowest expert; lane j keeps the
  // j-th choice.
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    Key best = -(Key)kInf;
    int at = 0x7fffffff;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v * L + l;
      }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) {
      const Key ob = __shfl_xor(best, d, L);
      const int oa = __shfl_xor(at, d, L);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    const bool none = at == 0x7fffffff;
    if (l == j) mine = none ? -1 : at;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at == v * L + l) key[v] = -(Key)kInf;
  }

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
             (int)(t.E / t.groups), t.renorm, 0, t.scale};
  // ceil(2^32 / per): exact quotients for experts below 2^16 (not for per = 1).
  a.per_magic = a.per > 1 ? (uint32_t)((0x100000000ull + (uint64_t)a.per - 1) / (uint64_t)a.per) : 0u;
  const bool keyed = t.bias != nullptr || t.groups > 1;
  const int64_t wgs = (t.T + 256 / L - 1) / (256 / L);
  if (wgs > (int64_t)(UINT32_MAX / 256)) return hipErrorInvalidConfiguration;
  const void *fn =
      t.score == kSoftmax ? (keyed ? reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSoftmax, true>)
                                   : reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSoftmax, false>))
                          : (keyed ? reinterpret_cast<const void *>(&topk_kernel<DT, L, V, kSigmoid, true>)
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
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * L + l;
      x[v] = e < a.E ? load_logit<DT>(a.logits, row + e) : -kInf;
      m = fmaxf(m, x[v]);
    }
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
