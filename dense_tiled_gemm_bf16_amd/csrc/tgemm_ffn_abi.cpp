// C-ABI front end of libtgemm_ffn.so: argument validation and dispatch to the
// feed-forward kernels.  Every argument that the host can see is checked here;
// what lies in device memory (row offsets, indices) the kernels clamp.
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/tgemm_ffn.h"
#include "tgemm_ffn_internal.hpp"
#include "tgemm_host.hpp"
#include "tgemm_internal.hpp"

using namespace tgemm::host;
namespace ffn = tgemm::ffn;

namespace {

thread_local int g_tile_m = 0, g_tile_n = 0;

typedef long long ll;

// One tensor argument: `rows` rows of `cols` elements of `elem` bytes, `ld`
// elements apart.  vec: 16-byte aligned rows (else aligned to the element).
struct Tensor {
  const char *name;
  const void *p;
  int64_t rows, cols, ld;
  int elem;
  bool vec;
  bool needed;  // may not be NULL
  uint64_t bytes() const {
    return !p || rows <= 0 || cols <= 0 ? 0 : ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols) * (uint64_t)elem;
  }
};

// Each tensor by itself, then each of the first `outs` against all the
// others.  same: pairs (output, input) that may be the very same array.
struct Same {
  int out, in;
};
int check(const char *fn, const Tensor *t, int n, int outs, const Same *same = nullptr, int nsame = 0) {
  for (int i = 0; i < n; ++i) {
    const Tensor &x = t[i];
    if (x.rows <= 0 || x.cols <= 0) continue;
    if (!x.p) {
      if (x.needed) return fail(TGEMM_EINVAL, "%s: %s is NULL", fn, x.name);
      continue;
    }
    if (x.ld > INT32_MAX) return fail(TGEMM_ETOOBIG, "%s: the row stride of %s must be below 2^31", fn, x.name);
    if (x.rows > 1 && x.ld < x.cols)
      return fail(TGEMM_EINVAL, "%s: the row stride of %s (%lld) is below its row length (%lld)", fn, x.name,
                  (ll)x.ld, (ll)x.cols);
    if (x.vec) {
      if (misaligned(x.p)) return fail(TGEMM_EALIGN, "%s: %s is not 16-byte aligned", fn, x.name);
      if (x.cols % 8 != 0)
        return fail(TGEMM_EALIGN, "%s: the row length of %s (%lld) must be a multiple of 8", fn, x.name, (ll)x.cols);
      if (x.rows > 1 && x.ld % 8 != 0)
        return fail(TGEMM_EALIGN, "%s: the row stride of %s (%lld) must be a multiple of 8", fn, x.name, (ll)x.ld);
    } else if ((uintptr_t)x.p % (uintptr_t)x.elem != 0) {
      return fail(TGEMM_EALIGN, "%s: %s is not aligned to its elements", fn, x.name);
    }
  }
  for (int i = 0; i < outs; ++i)
    for (int j = 0; j < n; ++j) {
      if (i == j || !overlaps(t[i].p, t[i].bytes(), t[j].p, t[j].bytes())) continue;
      bool ok = false;
      for (int s = 0; s < nsame; ++s)
        ok = ok || (same[s].out == i && same[s].in == j && t[i].p == t[j].p && t[i].ld == t[j].ld &&
                    t[i].cols == t[j].cols);
      if (!ok) return fail(TGEMM_EINVAL, "%s: %s overlaps %s", fn, t[i].name, t[j].name);
    }
  return TGEMM_OK;
}

bool bad16(int64_t dtype) { return dtype != TGEMM_DT_BF16 && dtype != TGEMM_DT_F16; }

// Sizes leave the kernels' 32-bit indexes room for one step past the end.
constexpr int64_t kSizeLimit = (int64_t)INT32_MAX - 4095;
// The kernels look up their group among all of them, and each chunk of a plan
// adds the counts of all the others, so that its time grows with their square
// (1024 experts: 2^22 choices 0.33 ms, 2^24 4.3, 2^26 67; 256: 0.12, 1.3, 17).
constexpr int64_t kMostGroups = 65536, kMostChoices = (int64_t)1 << 26;

int sizes(const char *fn, const int64_t *v, int n) {
  for (int i = 0; i < n; ++i)
    if (v[i] < 0) return fail(TGEMM_EINVAL, "%s: negative size (%lld)", fn, (ll)v[i]);
  for (int i = 0; i < n; ++i)
    if (v[i] >= kSizeLimit) return fail(TGEMM_ETOOBIG, "%s: sizes must be below 2^31 - 4096 (%lld)", fn, (ll)v[i]);
  return TGEMM_OK;
}
int check_groups(const char *fn, int64_t groups) {
  if (groups > kMostGroups) return fail(TGEMM_ETOOBIG, "%s: groups=%lld must be at most 65536", fn, (ll)groups);
  return TGEMM_OK;
}

int launched(const char *fn, hipError_t e) {
  if (e == hipErrorInvalidConfiguration)
    return fail(TGEMM_ETOOBIG, "%s: the problem takes more workgroups than one dispatch holds", fn);
  if (e != hipSuccess) return fail(TGEMM_EHIP, "%s: kernel launch failed: %s", fn, hipGetErrorString(e));
  return TGEMM_OK;
}

// What dense and grouped products share once their arguments are checked.
int run_gemm(const char *fn, ffn::Gemm &g) {
  const int rc = ensure_device(&g.cus, nullptr);
  if (rc != TGEMM_OK) return rc;
  g.tile_m = g_tile_m;
  g.tile_n = g_tile_n;
  if (g.tile_m != 0 && !ffn::tile_supported(g, g.tile_m, g.tile_n))
    return fail(TGEMM_EINVAL, "%s: no %dx%d tile for this call (set by tgemm_ffn_set_tile)", fn, g.tile_m, g.tile_n);
  return launched(fn, ffn::launch_gemm(g));
}

int check_act(const char *fn, int64_t act, int64_t N) {
  if (act < TGEMM_ACT_NONE || act > TGEMM_ACT_GEGLU) return fail(TGEMM_EINVAL, "%s: no activation %lld", fn, (ll)act);
  if (ffn::is_gated((int)act) && N % 16 != 0)
    return fail(TGEMM_EALIGN, "%s: N=%lld must be a multiple of 16 (two halves) for a gated activation", fn, (ll)N);
  return TGEMM_OK;
}

// 31-bit buffer offsets of the weight: a K-contiguous one is addressed per
// tile (both halves at once if gated), the other as a whole in slices of 64.
int check_b(const char *fn, bool trans_b, bool gated, int64_t N, int64_t K, int64_t ldb) {
  const uint64_t rows = trans_b ? (gated ? (uint64_t)N / 2 : 0) + (uint64_t)tgemm::kTileN : (uint64_t)(K + 63) / 64 * 64;
  if (rows * (uint64_t)ldb * 2 > kOffsetLimit) return fail(TGEMM_ETOOBIG, "%s: B too large for 31-bit offsets", fn);
  return TGEMM_OK;
}

}  // namespace

extern "C" {

const char *tgemm_ffn_last_error(void) { return g_err; }

int tgemm_ffn_set_tile(int tile_m, int tile_n) {
  g_err[0] = '\0';
  const bool known = (tile_m == tile_n && (tile_m == 0 || tile_m == 256 || tile_m == 128 || tile_m == 64 || tile_m == 16)) ||
                     (tile_m == 256 && tile_n == 192);
  if (!known)
    return fail(TGEMM_EINVAL, "tgemm_ffn_set_tile: no %dx%d tile (256x256, 256x192, 128x128, 64x64, 16x16 or 0x0)",
                tile_m, tile_n);
  g_tile_m = tile_m;
  g_tile_n = tile_n;
  return TGEMM_OK;
}

int gemm_epilogue(const tgemm_epilogue_args *p, hipStream_t stream) {
  static const char fn[] = "gemm_epilogue";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  if (bad16(p->dtype)) return fail(TGEMM_EINVAL, "%s: no element type %lld", fn, (ll)p->dtype);
  if ((p->trans_a != 0 && p->trans_a != 1) || (p->trans_b != 0 && p->trans_b != 1))
    return fail(TGEMM_EINVAL, "%s: trans_a and trans_b must be 0 or 1", fn);
  const int64_t v[] = {p->M, p->N, p->K};
  int rc = sizes(fn, v, 3);
  if (rc == TGEMM_OK) rc = check_act(fn, p->act, p->N);
  if (rc != TGEMM_OK) return rc;
  const bool gated = ffn::is_gated((int)p->act);
  if (gated && p->trans_a) return fail(TGEMM_EINVAL, "%s: a gated activation takes A stored M x K (trans_a 0)", fn);
  if (p->M == 0 || p->N == 0) return TGEMM_OK;
  const int64_t out_n = gated ? p->N / 2 : p->N;
  // K is split where that pays and the workspace holds the sums (a forced tile
  // other than 64 x 64 goes without).
  int splits = ffn::epilogue_splits(p->trans_a != 0, p->trans_b != 0, p->M, p->N, p->K);
  if (!p->workspace || (uint64_t)splits * (uint64_t)p->M * (uint64_t)p->N * 4u > p->workspace_bytes ||
      (g_tile_m != 0 && g_tile_m != 64))
    splits = 1;
  const Tensor t[] = {
      {"C", p->C, p->M, out_n, p->ldc, 2, true, true},
      {"preact", p->preact, p->M, p->N, p->ldp, 2, true, false},
      {"workspace", splits > 1 ? p->workspace : nullptr, splits > 1, (int64_t)splits * p->M * p->N,
       (int64_t)splits * p->M * p->N, 4, false, false},
      {"A", p->A, p->K == 0 ? 0 : p->trans_a ? p->K : p->M, p->trans_a ? p->M : p->K, p->lda, 2, true, true},
      {"B", p->B, p->K == 0 ? 0 : p->trans_b ? p->N : p->K, p->trans_b ? p->K : p->N, p->ldb, 2, true, true},
      {"bias", p->bias, 1, p->N, p->N, 2, true, false},
      {"residual", p->residual, p->M, out_n, p->ldr, 2, true, false}};
  static const Same same[] = {{0, 6}};
  rc = check(fn, t, 7, 3, same, 1);
  if (rc != TGEMM_OK) return rc;
  if (splits > 1 && misaligned(p->workspace)) return fail(TGEMM_EALIGN, "%s: workspace is not 16-byte aligned", fn);
  // (An empty K is never read: its operands need no pointer and no stride. One row needs no stride.)
  const Tensor &ta = t[3], &tb = t[4];
  const int64_t lda = p->K == 0 ? 0 : ta.rows == 1 ? ta.cols : p->lda;
  const int64_t ldb = p->K == 0 ? 0 : tb.rows == 1 ? tb.cols : p->ldb;
  const uint64_t a_span = (p->trans_a ? (uint64_t)(p->K + 63) / 64 * 64 : (uint64_t)tgemm::kTileM) * (uint64_t)lda * 2;
  if (a_span > kOffsetLimit) return fail(TGEMM_ETOOBIG, "%s: A too large for 31-bit offsets", fn);
  rc = check_b(fn, p->trans_b != 0, gated, p->N, p->K, ldb);
  if (rc != TGEMM_OK) return rc;
  ffn::Gemm g{};
  g.dtype = (int)p->dtype;
  g.trans_a = p->trans_a != 0;
  g.trans_b = p->trans_b != 0;
  g.M = p->M;
  g.N = p->N;
  g.K = p->K;
  g.A = p->A;
  g.lda = lda;
  g.B = p->B;
  g.ldb = ldb;
  g.bias = p->bias;
  g.residual = p->residual;
  g.ldr = p->ldr;
  g.preact = p->preact;
  g.ldp = p->ldp;
  g.C = p->C;
  g.ldc = p->ldc;
  g.act = (int)p->act;
  g.ws = static_cast<float *>(p->workspace);
  g.splits = splits;
  g.stream = stream;
  return run_gemm(fn, g);
}

uint64_t tgemm_epilogue_workspace_bytes(int64_t trans_a, int64_t trans_b, int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return 0;
  const int splits = ffn::epilogue_splits(trans_a != 0, trans_b != 0, M, N, K);
  return splits > 1 ? (uint64_t)splits * (uint64_t)M * (uint64_t)N * 4u : 0;
}

uint64_t tgemm_epilogue_backward_workspace_bytes(int64_t M, int64_t N, int64_t groups) {
  if (M <= 0 || N <= 0 || groups < 0 || M > INT32_MAX || N > INT32_MAX || groups > INT32_MAX) return 0;
  return (uint64_t)ffn::act_grad_chunks(M, groups) * (uint64_t)N * 4u;
}

int gemm_epilogue_backward(const tgemm_epilogue_backward_args *p, hipStream_t stream) {
  static const char fn[] = "gemm_epilogue_backward";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  if (bad16(p->dtype)) return fail(TGEMM_EINVAL, "%s: no element type %lld", fn, (ll)p->dtype);
  const int64_t v[] = {p->M, p->N, p->groups};
  int rc = sizes(fn, v, 3);
  if (rc == TGEMM_OK) rc = check_groups(fn, p->groups);
  if (rc == TGEMM_OK) rc = check_act(fn, p->act, p->N);
  if (rc != TGEMM_OK) return rc;
  const bool gated = ffn::is_gated((int)p->act), none = p->act == TGEMM_ACT_NONE;
  if (p->N == 0 || (p->M == 0 && !p->dbias)) return TGEMM_OK;
  const uint64_t need = p->dbias ? tgemm_epilogue_backward_workspace_bytes(p->M, p->N, p->groups) : 0;
  const Tensor t[] = {
      {"dz", p->dz, p->M, p->N, p->ldz, 2, true, !none},
      {"dbias", p->dbias, p->groups > 0 ? p->groups : 1, p->N, p->N, 2, true, false},
      {"workspace", p->workspace, need > 0, (int64_t)(need / 4), (int64_t)(need / 4), 4, false, true},
      {"dout", p->dout, p->M, gated ? p->N / 2 : p->N, p->ldd, 2, true, true},
      {"preact", none ? nullptr : p->preact, p->M, p->N, p->ldp, 2, true, !none},
      {"offsets", p->offsets, p->groups > 0, p->groups + 1, p->groups + 1, 4, false, true}};
  // (The workspace may be longer than INT32_MAX elements: its stride is checked with its size.)
  if (need / 4 > (uint64_t)INT32_MAX) return fail(TGEMM_ETOOBIG, "%s: the column sums need a workspace above 8 GiB", fn);
  static const Same same[] = {{0, 3}, {0, 4}};
  rc = check(fn, t, 6, 3, same, 2);
  if (rc != TGEMM_OK) return rc;
  if (need > 0 && misaligned(p->workspace)) return fail(TGEMM_EALIGN, "%s: workspace is not 16-byte aligned", fn);
  if (p->workspace_bytes < need)
    return fail(TGEMM_EINVAL, "%s: needs %llu workspace bytes, got %llu", fn, (unsigned long long)need,
                (unsigned long long)p->workspace_bytes);
  rc = ensure_device(nullptr, nullptr);
  if (rc != TGEMM_OK) return rc;
  ffn::ActGrad g{(int)p->dtype, p->M, p->N, p->dout, p->ldd, p->preact, p->ldp, (int)p->act, p->dz, p->ldz,
                 p->dbias, p->groups, p->offsets, static_cast<float *>(p->workspace), stream};
  return launched(fn, ffn::launch_act_grad(g));
}

int gemm_grouped(const tgemm_grouped_args *p, hipStream_t stream) {
  static const char fn[] = "gemm_grouped";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  if (bad16(p->dtype)) return fail(TGEMM_EINVAL, "%s: no element type %lld", fn, (ll)p->dtype);
  if (p->trans_b != 0 && p->trans_b != 1) return fail(TGEMM_EINVAL, "%s: trans_b must be 0 or 1", fn);
  const int64_t v[] = {p->R, p->N, p->K, p->groups, p->src_rows};
  int rc = sizes(fn, v, 5);
  if (rc == TGEMM_OK) rc = check_groups(fn, p->groups);
  if (rc == TGEMM_OK) rc = check_act(fn, p->act, p->N);
  if (rc != TGEMM_OK) return rc;
  const bool gated = ffn::is_gated((int)p->act);
  if (p->R == 0 || p->N == 0 || p->groups == 0) return TGEMM_OK;
  const int64_t out_n = gated ? p->N / 2 : p->N;
  const int64_t src = p->rows ? p->src_rows : p->R;
  const int64_t b_rows = p->trans_b ? p->N : p->K, b_cols = p->trans_b ? p->K : p->N;
  const Tensor t[] = {
      {"C", p->C, p->R, out_n, p->ldc, 2, true, true},
      {"preact", p->preact, p->R, p->N, p->ldp, 2, true, false},
      {"A", p->A, p->K == 0 ? 0 : src, p->K, p->lda, 2, true, true},
      {"B", p->B, p->K == 0 ? 0 : b_rows, b_cols, p->ldb, 2, true, true},
      {"bias", p->bias, p->groups, p->N, p->N, 2, true, false},
      {"offsets", p->offsets, 1, p->groups + 1, p->groups + 1, 4, false, true},
      {"rows", p->rows, 1, p->R, p->R, 4, false, false}};
  rc = check(fn, t, 7, 2);
  if (rc != TGEMM_OK) return rc;
  const int64_t lda = p->K == 0 ? 0 : src == 1 ? p->K : p->lda;
  const int64_t ldb = p->K == 0 ? 0 : b_rows == 1 ? b_cols : p->ldb;
  if (p->K > 0 && p->groups > 1) {
    if (p->stride_b < 0) return fail(TGEMM_EINVAL, "%s: stride_b is negative", fn);
    if (p->stride_b % 8 != 0) return fail(TGEMM_EALIGN, "%s: stride_b must be a multiple of 8", fn);
    if (p->stride_b > ((int64_t)1 << 40)) return fail(TGEMM_ETOOBIG, "%s: stride_b too large", fn);
    const uint64_t all = ((uint64_t)(p->groups - 1) * (uint64_t)p->stride_b) * 2 + t[3].bytes();
    for (int i = 0; i < 2; ++i)
      if (overlaps(t[i].p, t[i].bytes(), p->B, all)) return fail(TGEMM_EINVAL, "%s: %s overlaps B", fn, t[i].name);
  }
  const uint64_t a_rows = p->rows ? (uint64_t)p->src_rows : (uint64_t)tgemm::kTileM;
  if (a_rows * (uint64_t)lda * 2 > kOffsetLimit) return fail(TGEMM_ETOOBIG, "%s: A too large for 31-bit offsets", fn);
  rc = check_b(fn, p->trans_b != 0, gated, p->N, p->K, ldb);
  if (rc != TGEMM_OK) return rc;
  ffn::Gemm g{};
  g.dtype = (int)p->dtype;
  g.trans_b = p->trans_b != 0;
  g.M = p->R;
  g.N = p->N;
  g.K = p->K;
  g.A = p->A;
  g.lda = lda;
  g.B = p->B;
  g.ldb = ldb;
  g.bias = p->bias;
  g.preact = p->preact;
  g.ldp = p->ldp;
  g.C = p->C;
  g.ldc = p->ldc;
  g.act = (int)p->act;
  g.groups = p->groups;
  g.offsets = p->offsets;
  g.rows = p->rows;
  g.src_rows = src;
  g.stride_b = p->K == 0 ? 0 : p->stride_b;
  g.stride_bias = p->N;
  g.stream = stream;
  return run_gemm(fn, g);
}

int gemm_grouped_tn(const tgemm_grouped_tn_args *p, hipStream_t stream) {
  static const char fn[] = "gemm_grouped_tn";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  if (bad16(p->dtype)) return fail(TGEMM_EINVAL, "%s: no element type %lld", fn, (ll)p->dtype);
  const int64_t v[] = {p->R, p->P, p->Q, p->groups};
  int rc = sizes(fn, v, 4);
  if (rc == TGEMM_OK) rc = check_groups(fn, p->groups);
  if (rc != TGEMM_OK) return rc;
  if (p->P == 0 || p->Q == 0 || p->groups == 0) return TGEMM_OK;
  if (p->groups * p->P > INT32_MAX) return fail(TGEMM_ETOOBIG, "%s: groups * P must be below 2^31", fn);
  const Tensor t[] = {{"out", p->out, p->groups * p->P, p->Q, p->Q, 2, true, true},
                      {"X", p->X, p->R, p->P, p->ldx, 2, true, true},
                      {"Y", p->Y, p->R, p->Q, p->ldy, 2, true, true},
                      {"offsets", p->offsets, 1, p->groups + 1, p->groups + 1, 4, false, true}};
  rc = check(fn, t, 4, 1);
  if (rc != TGEMM_OK) return rc;
  if (p->P % 8 != 0) return fail(TGEMM_EALIGN, "%s: P=%lld must be a multiple of 8", fn, (ll)p->P);
  const int64_t ldx = p->R <= 1 ? p->P : p->ldx, ldy = p->R <= 1 ? p->Q : p->ldy;
  const uint64_t rows = (uint64_t)(p->R + 63) / 64 * 64;
  if (rows * (uint64_t)ldx * 2 > kOffsetLimit) return fail(TGEMM_ETOOBIG, "%s: X too large for 31-bit offsets", fn);
  if (rows * (uint64_t)ldy * 2 > kOffsetLimit) return fail(TGEMM_ETOOBIG, "%s: Y too large for 31-bit offsets", fn);
  ffn::GroupedTn g{(int)p->dtype, p->R, p->P, p->Q, p->groups, p->X, ldx, p->Y, ldy, p->offsets, p->out, stream,
                   0, g_tile_m, g_tile_n};
  rc = ensure_device(&g.cus, nullptr);
  if (rc != TGEMM_OK) return rc;
  if (g.tile_m != 0 && (g.tile_m != g.tile_n || g.tile_m == 16))
    return fail(TGEMM_EINVAL, "%s: no %dx%d tile for this call (set by tgemm_ffn_set_tile)", fn, g.tile_m, g.tile_n);
  return launched(fn, ffn::launch_grouped_tn(g));
}

static int check_route(const char *fn, int64_t dtype, int64_t T, int64_t E, int64_t k, int64_t score, int64_t renorm) {
  if (dtype != TGEMM_DT_BF16 && dtype != TGEMM_DT_F16 && dtype != TGEMM_DT_F32)
    return fail(TGEMM_EINVAL, "%s: no element type %lld", fn, (ll)dtype);
  const int64_t v[] = {T, E, k};
  const int rc = sizes(fn, v, 3);
  if (rc != TGEMM_OK) return rc;
  if (score != TGEMM_SCORE_SOFTMAX && score != TGEMM_SCORE_SIGMOID)
    return fail(TGEMM_EINVAL, "%s: no score %lld", fn, (ll)score);
  if (renorm != 0 && renorm != 1) return fail(TGEMM_EINVAL, "%s: renormalize must be 0 or 1", fn);
  if (E < 1 || E > 1024) return fail(TGEMM_EINVAL, "%s: E=%lld must be 1 .. 1024", fn, (ll)E);
  if (k < 1 || k > 64 || k > E) return fail(TGEMM_EINVAL, "%s: k=%lld must be 1 .. 64 and at most E", fn, (ll)k);
  if (T * k >= kSizeLimit) return fail(TGEMM_ETOOBIG, "%s: T k must be below 2^31 - 4096", fn);
  return TGEMM_OK;
}

int route_topk(const tgemm_route_args *p, hipStream_t stream) {
  static const char fn[] = "route_topk";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  int rc = check_route(fn, p->dtype, p->T, p->E, p->k, p->score, p->renormalize);
  if (rc != TGEMM_OK) return rc;
  if (p->groups < 1 || p->groups > 64 || p->E % p->groups != 0)
    return fail(TGEMM_EINVAL, "%s: groups=%lld must be 1 .. 64 and divide E=%lld", fn, (ll)p->groups, (ll)p->E);
  if (p->groups_used < 1 || p->groups_used > p->groups)
    return fail(TGEMM_EINVAL, "%s: groups_used=%lld must be 1 .. groups", fn, (ll)p->groups_used);
  if (p->k > p->groups_used * (p->E / p->groups))
    return fail(TGEMM_EINVAL, "%s: k=%lld is more than the experts of groups_used groups", fn, (ll)p->k);
  if (p->T == 0) return TGEMM_OK;
  const int elem = p->dtype == TGEMM_DT_F32 ? 4 : 2;
  const Tensor t[] = {{"weights", p->weights, p->T, p->k, p->k, 4, false, true},
                      {"ids", p->ids, p->T, p->k, p->k, 4, false, true},
                      {"logits", p->logits, p->T, p->E, p->ld, elem, false, true},
                      {"bias", p->bias, 1, p->E, p->E, 4, false, false}};
  rc = check(fn, t, 4, 2);
  if (rc != TGEMM_OK) return rc;
  // (The kernel takes up to 16 rows through one 31-bit resource.)
  const int64_t ld = p->T == 1 ? p->E : p->ld;
  if (16 * (uint64_t)ld * (uint64_t)elem > kOffsetLimit)
    return fail(TGEMM_ETOOBIG, "%s: 16 row strides of logits must be below 2^31 bytes", fn);
  rc = ensure_device(nullptr, nullptr);
  if (rc != TGEMM_OK) return rc;
  ffn::Topk g{(int)p->dtype, p->T, p->E, p->logits, ld, p->bias, (int)p->k, (int)p->score, (int)p->groups,
              (int)p->groups_used, (int)p->renormalize, (float)p->scale, p->weights, p->ids, stream};
  return launched(fn, ffn::launch_topk(g));
}

int route_topk_backward(const tgemm_route_backward_args *p, hipStream_t stream) {
  static const char fn[] = "route_topk_backward";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  int rc = check_route(fn, p->dtype, p->T, p->E, p->k, p->score, p->renormalize);
  if (rc != TGEMM_OK || p->T == 0) return rc;
  const int elem = p->dtype == TGEMM_DT_F32 ? 4 : 2;
  const Tensor t[] = {{"dlogits", p->dlogits, p->T, p->E, p->ldo, elem, false, true},
                      {"logits", p->logits, p->T, p->E, p->ld, elem, false, true},
                      {"ids", p->ids, p->T, p->k, p->k, 4, false, true},
                      {"dweights", p->dweights, p->T, p->k, p->k, 4, false, true}};
  static const Same same[] = {{0, 1}};
  rc = check(fn, t, 4, 1, same, 1);
  if (rc == TGEMM_OK) rc = ensure_device(nullptr, nullptr);
  if (rc != TGEMM_OK) return rc;
  ffn::TopkGrad g{(int)p->dtype, p->T, p->E, p->logits, p->ld, p->ids, p->dweights, (int)p->k, (int)p->score,
                  (int)p->renormalize, (float)p->scale, p->dlogits, p->ldo, stream};
  return launched(fn, ffn::launch_topk_grad(g));
}

uint64_t tgemm_route_plan_workspace_bytes(int64_t T, int64_t k, int64_t E) {
  if (T <= 0 || k <= 0 || E <= 0 || E > 1024 || T > kMostChoices || k > kMostChoices || T * k > kMostChoices)
    return 0;
  return (uint64_t)ffn::plan_ws_ints(T * k, E) * 4u;
}

int route_plan(const tgemm_route_plan_args *p, hipStream_t stream) {
  static const char fn[] = "route_plan";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  const int64_t v[] = {p->T, p->k, p->E};
  int rc = sizes(fn, v, 3);
  if (rc != TGEMM_OK) return rc;
  if (p->E < 1 || p->E > 1024) return fail(TGEMM_EINVAL, "%s: E=%lld must be 1 .. 1024", fn, (ll)p->E);
  if (p->k < 1) return fail(TGEMM_EINVAL, "%s: k=%lld must be at least 1", fn, (ll)p->k);
  if (p->T * p->k > kMostChoices) return fail(TGEMM_ETOOBIG, "%s: T k must be at most 2^26", fn);
  const uint64_t need = tgemm_route_plan_workspace_bytes(p->T, p->k, p->E);
  const Tensor t[] = {{"offsets", p->offsets, 1, p->E + 1, p->E + 1, 4, false, true},
                      {"rows", p->rows, p->T, p->k, p->k, 4, false, true},
                      {"slots", p->slots, p->T, p->k, p->k, 4, false, true},
                      {"workspace", p->workspace, need > 0, (int64_t)(need / 4), (int64_t)(need / 4), 4, false, true},
                      {"ids", p->ids, p->T, p->k, p->k, 4, false, true}};
  rc = check(fn, t, 5, 4);
  if (rc != TGEMM_OK) return rc;
  if (need > 0 && misaligned(p->workspace)) return fail(TGEMM_EALIGN, "%s: workspace is not 16-byte aligned", fn);
  if (p->workspace_bytes < need)
    return fail(TGEMM_EINVAL, "%s: needs %llu workspace bytes, got %llu", fn, (unsigned long long)need,
                (unsigned long long)p->workspace_bytes);
  rc = ensure_device(nullptr, nullptr);
  if (rc != TGEMM_OK) return rc;
  ffn::Plan g{p->T, p->E, (int)p->k, p->ids, p->offsets, p->rows, p->slots, static_cast<int32_t *>(p->workspace),
              stream};
  return launched(fn, ffn::launch_plan(g));
}

int expert_gather(const tgemm_expert_gather_args *p, hipStream_t stream) {
  static const char fn[] = "expert_gather";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  const int64_t v[] = {p->R, p->D, p->src_rows};
  int rc = sizes(fn, v, 3);
  if (rc != TGEMM_OK || p->R == 0 || p->D == 0 || p->src_rows == 0) return rc;
  const Tensor t[] = {{"out", p->out, p->R, p->D, p->ldo, 2, true, true},
                      {"x", p->x, p->src_rows, p->D, p->ldx, 2, true, true},
                      {"rows", p->rows, 1, p->R, p->R, 4, false, true}};
  rc = check(fn, t, 3, 1);
  if (rc == TGEMM_OK) rc = ensure_device(nullptr, nullptr);
  if (rc != TGEMM_OK) return rc;
  ffn::Gather g{p->R, p->D, p->src_rows, p->x, p->ldx, p->rows, p->out, p->ldo, stream};
  return launched(fn, ffn::launch_gather(g));
}

int expert_combine(const tgemm_expert_combine_args *p, hipStream_t stream) {
  static const char fn[] = "expert_combine";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  if (bad16(p->dtype)) return fail(TGEMM_EINVAL, "%s: no element type %lld", fn, (ll)p->dtype);
  const int64_t v[] = {p->T, p->D, p->R, p->k};
  int rc = sizes(fn, v, 4);
  if (rc != TGEMM_OK || p->T == 0 || p->D == 0) return rc;
  if (p->T * p->k >= kSizeLimit) return fail(TGEMM_ETOOBIG, "%s: T k must be below 2^31 - 4096", fn);
  const Tensor t[] = {{"out", p->out, p->T, p->D, p->ldo, 2, true, true},
                      {"h", p->h, p->k == 0 ? 0 : p->R, p->D, p->ldh, 2, true, true},
                      {"slots", p->slots, p->T, p->k, p->k, 4, false, true},
                      {"weights", p->weights, p->T, p->k, p->k, 4, false, false},
                      {"residual", p->residual, p->T, p->D, p->ldr, 2, true, false}};
  static const Same same[] = {{0, 4}};
  rc = check(fn, t, 5, 1, same, 1);
  if (rc == TGEMM_OK) rc = ensure_device(nullptr, nullptr);
  if (rc != TGEMM_OK) return rc;
  ffn::Combine g{(int)p->dtype, p->T, p->D, p->R, (int)p->k, p->h, p->ldh, p->slots, p->weights, p->residual,
                 p->ldr, p->out, p->ldo, stream};
  return launched(fn, ffn::launch_combine(g));
}

int expert_combine_backward(const tgemm_expert_combine_backward_args *p, hipStream_t stream) {
  static const char fn[] = "expert_combine_backward";
  g_err[0] = '\0';
  if (!p) return fail(TGEMM_EINVAL, "%s: args is NULL", fn);
  if (bad16(p->dtype)) return fail(TGEMM_EINVAL, "%s: no element type %lld", fn, (ll)p->dtype);
  const int64_t v[] = {p->T, p->D, p->R, p->k};
  int rc = sizes(fn, v, 4);
  if (rc != TGEMM_OK || p->T == 0 || p->k == 0) return rc;
  if (p->T * p->k >= kSizeLimit) return fail(TGEMM_ETOOBIG, "%s: T k must be below 2^31 - 4096", fn);
  const Tensor t[] = {{"dh", p->dh, p->R, p->D, p->ldg, 2, true, true},
                      {"dweights", p->dweights, p->T, p->k, p->k, 4, false, true},
                      {"dout", p->dout, p->T, p->D, p->ldd, 2, true, true},
                      {"h", p->h, p->R, p->D, p->ldh, 2, true, true},
                      {"slots", p->slots, p->T, p->k, p->k, 4, false, true},
                      {"weights", p->weights, p->T, p->k, p->k, 4, false, true}};
  rc = check(fn, t, 6, 2);
  if (rc == TGEMM_OK) rc = ensure_device(nullptr, nullptr);
  if (rc != TGEMM_OK) return rc;
  ffn::CombineGrad g{(int)p->dtype, p->T, p->D, p->R, (int)p->k, p->dout, p->ldd, p->h, p->ldh, p->slots,
                     p->weights, p->dh, p->ldg, p->dweights, stream};
  return launched(fn, ffn::launch_combine_grad(g));
}

}  // extern "C"
