/*
 * tgemm_ffn -- the operators of a model's feed-forward layers around the
 * dense products of tgemm.h, for AMD Instinct MI355X (gfx950): the product
 * with bias, activation and residual in its epilogue, the routing of tokens to
 * experts, the experts' products and the layer norm, each with its backward
 * pass; and the products on 4-bit operands (MXFP4), with their quantisation.
 *
 * C ABI of the library libtgemm_ffn.so.  Conventions are those of tgemm.h:
 * row-major matrices, plain device pointers, the caller owns every buffer
 * (workspaces too); an entry point validates its arguments, enqueues its
 * kernels on `stream` (NULL = the null stream) of the current device and
 * returns one of the TGEMM_* codes; it allocates nothing, never
 * synchronises, records kernel launches only (a caller may capture it into a
 * graph; two graphs that run at once need workspaces of their own), and may be
 * called from several threads.  After a non-zero return
 * tgemm_ffn_last_error() describes the failure of the calling thread.
 *
 * Arguments come in structs of 8-byte fields; a field that does not apply is
 * 0 or NULL.  Element types: TGEMM_DT_BF16, TGEMM_DT_F16 and, for logits, norms
 * and quantisation, TGEMM_DT_F32.  Sums are held in 32 bits; each output is
 * rounded once, to nearest even.  16-bit tensors are 16-byte aligned with row strides and
 * contiguous dimensions that are multiples of 8 (TGEMM_EALIGN otherwise).
 * An output may overlap no other argument, except where said.  Sizes (and T k)
 * are below 2^31 - 4096, row strides below 2^31, row groups at most 65536
 * (TGEMM_ETOOBIG otherwise).
 *
 * Row groups: offsets is a device array of groups + 1 int32, and group e is
 * the rows offsets[e] .. offsets[e + 1] - 1 (none if that is empty).  The
 * values are clamped to the rows there are; rows in no group are left as they
 * were.  If they do not ascend, which rows are computed is unspecified (memory
 * outside the outputs is never touched).
 */
#ifndef TGEMM_FFN_H
#define TGEMM_FFN_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "tgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TGEMM_DT_BF16 0
#define TGEMM_DT_F16 1
#define TGEMM_DT_F32 2

/* Activations.  gelu is z Phi(z); gelu_tanh z (1 + tanh(sqrt(2/pi) (z +
 * 0.044715 z^3))) / 2; silu z / (1 + exp(-z)).  The gated ones take Z =
 * [G | U], two halves of N / 2 columns, and give silu(G) * U or gelu(G) * U. */
#define TGEMM_ACT_NONE 0
#define TGEMM_ACT_RELU 1
#define TGEMM_ACT_GELU 2
#define TGEMM_ACT_GELU_TANH 3
#define TGEMM_ACT_SILU 4
#define TGEMM_ACT_SWIGLU 5
#define TGEMM_ACT_GEGLU 6

TGEMM_API const char *tgemm_ffn_last_error(void);

/* Sets the calling thread's output tile for the products below: 256 x 256,
 * 256 x 192, 128 x 128, 64 x 64, or 16 x 16 for the kernel for few rows;
 * 0, 0 (the default) chooses by size.  For measurements and tests. */
TGEMM_API int tgemm_ffn_set_tile(int tile_m, int tile_n);

/*
 * C = act(Z) + residual, Z = op(A) op(B) + bias.
 *
 * A, B, trans_a, trans_b and the strides are those of gemm_bf16 (tgemm.h).
 * N counts B's columns; C and the residual have N columns, or N / 2 with a
 * gated activation (which takes trans_a == 0).  bias (N values) and residual
 * may be NULL.  The residual may be C itself (same pointer and stride).
 * preact, if not NULL, receives Z rounded to the element type, M x N (the
 * activation takes the sums before that rounding).
 * workspace: few output tiles under a deep K leave most of the chip idle; with
 * tgemm_epilogue_workspace_bytes(trans_a, trans_b, M, N, K) bytes of it
 * (16-byte aligned; 0: it would not be used) K is split over several
 * workgroups a tile.  With less, or NULL, it is not.
 * Limits: as gemm_bf16; gated with trans_b, (N / 2 + 256) ldb 2 < 2^31.
 */
typedef struct {
  int64_t dtype, trans_a, trans_b, M, N, K;
  const void *A;
  int64_t lda;
  const void *B;
  int64_t ldb;
  const void *bias;
  const void *residual;
  int64_t ldr;
  void *preact;
  int64_t ldp;
  void *C;
  int64_t ldc;
  int64_t act;
  void *workspace;
  uint64_t workspace_bytes;
} tgemm_epilogue_args;
TGEMM_API int gemm_epilogue(const tgemm_epilogue_args *args, hipStream_t stream);
TGEMM_API uint64_t tgemm_epilogue_workspace_bytes(int64_t trans_a, int64_t trans_b, int64_t M, int64_t N, int64_t K);

/*
 * The epilogue's backward pass: dZ = dC * act'(Z) (gated: dG = dC U act'(G),
 * dU = dC act(G)) and, if dbias is not NULL, the column sums of dZ before its
 * rounding, for each group of rows (groups > 0: dbias is groups x N, zeros for
 * an empty group) or over all of them (groups == 0).  M x N is the size of Z;
 * dout has N columns, N / 2 if gated.  act NONE reads no preact; its dz may
 * be NULL (it would be a copy of dout).  dz may be preact itself or, not
 * gated, dout itself (same pointer and stride).
 * workspace: tgemm_epilogue_backward_workspace_bytes(M, N, groups) bytes,
 * 16-byte aligned; NULL without dbias.
 */
typedef struct {
  int64_t dtype, M, N;
  const void *dout;
  int64_t ldd;
  const void *preact;
  int64_t ldp;
  int64_t act;
  void *dz;
  int64_t ldz;
  void *dbias;
  int64_t groups;
  const int32_t *offsets;
  void *workspace;
  uint64_t workspace_bytes;
} tgemm_epilogue_backward_args;
TGEMM_API int gemm_epilogue_backward(const tgemm_epilogue_backward_args *args, hipStream_t stream);
TGEMM_API uint64_t tgemm_epilogue_backward_workspace_bytes(int64_t M, int64_t N, int64_t groups);

/*
 * The experts' products: for each row r of group e (row groups as above, of at
 * most R rows), C[r] = act(A[s] . op(B_e) + bias_e) with s = rows[r], or r if
 * rows is NULL.  A has src_rows rows (R if rows is NULL); an s outside them
 * reads zeros.  B_e is the matrix at B + e stride_b elements: N x K rows if
 * trans_b, else K x N.  bias is groups x N or NULL; preact as above, R x N.
 * Limits: with rows, src_rows lda 2 < 2^31; else 256 lda 2 < 2^31; B_e as in
 * gemm_epilogue.
 */
typedef struct {
  int64_t dtype, trans_b, R, N, K, groups;
  const int32_t *offsets;
  const int32_t *rows;
  int64_t src_rows;
  const void *A;
  int64_t lda;
  const void *B;
  int64_t ldb, stride_b;
  const void *bias;
  void *preact;
  int64_t ldp;
  void *C;
  int64_t ldc;
  int64_t act;
} tgemm_grouped_args;
TGEMM_API int gemm_grouped(const tgemm_grouped_args *args, hipStream_t stream);

/*
 * out_e = X_e^T . Y_e over the rows of group e: the weights' gradients of the
 * experts' products.  X is R x P, Y R x Q; out is groups x P x Q, packed
 * (zeros for an empty group).  Limits: R, rounded up to 64, times ldx or ldy
 * times 2 < 2^31.
 */
typedef struct {
  int64_t dtype, R, P, Q, groups;
  const int32_t *offsets;
  const void *X;
  int64_t ldx;
  const void *Y;
  int64_t ldy;
  void *out;
} tgemm_grouped_tn_args;
TGEMM_API int gemm_grouped_tn(const tgemm_grouped_tn_args *args, hipStream_t stream);

#define TGEMM_SCORE_SOFTMAX 0
#define TGEMM_SCORE_SIGMOID 1

/*
 * The choice of k experts for each of T tokens.
 *
 * A logit of -inf or NaN is masked: its expert is never chosen and takes no
 * part in the row's softmax.  s is the softmax of the row's logits or their
 * sigmoid; the keys are s + bias (bias: E binary32, or NULL), compared as
 * computed in 64 bits.  A key of -inf or NaN is never chosen.  groups > 1 cuts
 * the experts into that many runs of E / groups; a group's score is the sum of
 * its two largest keys (its one key, where one is left), and only the
 * groups_used best groups are chosen from.  Without bias experts are then
 * ordered by the logits themselves (as by s, without the ties that rounding
 * makes).  The choices are the k largest keys in falling order; ties go
 * to the lowest index, of groups too.  weights are the chosen s times scale;
 * with renormalize, scale times the softmax of the chosen logits (which is s
 * over the sum of the chosen s, and holds also where a bias or groups leave
 * only scores too small for binary32), or the chosen sigmoids divided by
 * their sum + 1e-20.  Where fewer than k experts can be chosen the last ids
 * are -1 and their weights 0.
 *
 *   logits   T x E, rows ld elements apart, TGEMM_DT_BF16, F16 or F32 (aligned
 *            to the element)
 *   weights  T x k binary32;  ids  T x k int32, packed
 * Limits: 1 <= E <= 1024, k <= 64, groups <= 64 dividing E,
 * k <= groups_used E / groups; 16 rows of logits below 2^31 bytes.
 */
typedef struct {
  int64_t dtype, T, E;
  const void *logits;
  int64_t ld;
  const float *bias;
  int64_t k, score, groups, groups_used, renormalize;
  double scale;
  float *weights;
  int32_t *ids;
} tgemm_route_args;
TGEMM_API int route_topk(const tgemm_route_args *args, hipStream_t stream);

/*
 * Its gradient: dlogits (T x E, the logits' type, rows ldo apart) from
 * dweights (T x k binary32), the logits and the ids that route_topk gave
 * (distinct in a row; an id outside 0 .. E - 1 has no gradient).  The choice
 * itself, the bias and the groups have none.  dlogits may be logits itself.
 */
typedef struct {
  int64_t dtype, T, E;
  const void *logits;
  int64_t ld;
  const int32_t *ids;
  const float *dweights;
  int64_t k, score, renormalize;
  double scale;
  void *dlogits;
  int64_t ldo;
} tgemm_route_backward_args;
TGEMM_API int route_topk_backward(const tgemm_route_backward_args *args, hipStream_t stream);

/*
 * The plan of the experts' products: the T x k choices sorted by expert,
 * tokens in order.  offsets (E + 1 int32) are the row groups, rows (T k
 * int32) the token of each row (-1 behind the last), slots (T x k int32) the
 * row of each choice (-1 for an id outside 0 .. E - 1, which has none).
 * workspace: tgemm_route_plan_workspace_bytes(T, k, E) bytes, 16-byte
 * aligned (may be NULL if 0).  Limits: E <= 1024, T k <= 2^26.
 */
typedef struct {
  int64_t T, k, E;
  const int32_t *ids;
  int32_t *offsets, *rows, *slots;
  void *workspace;
  uint64_t workspace_bytes;
} tgemm_route_plan_args;
TGEMM_API int route_plan(const tgemm_route_plan_args *args, hipStream_t stream);
TGEMM_API uint64_t tgemm_route_plan_workspace_bytes(int64_t T, int64_t k, int64_t E);

/*
 * out[r] = x[rows[r]] for r < R (D columns, x of src_rows rows); a row whose
 * index is outside x is left as it was.
 */
typedef struct {
  int64_t R, D, src_rows;
  const void *x;
  int64_t ldx;
  const int32_t *rows;
  void *out;
  int64_t ldo;
} tgemm_expert_gather_args;
TGEMM_API int expert_gather(const tgemm_expert_gather_args *args, hipStream_t stream);

/*
 * out[t] = sum over j of weights[t][j] h[slots[t][j]] + residual[t], for T
 * tokens of D columns; h has R rows.  weights (T x k binary32) NULL: ones; a
 * slot outside 0 .. R - 1 adds nothing.  residual may be NULL, or out itself.
 */
typedef struct {
  int64_t dtype, T, D, R, k;
  const void *h;
  int64_t ldh;
  const int32_t *slots;
  const float *weights;
  const void *residual;
  int64_t ldr;
  void *out;
  int64_t ldo;
} tgemm_expert_combine_args;
TGEMM_API int expert_combine(const tgemm_expert_combine_args *args, hipStream_t stream);

/*
 * Its gradients: dh[slots[t][j]] = weights[t][j] dout[t] and dweights[t][j] =
 * dout[t] . h[slots[t][j]] (0 for a slot outside 0 .. R - 1); rows of dh that
 * no slot names are left as they were.  The slots of a plan name each row
 * once; of a row that several name each element is that of one of them (which
 * one may differ from element to element and from call to call), while their
 * dweights are right.
 */
typedef struct {
  int64_t dtype, T, D, R, k;
  const void *dout;
  int64_t ldd;
  const void *h;
  int64_t ldh;
  const int32_t *slots;
  const float *weights;
  void *dh;
  int64_t ldg;
  float *dweights;
} tgemm_expert_combine_backward_args;
TGEMM_API int expert_combine_backward(const tgemm_expert_combine_backward_args *args, hipStream_t stream);

/*
 * Layer norm over rows of N values: y = (x - mean) * rstd * weight + bias with
 * mean = sum(x) / N and rstd = 1 / sqrt(sum((x - mean)^2) / N + eps).
 *
 *   x, y     M x N of type dtype (BF16, F16 or F32); y may be x itself (same
 *            pointer and stride)
 *   weight, bias   N values of type wdtype (dtype or F32), or NULL: ones, zeros
 *   mean, rstd     M binary32 each, for the backward pass, or NULL
 * Sums are binary32, the variance's over differences from the mean, and lose no
 * digits as N grows; they overflow where the formula's own sums leave binary32 (values
 * past 2^127 / N or so, differences past 2^63 / sqrt(N)).  Binary32 tensors are
 * 16-byte aligned too, with strides that are multiples of 8.
 * N >= 8; eps finite and not negative (0: a row of equal values gives NaN or
 * infinity, as the formula does).
 */
typedef struct {
  int64_t dtype, wdtype, M, N;
  const void *x;
  int64_t ldx;
  const void *weight;
  const void *bias;
  double eps;
  void *y;
  int64_t ldy;
  float *mean;
  float *rstd;
} tgemm_layer_norm_args;
TGEMM_API int layer_norm(const tgemm_layer_norm_args *args, hipStream_t stream);

/*
 * Its gradients.  With g = dy * weight and h = (x - mean) * rstd:
 *   dx = rstd * (g - mean(g) - h * mean(g * h)) + residual
 *   dweight = column sums of dy * h, dbias = column sums of dy (type wdtype;
 *   either may be NULL; M = 0: zeros)
 * mean, rstd: as layer_norm gave them.  residual (M x N of dtype, or NULL): a
 * gradient that reaches x another way.  dx may be dy, x or residual itself
 * (same pointer and stride).
 * workspace: tgemm_layer_norm_backward_workspace_bytes(M, N) bytes, 16-byte
 * aligned; its sums are added in a fixed order.
 */
typedef struct {
  int64_t dtype, wdtype, M, N;
  const void *dy;
  int64_t ldd;
  const void *x;
  int64_t ldx;
  const void *weight;
  const float *mean;
  const float *rstd;
  const void *residual;
  int64_t ldr;
  void *dx;
  int64_t ldo;
  void *dweight;
  void *dbias;
  void *workspace;
  uint64_t workspace_bytes;
} tgemm_layer_norm_backward_args;
TGEMM_API int layer_norm_backward(const tgemm_layer_norm_backward_args *args, hipStream_t stream);
TGEMM_API uint64_t tgemm_layer_norm_backward_workspace_bytes(int64_t M, int64_t N);

/*
 * MXFP4, as gemm_mxfp4_nt takes it (tgemm.h): OCP E2M1 elements, two a byte
 * (element 2 i in the low nibble of byte i), one e8m0 scale byte per 32
 * consecutive elements of a row.  Rows of element bytes are 16-byte aligned,
 * ld bytes apart (a multiple of 16); scales are packed, in any alignment.
 *
 * Quantisation of x (M x N of type dtype: BF16, F16 or F32) along its rows,
 * along its columns, or both in one read of it:
 *   q   M x N / 2 bytes, scales M x N / 32: x's rows (or NULL, both)
 *   qt  N x P / 2 bytes, scalest N x P / 32, P = M rounded up to 32: x's
 *       columns, as rows, zeros behind the M values (or NULL, both)
 * A block's scale 2^e is the least power of two with max|x| <= 6 * 2^e, e
 * clamped to -127 .. 127 (-127 for zeros), stored as e + 127; an element is
 * x * 2^-e rounded once, to nearest even, its sign kept (zeros' too).  A block
 * that holds an infinity or a NaN has the scale byte 255 (a NaN: every product
 * with it is one) and elements 0.
 * N % 32 == 0 with q, N % 8 == 0 without.
 */
typedef struct {
  int64_t dtype, M, N;
  const void *x;
  int64_t ldx;
  void *q;
  int64_t ldq;
  void *scales;
  void *qt;
  int64_t ldqt;
  void *scalest;
} tgemm_quantize_mxfp4_args;
TGEMM_API int quantize_mxfp4(const tgemm_quantize_mxfp4_args *args, hipStream_t stream);

/*
 * What MXFP4 rows stand for: out[m][n] = element * 2^(scale - 127), M x N of
 * type dtype; NaN where the scale byte is 255.  BF16 and F32 hold every value
 * below 2^128 exactly, F16 rounds to nearest even; what is past the type's
 * largest value is infinite.  (Quantised, that can be a finite number: from
 * 1.75 * 2^127 on an element rounds to 4 * 2^126.)  N % 32 == 0.
 */
typedef struct {
  int64_t dtype, M, N;
  const void *q;
  int64_t ldq;
  const void *scales;
  void *out;
  int64_t ldo;
} tgemm_dequantize_mxfp4_args;
TGEMM_API int dequantize_mxfp4(const tgemm_dequantize_mxfp4_args *args, hipStream_t stream);

/*
 * gemm_epilogue on MXFP4 operands: C = act(Z) + residual, Z = A . B^T + bias,
 * A M x K and B N x K as above (lda, ldb in bytes), C, bias, residual and
 * preact of type dtype (BF16 or F16).  K % 32 == 0.
 * workspace: for a K split, tgemm_mxfp4_workspace_bytes(M, N, K) bytes,
 * 16-byte aligned; with less, or NULL, there is none.
 * tgemm_ffn_set_tile: 256 x 256 (K % 256 == 0, scales on dwords), 128 x 128, 64 x 64
 * or 16 x 16 here and in gemm_mxfp4_grouped; TGEMM_EINVAL otherwise.
 * Limits: 256 lda < 2^31 and 256 ldb < 2^31; gated, (N / 2 + 256) ldb < 2^31.
 */
typedef struct {
  int64_t dtype, M, N, K;
  const void *A;
  int64_t lda;
  const void *scale_A;
  const void *B;
  int64_t ldb;
  const void *scale_B;
  const void *bias;
  const void *residual;
  int64_t ldr;
  void *preact;
  int64_t ldp;
  void *C;
  int64_t ldc;
  int64_t act;
  void *workspace;
  uint64_t workspace_bytes;
} tgemm_mxfp4_epilogue_args;
TGEMM_API int gemm_mxfp4_epilogue(const tgemm_mxfp4_epilogue_args *args, hipStream_t stream);
TGEMM_API uint64_t tgemm_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * gemm_grouped on MXFP4 operands: for each row r of group e, C[r] = act(A[s] .
 * B_e^T + bias_e) with s = rows[r], or r if rows is NULL.  A and its scales
 * have src_rows rows (R if rows is NULL); an s outside them reads zeros.  B_e
 * is N x K at B + e stride_b bytes (a multiple of 16), its scales at scale_B +
 * e stride_sb bytes.
 * Limits: with rows, src_rows lda < 2^31; else 256 lda < 2^31; B_e as in
 * gemm_mxfp4_epilogue.
 */
typedef struct {
  int64_t dtype, R, N, K, groups;
  const int32_t *offsets;
  const int32_t *rows;
  int64_t src_rows;
  const void *A;
  int64_t lda;
  const void *scale_A;
  const void *B;
  int64_t ldb, stride_b;
  const void *scale_B;
  int64_t stride_sb;
  const void *bias;
  void *preact;
  int64_t ldp;
  void *C;
  int64_t ldc;
  int64_t act;
} tgemm_mxfp4_grouped_args;
TGEMM_API int gemm_mxfp4_grouped(const tgemm_mxfp4_grouped_args *args, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif
