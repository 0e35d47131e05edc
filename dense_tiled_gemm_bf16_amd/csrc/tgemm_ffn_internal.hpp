// Internal interface between the front end of libtgemm_ffn.so
// (tgemm_ffn_abi.cpp) and its gfx950 kernels.  Not installed, not part of
// the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace tgemm {
namespace ffn {

// The activations, as TGEMM_ACT_* in include/tgemm_ffn.h.
enum Act : int { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4, kSwiglu = 5, kGeglu = 6 };
inline bool is_gated(int act) { return act == kSwiglu || act == kGeglu; }

// A validated product with an epilogue, dense (groups == 0) or grouped.
// N counts the product's columns; a gated activation leaves N / 2 of them.
struct Gemm {
  int dtype;  // 0 bf16, 1 fp16
  bool trans_a, trans_b;
  int64_t M, N, K;  // grouped: M is the rows the groups may take
  const void *A;
  int64_t lda;
  const void *B;
  int64_t ldb;
  const void *bias;      // N of the element type, or nullptr
  const void *residual;  // M x Nout, or nullptr
  int64_t ldr;
  void *preact;  // M x N, or nullptr
  int64_t ldp;
  void *C;
  int64_t ldc;
  int act;
  // Grouped: rows offsets[e] .. offsets[e + 1] - 1 take weight e.
  int64_t groups;
  const int32_t *offsets;
  const int32_t *rows;  // A's row of each, or nullptr (row r itself)
  int64_t src_rows;     // rows of A
  int64_t stride_b, stride_bias;
  float *ws;  // dense: room for `splits` planes of M x N sums, or nullptr
  int splits;
  hipStream_t stream;
  int cus;
  int tile_m, tile_n;  // forced tile (16 x 16: the kernel for few rows), or 0, 0
};
hipError_t launch_gemm(const Gemm &g);       // tgemm_ffn_gemm.hip
hipError_t launch_gemm_bf16(const Gemm &g, int tm, int tn);  // tgemm_ffn_gemm_bf16.hip
hipError_t launch_gemm_f16(const Gemm &g, int tm, int tn);   // tgemm_ffn_gemm_f16.hip
hipError_t launch_rows(const Gemm &g);       // tgemm_ffn_rows.hip: few rows for each weight
hipError_t launch_split_bf16(const Gemm &g);  // the K split's partial sums, then
hipError_t launch_split_f16(const Gemm &g);
hipError_t launch_join(const Gemm &g);        // tgemm_ffn_rowops.hip: their sum and the epilogue
// Splits of K for a dense product (1: none).
int epilogue_splits(bool trans_a, bool trans_b, int64_t M, int64_t N, int64_t K);
bool tile_supported(const Gemm &g, int tm, int tn);

// out[e] = X_e^T Y_e over the rows of group e: P x Q, both 16-bit.
struct GroupedTn {
  int dtype;
  int64_t R, P, Q, groups;
  const void *X;
  int64_t ldx;
  const void *Y;
  int64_t ldy;
  const int32_t *offsets;
  void *out;  // groups x P x Q, packed
  hipStream_t stream;
  int cus;
  int tile_m, tile_n;
};
hipError_t launch_grouped_tn(const GroupedTn &g);
hipError_t launch_tn_bf16(const GroupedTn &g, int tm, int tn);
hipError_t launch_tn_f16(const GroupedTn &g, int tm, int tn);

// dZ = dC * act'(Z) and its column sums (per group where groups > 0).
struct ActGrad {
  int dtype;
  int64_t M, N;  // N: columns of Z and dZ
  const void *dout;
  int64_t ldd;
  const void *preact;
  int64_t ldp;
  int act;
  void *dz;  // nullptr with kNone
  int64_t ldz;
  void *dbias;  // groups (or 1) x N of the element type, or nullptr
  int64_t groups;
  const int32_t *offsets;
  float *ws;  // act_grad_chunks() x N sums; unused without dbias
  hipStream_t stream;
};
constexpr int kGradRows = 64;  // rows of one workgroup's column sums
inline int64_t act_grad_chunks(int64_t M, int64_t groups) {
  return (M + kGradRows - 1) / kGradRows + (groups > M ? M : groups);
}
hipError_t launch_act_grad(const ActGrad &g);

// Routing.
struct Topk {
  int dtype;  // 0 bf16, 1 fp16, 2 fp32
  int64_t T, E;
  const void *logits;
  int64_t ld;
  const float *bias;  // E, or nullptr
  int k, score, groups, used, renorm;
  float scale;
  float *weights;  // T x k
  int32_t *ids;    // T x k
  hipStream_t stream;
};
hipError_t launch_topk(const Topk &t);

struct TopkGrad {
  int dtype;
  int64_t T, E;
  const void *logits;
  int64_t ld;
  const int32_t *ids;
  const float *dweights;
  int k, score, renorm;
  float scale;
  void *dlogits;
  int64_t ldo;
  hipStream_t stream;
};
hipError_t launch_topk_grad(const TopkGrad &t);

struct Plan {
  int64_t T, E;
  int k;
  const int32_t *ids;
  int32_t *offsets, *rows, *slots;
  int32_t *ws;
  hipStream_t stream;
};
constexpr int kPlanChunk = 4096;  // choices of one workgroup
inline int64_t plan_ws_ints(int64_t n, int64_t E) {
  const int64_t chunks = (n + kPlanChunk - 1) / kPlanChunk;
  return chunks > 1 ? chunks * E : 0;
}
hipError_t launch_plan(const Plan &p);

// Moving rows between tokens and experts.
struct Gather {
  int64_t R, D, src_rows;
  const void *x;
  int64_t ldx;
  const int32_t *rows;
  void *out;
  int64_t ldo;
  hipStream_t stream;
};
hipError_t launch_gather(const Gather &g);

struct Combine {
  int dtype;
  int64_t T, D, R;
  int k;
  const void *h;
  int64_t ldh;
  const int32_t *slots;
  const float *weights;  // or nullptr: ones
  const void *residual;
  int64_t ldr;
  void *out;
  int64_t ldo;
  hipStream_t stream;
};
hipError_t launch_combine(const Combine &c);

struct CombineGrad {
  int dtype;
  int64_t T, D, R;
  int k;
  const void *dout;
  int64_t ldd;
  const void *h;
  int64_t ldh;
  const int32_t *slots;
  const float *weights;
  void *dh;
  int64_t ldg;
  float *dweights;
  hipStream_t stream;
};
hipError_t launch_combine_grad(const CombineGrad &c);

}  // namespace ffn
}  // namespace tgemm
