// Declarations of the training operators: layer norm with its backward pass,
// the gated feed-forward, the linear layer's backward pass and the softmax
// cross entropy of a linear classifier.
#pragma once
#include "internal.h"

namespace jepa {

// ----------------------------------------------------------------------------- layer norm (layernorm_fwd.cu, layernorm_bwd.cu)
// x_dtype / y_dtype: equal, or x in fp32 and y in a 16-bit type.
cudaError_t layernorm_fwd(int x_dtype, int y_dtype, const void* x, const float* w, const float* b, void* y, float* mean,
                          float* rstd, long rows, int dim, float eps, cudaStream_t s);
size_t layernorm_bwd_workspace(long rows, int dim);
struct LnBwdArgs {
  const void *dy, *x, *res;       // res or null
  const float *w, *mean, *rstd;
  void* dx;
  float *dw, *db, *ws;            // dw, db or null
  long rows;
  int dim;
};
cudaError_t layernorm_bwd(int x_dtype, int y_dtype, const LnBwdArgs& a, cudaStream_t s);
cudaError_t layernorm_bwd_f32(const LnBwdArgs& a, cudaStream_t s);
cudaError_t layernorm_bwd_f32_f16(const LnBwdArgs& a, cudaStream_t s);
cudaError_t layernorm_bwd_f32_bf16(const LnBwdArgs& a, cudaStream_t s);
cudaError_t layernorm_bwd_f16(const LnBwdArgs& a, cudaStream_t s);
cudaError_t layernorm_bwd_bf16(const LnBwdArgs& a, cudaStream_t s);

// ----------------------------------------------------------------------------- operators (train_ops.cu)
enum GateAct : int { ACT_SILU = 0, ACT_GELU = 1 };

struct CeArgs {
  const void* x;          // T [M, D]
  const void* w;          // T [V, D]
  const float* bias;      // [V] or null
  const int64_t* labels;  // [M]
  int M, D, V, dtype;
  long ignore_index;
  float smoothing;
  int* status;
  int num_sms;
};
size_t linear_ce_workspace(int M, int D, int V, int dtype, bool backward);
cudaError_t linear_ce_fwd(const CeArgs& a, float* loss, float* lse, void* ws, cudaStream_t s);
cudaError_t linear_ce_bwd(const CeArgs& a, const float* lse, const float* dloss, void* dx, void* dw, float* dbias,
                          void* ws, cudaStream_t s);

// Distillation from a teacher's top logits: the classifier's arguments (labels,
// ignore_index, smoothing unused) and the teacher's.
struct DistillArgs {
  CeArgs ce;
  const void* top;       // top_dtype [M, K]
  const int64_t* ids;    // [M, K]
  int K, top_dtype;
  long ignore_index;
  float tau;
};
size_t linear_distill_workspace(int M, int D, int V, int K, int dtype, bool backward);
cudaError_t linear_distill_fwd(const DistillArgs& a, float* loss, float* lse, float* z, void* ws, cudaStream_t s);
cudaError_t linear_distill_bwd(const DistillArgs& a, const float* lse, const float* z, const float* dloss, void* dx,
                               void* dw, float* dbias, void* ws, cudaStream_t s);
// Its kernels beside the products (distill.cu).
// The rows' entries in the order in which the product's epilogue takes them
// (tg::Hits), which goes over `runs` runs of `run` column tiles, and 0 as z of those
// that are out.
cudaError_t distill_hits(const DistillArgs& a, int run, int runs, uint32_t* hits, uint16_t* starts, float* z, cudaStream_t s);
// loss and lse of each row from its statistics in parts [parts][M] and the entries' z.
cudaError_t distill_join(const DistillArgs& a, const float2* ms, int parts, const float* z, float* loss, float* lse,
                         cudaStream_t s);
// Of each row: label (0, or -1 where it has no gradient) and dloss tau; of each
// entry its class, or -1 (out, or joined with an earlier one of its class), and probability.
// acc [2][V], or null: set to 0.
cudaError_t distill_teacher(const DistillArgs& a, const float* dloss, int64_t* label, float* dl, int* cls, float* prob,
                            long long* acc, cudaStream_t s);
// The entries' dz, written over those of the columns v0 .. v0 + n.
struct DistillPut {
  const int* cls;
  const float *prob, *z, *lse, *dl;
  int M, K, v0, n, V;
  float z_scale, factor;      // log2 e / tau; what dz is multiplied by
  const float* unit;          // on the device: what dl is divided by (acc: always; 16-bit dz: also)
  uint16_t* dz;               // [M][ld], fp32: planes of plane_rows rows
  long ld, plane_rows;
  long long* acc;             // [2][V] or null: gets prob dl / unit 2^shift, and what is left of that times 2^shift
  int shift;
};
cudaError_t distill_put(int dtype, const DistillPut& q, int num_sms, cudaStream_t s);

struct FfnArgs {
  const void* x;        // T [M, D]
  const void* wg;       // T [F, D]
  const void* wu;       // T [F, D]
  const float* bg;      // [F] or null
  const float* bu;      // [F] or null
  int M, D, F, dtype, act;
  int* status;
  int num_sms;
};
size_t gated_ffn_workspace(int M, int D, int F, int dtype, bool backward);
cudaError_t gated_ffn_fwd(const FfnArgs& a, void* h, void* ws, cudaStream_t s);
cudaError_t gated_ffn_bwd(const FfnArgs& a, const void* dh, void* dx, void* dwg, void* dwu, float* dbg, float* dbu,
                          void* ws, cudaStream_t s);

// The forward passes for a few rows (few_rows.cu): at most 16, of 16-byte pieces.
bool few_rows_ok(int dtype, int M, int D);
cudaError_t few_rows_gate(const FfnArgs& a, void* h, cudaStream_t s);
// Statistics of each row in parts [few_rows_ce_parts(V)][M], as the tiles leave them.
int few_rows_ce_parts(int V);
// scale: log2 e, over the temperature; a.labels and zy may be null.  e: a
// distillation's entries, whose logits are wanted, or none (top 0).
struct FewEntries {
  const int64_t* ids;   // [M, top]
  int top;
  long ignore;
  float* z;
  int blocks;
};
cudaError_t few_rows_ce(const CeArgs& a, const FewEntries& e, float2* ms, float* sums, float* zy, float scale, cudaStream_t s);

size_t linear_bwd_workspace(int M, int N, int K, int dtype);
cudaError_t linear_bwd(int dtype, const void* dout, const void* A, const void* W, void* dA, void* dW, float* dbias,
                       int M, int N, int K, void* ws, int* status, int num_sms, cudaStream_t s);

}  // namespace jepa
