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
cudaError_t few_rows_ce(const CeArgs& a, float2* ms, float* sums, float* zy, cudaStream_t s);

size_t linear_bwd_workspace(int M, int N, int K, int dtype);
cudaError_t linear_bwd(int dtype, const void* dout, const void* A, const void* W, void* dA, void* dW, float* dbias,
                       int M, int N, int K, void* ws, int* status, int num_sms, cudaStream_t s);

}  // namespace jepa
