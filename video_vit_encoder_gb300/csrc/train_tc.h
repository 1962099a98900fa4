// The tensor-core forms of the training operators (train_tc.cu): which calls
// they take, their workspaces, and the calls.
#pragma once
#include "train.h"

namespace jepa {

// Whether every matrix starts on 16 bytes and has rows of 16 bytes, as TMA
// wants; a null output is no hindrance.
bool linear_ce_tc_ok(const CeArgs& a, const void* dx, const void* dw);
bool gated_ffn_tc_ok(const FfnArgs& a, const void* h, const void* dx, const void* dwg, const void* dwu);
bool linear_bwd_tc_ok(int dtype, const void* dout, const void* A, const void* W, const void* dA, const void* dW, int N,
                      int K);

size_t linear_ce_tc_workspace(int M, int D, int V, bool backward);
cudaError_t linear_ce_fwd_tc(const CeArgs& a, float* loss, float* lse, void* ws, cudaStream_t s);
cudaError_t linear_ce_bwd_tc(const CeArgs& a, const float* lse, const float* dloss, void* dx, void* dw, float* dbias,
                             void* ws, cudaStream_t s);
size_t gated_ffn_tc_workspace(int M, int D, int F, bool backward);
cudaError_t gated_ffn_fwd_tc(const FfnArgs& a, void* h, cudaStream_t s);
cudaError_t gated_ffn_bwd_tc(const FfnArgs& a, const void* dh, void* dx, void* dwg, void* dwu, float* dbg, float* dbu,
                             void* ws, cudaStream_t s);
size_t linear_bwd_tc_workspace(int M, int N, int K);
cudaError_t linear_bwd_tc(int dtype, const void* dout, const void* A, const void* W, void* dA, void* dW, float* dbias,
                          int M, int N, int K, void* ws, int* status, int num_sms, cudaStream_t s);

}  // namespace jepa
