// C entry points of the training operators: argument checks, then the kernels.
// Everything a call can refuse is refused here, before anything is enqueued.
#include <initializer_list>

#include "api_internal.h"
#include "train.h"

using namespace jepa;

namespace {

constexpr int kMaxSize = 1 << 24;   // of every row count and width

bool bad_dtype(int dt) { return dt < 0 || dt > 2; }
size_t elem_size(int dt) { return dt == DTYPE_F32 ? 4 : 2; }
// Device pointers have to be aligned to their element.
bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

jepa_status cuda_result(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return JEPA_OK;
  return api_fail(JEPA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

jepa_status device_of_call(int** status, int* sms) {
  const jepa_status st = api_ops_status(status);
  if (st != JEPA_OK) return st;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return cuda_result(e, "device query");
}

jepa_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return JEPA_OK;
  if (ws == nullptr) return api_fail(JEPA_ERR_ARG, "workspace is NULL (%zu bytes needed)", need);
  if (misaligned(ws, 256)) return api_fail(JEPA_ERR_ARG, "workspace must be 256-byte aligned");
  if (bytes < need) return api_fail(JEPA_ERR_ARG, "workspace holds %zu bytes, %zu needed", bytes, need);
  return JEPA_OK;
}

// Matrices of products start on 16 bytes, as TMA wants.
bool matrix_misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (misaligned(p, 16)) return true;
  return false;
}
jepa_status bad_matrix() { return api_fail(JEPA_ERR_ARG, "matrices must be 16-byte aligned"); }

bool bad_rows(int m) { return m < 0 || m > kMaxSize; }
bool bad_width(int n) { return n < 1 || n > kMaxSize; }

#define ARG_TRY(expr)                  \
  do {                                 \
    const jepa_status s_ = (expr);     \
    if (s_ != JEPA_OK) return s_;      \
  } while (0)

// ----------------------------------------------------------------------------- layer norm
jepa_status check_ln(int rows, int dim, int x_dtype, int y_dtype) {
  if (bad_rows(rows) || dim < 1 || dim > (1 << 20))
    return api_fail(JEPA_ERR_ARG, "rows %d (0 .. 2^24) / dim %d (1 .. 2^20)", rows, dim);
  if (bad_dtype(x_dtype) || bad_dtype(y_dtype)) return api_fail(JEPA_ERR_ARG, "dtype %d / %d", x_dtype, y_dtype);
  if (x_dtype != y_dtype && x_dtype != DTYPE_F32)
    return api_fail(JEPA_ERR_UNSUPPORTED, "x dtype %d with y dtype %d (equal, or x in fp32)", x_dtype, y_dtype);
  return JEPA_OK;
}

// ----------------------------------------------------------------------------- products
jepa_status check_ce(int M, int D, int V, int dtype, float smoothing) {
  if (bad_rows(M) || bad_width(D) || bad_width(V))
    return api_fail(JEPA_ERR_ARG, "M %d (0 .. 2^24), D %d, V %d (1 .. 2^24)", M, D, V);
  if (bad_dtype(dtype)) return api_fail(JEPA_ERR_ARG, "dtype %d", dtype);
  if (!(smoothing >= 0.f && smoothing < 1.f)) return api_fail(JEPA_ERR_ARG, "smoothing %g (0 <= s < 1)", smoothing);
  return JEPA_OK;
}
jepa_status check_ffn(int M, int D, int F, int dtype, int act) {
  if (bad_rows(M) || bad_width(D) || bad_width(F))
    return api_fail(JEPA_ERR_ARG, "M %d (0 .. 2^24), D %d, F %d (1 .. 2^24)", M, D, F);
  if (bad_dtype(dtype)) return api_fail(JEPA_ERR_ARG, "dtype %d", dtype);
  if (act != ACT_SILU && act != ACT_GELU) return api_fail(JEPA_ERR_ARG, "act %d (JEPA_GATE_SILU or JEPA_GATE_GELU)", act);
  return JEPA_OK;
}

}  // namespace

extern "C" {

// ============================================================================= layer norm
jepa_status jepa_layernorm_fwd(const void* x, const float* w, const float* b, void* y, float* mean, float* rstd,
                               int rows, int dim, int x_dtype, int y_dtype, float eps, void* stream) {
  ARG_TRY(check_ln(rows, dim, x_dtype, y_dtype));
  if (!(eps > 0.f)) return api_fail(JEPA_ERR_ARG, "eps must be > 0");
  if (rows == 0) return JEPA_OK;
  if (!x || !w || !b || !y) return api_fail(JEPA_ERR_ARG, "NULL buffer");
  if (misaligned(x, elem_size(x_dtype)) || misaligned(y, elem_size(y_dtype)) || misaligned(w, 4) || misaligned(b, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element");
  return cuda_result(layernorm_fwd(x_dtype, y_dtype, x, w, b, y, mean, rstd, rows, dim, eps, (cudaStream_t)stream),
                     "layernorm_fwd");
}

size_t jepa_layernorm_bwd_workspace_bytes(int rows, int dim) {
  if (bad_rows(rows) || dim < 1 || dim > (1 << 20)) return 0;
  return layernorm_bwd_workspace(rows, dim);
}

jepa_status jepa_layernorm_bwd(const void* dy, const void* x, const float* w, const float* mean, const float* rstd,
                               const void* residual, void* dx, float* dw, float* db, int rows, int dim, int x_dtype,
                               int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  ARG_TRY(check_ln(rows, dim, x_dtype, y_dtype));
  if (rows > 0 && (!dy || !x || !w || !mean || !rstd || !dx)) return api_fail(JEPA_ERR_ARG, "NULL buffer");
  const size_t ex = elem_size(x_dtype), ey = elem_size(y_dtype);
  if (misaligned(dy, ey) || misaligned(x, ex) || misaligned(residual, ex) || misaligned(dx, ex) || misaligned(w, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(dw, 4) || misaligned(db, 4))
    return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element");
  ARG_TRY(check_ws(workspace, workspace_bytes, layernorm_bwd_workspace(rows, dim)));
  const LnBwdArgs a{dy, x, residual, w, mean, rstd, dx, dw, db, (float*)workspace, rows, dim};
  return cuda_result(layernorm_bwd(x_dtype, y_dtype, a, (cudaStream_t)stream), "layernorm_bwd");
}

// ============================================================================= softmax cross entropy
size_t jepa_linear_ce_workspace_bytes(int M, int D, int V, int dtype, int backward) {
  if (bad_rows(M) || bad_width(D) || bad_width(V) || bad_dtype(dtype)) return 0;
  return linear_ce_workspace(M, D, V, dtype, backward != 0);
}

jepa_status jepa_linear_ce_fwd(const void* x, const void* W, const float* bias, const int64_t* labels, float* loss,
                               float* lse, int M, int D, int V, int dtype, int64_t ignore_index, float smoothing,
                               void* workspace, size_t workspace_bytes, void* stream) {
  ARG_TRY(check_ce(M, D, V, dtype, smoothing));
  if (M == 0) return JEPA_OK;
  if (!x || !W || !labels || !lse) return api_fail(JEPA_ERR_ARG, "NULL buffer");
  if (matrix_misaligned({x, W})) return bad_matrix();
  if (misaligned(bias, 4) || misaligned(labels, 8) || misaligned(loss, 4) ||
      misaligned(lse, 4))
    return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element");
  ARG_TRY(check_ws(workspace, workspace_bytes, linear_ce_workspace(M, D, V, dtype, false)));
  CeArgs a{x, W, bias, labels, M, D, V, dtype, (long)ignore_index, smoothing, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(linear_ce_fwd(a, loss, lse, workspace, (cudaStream_t)stream), "linear_ce_fwd");
}

jepa_status jepa_linear_ce_bwd(const void* x, const void* W, const float* bias, const int64_t* labels, const float* lse,
                               const float* dloss, void* dx, void* dW, float* dbias, int M, int D, int V, int dtype,
                               int64_t ignore_index, float smoothing, void* workspace, size_t workspace_bytes,
                               void* stream) {
  ARG_TRY(check_ce(M, D, V, dtype, smoothing));
  if (M > 0 && (!x || !W || !labels || !lse || !dloss)) return api_fail(JEPA_ERR_ARG, "NULL buffer");
  if (!dx && !dW && !dbias) return api_fail(JEPA_ERR_ARG, "no gradient asked for (dx, dW and dbias are NULL)");
  if (matrix_misaligned({x, W, dx, dW})) return bad_matrix();
  if (misaligned(bias, 4) || misaligned(labels, 8) || misaligned(lse, 4) || misaligned(dloss, 4) || misaligned(dbias, 4))
    return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element");
  if (M > 0) ARG_TRY(check_ws(workspace, workspace_bytes, linear_ce_workspace(M, D, V, dtype, true)));
  CeArgs a{x, W, bias, labels, M, D, V, dtype, (long)ignore_index, smoothing, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(linear_ce_bwd(a, lse, dloss, dx, dW, dbias, workspace, (cudaStream_t)stream), "linear_ce_bwd");
}

// ============================================================================= gated feed-forward
size_t jepa_gated_ffn_workspace_bytes(int M, int D, int F, int dtype, int backward) {
  if (bad_rows(M) || bad_width(D) || bad_width(F) || bad_dtype(dtype)) return 0;
  return gated_ffn_workspace(M, D, F, dtype, backward != 0);
}

jepa_status jepa_gated_ffn_fwd(const void* x, const void* Wg, const void* Wu, const float* bg, const float* bu, void* h,
                               int M, int D, int F, int dtype, int act, void* workspace, size_t workspace_bytes,
                               void* stream) {
  ARG_TRY(check_ffn(M, D, F, dtype, act));
  if (M == 0) return JEPA_OK;
  if (!x || !Wg || !Wu || !h) return api_fail(JEPA_ERR_ARG, "NULL buffer");
  if (matrix_misaligned({x, Wg, Wu, h})) return bad_matrix();
  if (misaligned(bg, 4) || misaligned(bu, 4))
    return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element");
  ARG_TRY(check_ws(workspace, workspace_bytes, gated_ffn_workspace(M, D, F, dtype, false)));
  FfnArgs a{x, Wg, Wu, bg, bu, M, D, F, dtype, act, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(gated_ffn_fwd(a, h, workspace, (cudaStream_t)stream), "gated_ffn_fwd");
}

jepa_status jepa_gated_ffn_bwd(const void* dh, const void* x, const void* Wg, const void* Wu, const float* bg,
                               const float* bu, void* dx, void* dWg, void* dWu, float* dbg, float* dbu, int M, int D,
                               int F, int dtype, int act, void* workspace, size_t workspace_bytes, void* stream) {
  ARG_TRY(check_ffn(M, D, F, dtype, act));
  if (M > 0 && (!dh || !x || !Wg || !Wu)) return api_fail(JEPA_ERR_ARG, "NULL buffer");
  if (!dx && !dWg && !dWu && !dbg && !dbu) return api_fail(JEPA_ERR_ARG, "no gradient asked for (every output is NULL)");
  if (matrix_misaligned({dh, x, Wg, Wu, dx, dWg, dWu})) return bad_matrix();
  if (misaligned(bg, 4) || misaligned(bu, 4) || misaligned(dbg, 4) || misaligned(dbu, 4))
    return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element");
  if (M > 0) ARG_TRY(check_ws(workspace, workspace_bytes, gated_ffn_workspace(M, D, F, dtype, true)));
  FfnArgs a{x, Wg, Wu, bg, bu, M, D, F, dtype, act, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(gated_ffn_bwd(a, dh, dx, dWg, dWu, dbg, dbu, workspace, (cudaStream_t)stream), "gated_ffn_bwd");
}

// ============================================================================= linear layer backward
size_t jepa_linear_bwd_workspace_bytes(int M, int N, int K, int dtype) {
  if (bad_rows(M) || bad_width(N) || bad_width(K) || bad_dtype(dtype)) return 0;
  return linear_bwd_workspace(M, N, K, dtype);
}

jepa_status jepa_linear_bwd(const void* dout, const void* A, const void* W, void* dA, void* dW, float* dbias, int M,
                            int N, int K, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (bad_rows(M) || bad_width(N) || bad_width(K))
    return api_fail(JEPA_ERR_ARG, "M %d (0 .. 2^24), N %d, K %d (1 .. 2^24)", M, N, K);
  if (bad_dtype(dtype)) return api_fail(JEPA_ERR_ARG, "dtype %d", dtype);
  if (!dA && !dW && !dbias) return api_fail(JEPA_ERR_ARG, "no gradient asked for (dA, dW and dbias are NULL)");
  if (M > 0 && (!dout || (dA && !W) || (dW && !A))) return api_fail(JEPA_ERR_ARG, "NULL buffer");
  if (matrix_misaligned({dout, A, W, dA, dW})) return bad_matrix();
  if (misaligned(dbias, 4)) return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element");
  if (M > 0) ARG_TRY(check_ws(workspace, workspace_bytes, linear_bwd_workspace(M, N, K, dtype)));
  int* st = nullptr;
  int sms = 0;
  ARG_TRY(device_of_call(&st, &sms));
  return cuda_result(linear_bwd(dtype, dout, A, W, dA, dW, dbias, M, N, K, workspace, st, sms, (cudaStream_t)stream),
                     "linear_bwd");
}

}  // extern "C"
