// C entry points of the decoder operators: argument checks, then the kernels.
// Everything a call can refuse is refused here, before anything is enqueued.
#include <initializer_list>

#include "api_internal.h"
#include "decoder.h"
#include "train.h"

using namespace jepa;

namespace {

constexpr int kMaxSize = 1 << 24;   // of every row count and width
constexpr int kMaxTop = 1024;

bool bad_dtype(int dt) { return dt < 0 || dt > 2; }
size_t elem_size(int dt) { return dt == DTYPE_F32 ? 4 : 2; }
bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
bool any_misaligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (misaligned(p, a)) return true;
  return false;
}
bool bad_rows(int m) { return m < 0 || m > kMaxSize; }
bool bad_width(int n) { return n < 1 || n > kMaxSize; }
jepa_status bad_buffer() { return api_fail(JEPA_ERR_ARG, "a buffer is not aligned to its element"); }
jepa_status null_buffer() { return api_fail(JEPA_ERR_ARG, "NULL buffer"); }

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

#define ARG_TRY(expr)                  \
  do {                                 \
    const jepa_status s_ = (expr);     \
    if (s_ != JEPA_OK) return s_;      \
  } while (0)

// ----------------------------------------------------------------------------- embedding
jepa_status check_embedding(int n, int dim, int vocab, int table_dtype, int out_dtype, float scale) {
  if (bad_rows(n) || bad_width(dim) || bad_width(vocab))
    return api_fail(JEPA_ERR_ARG, "n %d (0 .. 2^24), dim %d, vocab %d (1 .. 2^24)", n, dim, vocab);
  if (bad_dtype(table_dtype) || bad_dtype(out_dtype))
    return api_fail(JEPA_ERR_ARG, "dtype %d / %d", table_dtype, out_dtype);
  if (out_dtype != table_dtype && out_dtype != DTYPE_F32)
    return api_fail(JEPA_ERR_UNSUPPORTED, "table dtype %d with rows of dtype %d (equal, or rows in fp32)", table_dtype,
                    out_dtype);
  if (!(scale - scale == 0.f)) return api_fail(JEPA_ERR_ARG, "scale must be finite");
  return JEPA_OK;
}

// ----------------------------------------------------------------------------- gated linear recurrence
jepa_status check_scan(int batch, int steps, int width, int dtype) {
  if (batch < 0 || steps < 0 || (long)batch * steps > kMaxSize || batch > 65535 || width < 1 || width > (1 << 20))
    return api_fail(JEPA_ERR_ARG, "batch %d (0 .. 65535), steps %d (batch x steps at most 2^24), width %d (1 .. 2^20)",
                    batch, steps, width);
  if (bad_dtype(dtype)) return api_fail(JEPA_ERR_ARG, "dtype %d", dtype);
  return JEPA_OK;
}

// ----------------------------------------------------------------------------- distillation
jepa_status check_distill(int M, int D, int V, int K, int dtype, int top_dtype, float tau) {
  if (bad_rows(M) || bad_width(D) || bad_width(V) || K < 1 || K > kMaxTop)
    return api_fail(JEPA_ERR_ARG, "M %d (0 .. 2^24), D %d, V %d (1 .. 2^24), K %d (1 .. %d)", M, D, V, K, kMaxTop);
  if (bad_dtype(dtype) || bad_dtype(top_dtype)) return api_fail(JEPA_ERR_ARG, "dtype %d / %d", dtype, top_dtype);
  if (!(tau >= 1e-3f && tau <= 1e3f)) return api_fail(JEPA_ERR_ARG, "temperature %g (0.001 .. 1000)", tau);
  return JEPA_OK;
}

}  // namespace

extern "C" {

// ============================================================================= embedding
jepa_status jepa_embedding_fwd(const int64_t* tokens, const void* table, void* out, int n, int dim, int vocab,
                               int table_dtype, int out_dtype, float scale, int64_t ignore_index, void* stream) {
  ARG_TRY(check_embedding(n, dim, vocab, table_dtype, out_dtype, scale));
  if (n == 0) return JEPA_OK;
  if (!tokens || !table || !out) return null_buffer();
  if (misaligned(tokens, 8) || misaligned(table, elem_size(table_dtype)) || misaligned(out, elem_size(out_dtype)))
    return bad_buffer();
  EmbedArgs a{tokens, n, dim, vocab, table_dtype, out_dtype, scale, (long)ignore_index, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(embedding_fwd(a, table, out, (cudaStream_t)stream), "embedding_fwd");
}

size_t jepa_embedding_bwd_workspace_bytes(int n, int dim, int vocab) {
  if (bad_rows(n) || bad_width(dim) || bad_width(vocab)) return 0;
  return embedding_bwd_workspace(n, dim, vocab);
}

jepa_status jepa_embedding_bwd(const int64_t* tokens, const void* dout, void* dtable, int n, int dim, int vocab,
                               int dout_dtype, int dtable_dtype, float scale, int64_t ignore_index, void* workspace,
                               size_t workspace_bytes, void* stream) {
  ARG_TRY(check_embedding(n, dim, vocab, dtable_dtype, dout_dtype, scale));
  if (!dtable || (n > 0 && (!tokens || !dout))) return null_buffer();
  if (misaligned(tokens, 8) || misaligned(dout, elem_size(dout_dtype)) || misaligned(dtable, elem_size(dtable_dtype)))
    return bad_buffer();
  ARG_TRY(check_ws(workspace, workspace_bytes, embedding_bwd_workspace(n, dim, vocab)));
  EmbedArgs a{tokens, n, dim, vocab, dtable_dtype, dout_dtype, scale, (long)ignore_index, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(embedding_bwd(a, dout, dtable, workspace, (cudaStream_t)stream), "embedding_bwd");
}

// ============================================================================= gated linear recurrence
jepa_status jepa_gated_scan_fwd(const void* gv, const float* h0, const int32_t* lengths, void* h, float* last,
                                float* states, int batch, int steps, int width, int dtype, void* stream) {
  ARG_TRY(check_scan(batch, steps, width, dtype));
  if (batch == 0) return JEPA_OK;
  if (steps > 0 && (!gv || !h)) return null_buffer();
  if (any_misaligned({gv, h}, elem_size(dtype)) || any_misaligned({h0, lengths, last, states}, 4)) return bad_buffer();
  ScanArgs a{gv, lengths, batch, steps, width, dtype, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(gated_scan_fwd(a, h0, h, last, states, (cudaStream_t)stream), "gated_scan_fwd");
}

jepa_status jepa_gated_scan_bwd(const void* dh, const void* gv, const float* states, const int32_t* lengths,
                                const float* dlast, void* dgv, float* dh0, int batch, int steps, int width, int dtype,
                                void* stream) {
  ARG_TRY(check_scan(batch, steps, width, dtype));
  if (batch == 0) return JEPA_OK;
  if (steps > 0 && (!dh || !gv || !states || !dgv)) return null_buffer();
  if (any_misaligned({dh, gv, dgv}, elem_size(dtype)) || any_misaligned({states, lengths, dlast, dh0}, 4))
    return bad_buffer();
  ScanArgs a{gv, lengths, batch, steps, width, dtype, nullptr, 0};
  ARG_TRY(device_of_call(&a.status, &a.num_sms));
  return cuda_result(gated_scan_bwd(a, dh, states, dlast, dgv, dh0, (cudaStream_t)stream), "gated_scan_bwd");
}

jepa_status jepa_selftest_scan_wait_timeout(int timeout_us, void* stream) {
  if (timeout_us < 1 || timeout_us > 5000000) return api_fail(JEPA_ERR_ARG, "timeout_us %d (1 .. 5e6)", timeout_us);
  int* status = nullptr;
  ARG_TRY(api_ops_status(&status));
  const uint64_t limit_ns = (uint64_t)timeout_us * 1000ull;
  ARG_TRY(cuda_result(gated_scan_wait_selftest(status, limit_ns, (cudaStream_t)stream), "gated_scan_wait_selftest"));
  return jepa_ops_sync(stream);
}

// ============================================================================= distillation
size_t jepa_linear_distill_workspace_bytes(int M, int D, int V, int K, int dtype, int backward) {
  if (bad_rows(M) || bad_width(D) || bad_width(V) || K < 1 || K > kMaxTop || bad_dtype(dtype)) return 0;
  return linear_distill_workspace(M, D, V, K, dtype, backward != 0);
}

jepa_status jepa_linear_distill_fwd(const void* x, const void* W, const float* bias, const void* top_logits,
                                    const int64_t* top_ids, float* loss, float* lse, float* z, int M, int D, int V,
                                    int K, int dtype, int top_dtype, int64_t ignore_index, float temperature,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  ARG_TRY(check_distill(M, D, V, K, dtype, top_dtype, temperature));
  if (M == 0) return JEPA_OK;
  if (!x || !W || !top_logits || !top_ids || !lse || !z) return null_buffer();
  if (any_misaligned({x, W}, 16)) return api_fail(JEPA_ERR_ARG, "matrices must be 16-byte aligned");
  if (any_misaligned({bias, loss, lse, z}, 4) || misaligned(top_ids, 8) || misaligned(top_logits, elem_size(top_dtype)))
    return bad_buffer();
  ARG_TRY(check_ws(workspace, workspace_bytes, linear_distill_workspace(M, D, V, K, dtype, false)));
  DistillArgs a{{x, W, bias, nullptr, M, D, V, dtype, 0, 0.f, nullptr, 0}, top_logits, top_ids, K, top_dtype,
                (long)ignore_index, temperature};
  ARG_TRY(device_of_call(&a.ce.status, &a.ce.num_sms));
  return cuda_result(linear_distill_fwd(a, loss, lse, z, workspace, (cudaStream_t)stream), "linear_distill_fwd");
}

jepa_status jepa_linear_distill_bwd(const void* x, const void* W, const float* bias, const void* top_logits,
                                    const int64_t* top_ids, const float* lse, const float* z, const float* dloss,
                                    void* dx, void* dW, float* dbias, int M, int D, int V, int K, int dtype,
                                    int top_dtype, int64_t ignore_index, float temperature, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  ARG_TRY(check_distill(M, D, V, K, dtype, top_dtype, temperature));
  if (M > 0 && (!x || !W || !top_logits || !top_ids || !lse || !z || !dloss)) return null_buffer();
  if (!dx && !dW && !dbias) return api_fail(JEPA_ERR_ARG, "no gradient asked for (dx, dW and dbias are NULL)");
  if (any_misaligned({x, W, dx, dW}, 16)) return api_fail(JEPA_ERR_ARG, "matrices must be 16-byte aligned");
  if (any_misaligned({bias, lse, z, dloss, dbias}, 4) || misaligned(top_ids, 8) ||
      misaligned(top_logits, elem_size(top_dtype)))
    return bad_buffer();
  if (M > 0) ARG_TRY(check_ws(workspace, workspace_bytes, linear_distill_workspace(M, D, V, K, dtype, true)));
  DistillArgs a{{x, W, bias, nullptr, M, D, V, dtype, 0, 0.f, nullptr, 0}, top_logits, top_ids, K, top_dtype,
                (long)ignore_index, temperature};
  ARG_TRY(device_of_call(&a.ce.status, &a.ce.num_sms));
  return cuda_result(linear_distill_bwd(a, lse, z, dloss, dx, dW, dbias, workspace, (cudaStream_t)stream),
                     "linear_distill_bwd");
}

}  // extern "C"
