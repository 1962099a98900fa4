// Declarations of the decoder operators: embedding of tokens and the gated
// linear recurrence (the distillation is in train.h, beside the cross entropy).
#pragma once
#include "internal.h"

namespace jepa {

// ----------------------------------------------------------------------------- embedding (embedding.cu)
struct EmbedArgs {
  const int64_t* tokens;   // [n]
  int n, dim, vocab;
  int table_dtype, out_dtype;
  float scale;
  long ignore_index;
  int* status;
  int num_sms;
};
cudaError_t embedding_fwd(const EmbedArgs& a, const void* table, void* out, cudaStream_t s);
size_t embedding_bwd_workspace(int n, int dim, int vocab);
cudaError_t embedding_bwd(const EmbedArgs& a, const void* dout, void* dtable, void* ws, cudaStream_t s);

// ----------------------------------------------------------------------------- gated linear recurrence (gated_scan.cu)
constexpr int kScanPiece = 128;   // steps from one kept state to the next
struct ScanArgs {
  const void* gv;          // [batch, steps, 2 width]
  const int* lengths;      // [batch] or null
  int batch, steps, width, dtype;
  int* status;
  int num_sms;
};
cudaError_t gated_scan_fwd(const ScanArgs& a, const float* h0, void* h, float* last, float* states, cudaStream_t s);
cudaError_t gated_scan_bwd(const ScanArgs& a, const void* dh, const float* states, const float* dlast, void* dgv,
                           float* dh0, cudaStream_t s);
// A wait of the exchange between blocks that runs out after limit_ns.
cudaError_t gated_scan_wait_selftest(int* status, uint64_t limit_ns, cudaStream_t s);

}  // namespace jepa
