// Layer norm backward: the workspace and the choice of types (layernorm_bwd.cuh
// has the kernels, one translation unit per kind of types).
#include "train.h"

namespace jepa {

size_t layernorm_bwd_workspace(long rows, int dim) {
  // two sums per column for each block, of which there are at most two per SM
  const long strips = rows < 2 * 152 ? rows : 2 * 152;
  return sizeof(float) * 2 * (size_t)dim * strips;
}

cudaError_t layernorm_bwd(int x_dtype, int y_dtype, const LnBwdArgs& a, cudaStream_t s) {
  if (a.rows == 0) {
    cudaError_t e = a.dw != nullptr ? cudaMemsetAsync(a.dw, 0, sizeof(float) * (size_t)a.dim, s) : cudaSuccess;
    if (e == cudaSuccess && a.db != nullptr) e = cudaMemsetAsync(a.db, 0, sizeof(float) * (size_t)a.dim, s);
    return e;
  }
  if (x_dtype == DTYPE_F32) {
    if (y_dtype == DTYPE_F32) return layernorm_bwd_f32(a, s);
    return y_dtype == DTYPE_F16 ? layernorm_bwd_f32_f16(a, s) : layernorm_bwd_f32_bf16(a, s);
  }
  return x_dtype == DTYPE_F16 ? layernorm_bwd_f16(a, s) : layernorm_bwd_bf16(a, s);
}

}  // namespace jepa
