#include "layernorm_bwd.cuh"

namespace jepa {
JEPA_LN_BWD_INSTANCE(float, __half, layernorm_bwd_f32_f16)
JEPA_LN_BWD_INSTANCE(float, __nv_bfloat16, layernorm_bwd_f32_bf16)
}  // namespace jepa
