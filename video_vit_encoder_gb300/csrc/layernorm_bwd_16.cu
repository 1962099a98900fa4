#include "layernorm_bwd.cuh"

namespace jepa {
JEPA_LN_BWD_INSTANCE(__half, __half, layernorm_bwd_f16)
JEPA_LN_BWD_INSTANCE(__nv_bfloat16, __nv_bfloat16, layernorm_bwd_bf16)
}  // namespace jepa
