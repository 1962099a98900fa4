#include "layernorm_bwd.cuh"

namespace jepa {
JEPA_LN_BWD_INSTANCE(float, float, layernorm_bwd_f32)
}  // namespace jepa
