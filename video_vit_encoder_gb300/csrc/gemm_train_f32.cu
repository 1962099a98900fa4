#include "gemm_train.cuh"

JEPA_TRAIN_GEMM_INSTANCES(__nv_bfloat16, true, gemm_f32)
