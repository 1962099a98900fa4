#include "gemm_train.cuh"

JEPA_TRAIN_GEMM_INSTANCES(__nv_bfloat16, false, gemm_bf16)
