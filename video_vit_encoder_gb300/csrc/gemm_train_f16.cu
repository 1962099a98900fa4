#include "gemm_train.cuh"

JEPA_TRAIN_GEMM_INSTANCES(__half, false, gemm_f16)
