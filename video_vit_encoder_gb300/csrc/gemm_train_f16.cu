#include "gemm_train.cuh"

JEPA_TRAIN_GEMM_INSTANCES(__half, gemm_f16)
