// Layer norm forward for training: y = (x - mean) * rstd * w + b over the last
// dimension, keeping mean and rstd of each row for the backward pass.
//
// mean = sum x / n, rstd = 1 / sqrt(sum (x - mean)^2 / n + eps): the centred
// variance, both sums in fp32 over a row that stays in registers, so x is read
// once and y written once.  Bound by HBM.
#include "layernorm_train.cuh"

namespace jepa {

namespace {

constexpr int kBlock = 256;

template <typename TX, typename TY, int V, int NV, int TPR>
__global__ void __launch_bounds__(kBlock) ln_fwd_kernel(const TX* __restrict__ x, const float* __restrict__ w,
                                                        const float* __restrict__ b, TY* __restrict__ y,
                                                        float* __restrict__ mean, float* __restrict__ rstd, long rows,
                                                        int dim, float eps) {
  __shared__ float red[kBlock / 32];
  constexpr int kRows = kBlock / TPR;   // rows a block works on at a time
  const int t = threadIdx.x % TPR;
  const long stride = (long)gridDim.x * kRows;
  const float inv = 1.0f / (float)dim;
  for (long row = (long)blockIdx.x * kRows + threadIdx.x / TPR; row < rows; row += stride) {
    const TX* xr = x + row * dim;
    float v[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * TPR) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      if (c < dim) ln_load<TX, V>(xr + c, v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) s[0] += v[i][j];
    ln_row_sum<TPR, 1>(s, red);
    const float mu = s[0] * inv;
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((t + i * TPR) * V < dim) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[i][j] -= mu;
          q[0] = fmaf(v[i][j], v[i][j], q[0]);
        }
      }
    ln_row_sum<TPR, 1>(q, red);
    const float rs = 1.0f / sqrtf(q[0] * inv + eps);
    if (t == 0) {
      if (mean != nullptr) mean[row] = mu;
      if (rstd != nullptr) rstd[row] = rs;
    }
    TY* yr = y + row * dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * TPR) * V;
      if (c < dim) {
        float ww[V], bb[V], o[V];
        ln_load<float, V>(w + c, ww);
        ln_load<float, V>(b + c, bb);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = v[i][j] * rs * ww[j] + bb[j];
        ln_store<TY, V>(yr + c, o);
      }
    }
  }
}

// Rows wider than a block's registers: three sweeps over the row, the second
// and third out of L2.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kBlock) ln_fwd_wide_kernel(const TX* __restrict__ x, const float* __restrict__ w,
                                                             const float* __restrict__ b, TY* __restrict__ y,
                                                             float* __restrict__ mean, float* __restrict__ rstd,
                                                             long rows, int dim, float eps) {
  __shared__ float red[kBlock / 32];
  const float inv = 1.0f / (float)dim;
  for (long row = blockIdx.x; row < rows; row += gridDim.x) {
    const TX* xr = x + row * dim;
    float s[1] = {0.f};
    for (int c = threadIdx.x; c < dim; c += kBlock) s[0] += DT<TX>::to(xr[c]);
    ln_row_sum<kBlock, 1>(s, red);
    const float mu = s[0] * inv;
    float q[1] = {0.f};
    for (int c = threadIdx.x; c < dim; c += kBlock) {
      const float d = DT<TX>::to(xr[c]) - mu;
      q[0] = fmaf(d, d, q[0]);
    }
    ln_row_sum<kBlock, 1>(q, red);
    const float rs = 1.0f / sqrtf(q[0] * inv + eps);
    if (threadIdx.x == 0) {
      if (mean != nullptr) mean[row] = mu;
      if (rstd != nullptr) rstd[row] = rs;
    }
    TY* yr = y + row * dim;
    for (int c = threadIdx.x; c < dim; c += kBlock)
      yr[c] = DT<TY>::from((DT<TX>::to(xr[c]) - mu) * rs * __ldg(w + c) + __ldg(b + c));
  }
}

template <typename TX, typename TY, int V>
cudaError_t fwd_v(const TX* x, const float* w, const float* b, TY* y, float* mean, float* rstd, long rows, int dim,
                  float eps, cudaStream_t s) {
  const int per_row = dim <= 1024 ? kBlock / 32 : 1;
  const long need = (rows + per_row - 1) / per_row;
  const int blocks = (int)(need < 152 * 8 ? need : 152 * 8);
#define JEPA_LN_FWD(NVE, TPR) \
  ln_fwd_kernel<TX, TY, V, (NVE) / V, TPR><<<blocks, kBlock, 0, s>>>(x, w, b, y, mean, rstd, rows, dim, eps)
  if (dim <= 256) JEPA_LN_FWD(8, 32);
  else if (dim <= 512) JEPA_LN_FWD(16, 32);
  else if (dim <= 1024) JEPA_LN_FWD(32, 32);
  else if (dim <= 2048) JEPA_LN_FWD(8, 256);
  else if (dim <= 4096) JEPA_LN_FWD(16, 256);
  else if (dim <= 8192) JEPA_LN_FWD(32, 256);
  else ln_fwd_wide_kernel<TX, TY><<<blocks, kBlock, 0, s>>>(x, w, b, y, mean, rstd, rows, dim, eps);
#undef JEPA_LN_FWD
  return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t fwd_t(const void* x, const float* w, const float* b, void* y, float* mean, float* rstd, long rows, int dim,
                  float eps, cudaStream_t s) {
  constexpr int V = sizeof(TX) == 4 ? 4 : 8;
  const bool vec = dim % V == 0 && ln_aligned(x, V * sizeof(TX)) && ln_aligned(y, V * sizeof(TY)) &&
                   ln_aligned(w, 16) && ln_aligned(b, 16);
  const TX* xx = static_cast<const TX*>(x);
  TY* yy = static_cast<TY*>(y);
  return vec ? fwd_v<TX, TY, V>(xx, w, b, yy, mean, rstd, rows, dim, eps, s)
             : fwd_v<TX, TY, 1>(xx, w, b, yy, mean, rstd, rows, dim, eps, s);
}

}  // namespace

cudaError_t layernorm_fwd(int x_dtype, int y_dtype, const void* x, const float* w, const float* b, void* y, float* mean,
                          float* rstd, long rows, int dim, float eps, cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  if (x_dtype == DTYPE_F32) {
    if (y_dtype == DTYPE_F32) return fwd_t<float, float>(x, w, b, y, mean, rstd, rows, dim, eps, s);
    if (y_dtype == DTYPE_F16) return fwd_t<float, __half>(x, w, b, y, mean, rstd, rows, dim, eps, s);
    return fwd_t<float, __nv_bfloat16>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  }
  if (x_dtype == DTYPE_F16) return fwd_t<__half, __half>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  return fwd_t<__nv_bfloat16, __nv_bfloat16>(x, w, b, y, mean, rstd, rows, dim, eps, s);
}

}  // namespace jepa
