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

template <typename TX, typename TY, int V, int NV, int TPR, bool SHIFT>
__global__ void __launch_bounds__(kBlock) ln_fwd_kernel(const TX* __restrict__ x, const float* __restrict__ w,
                                                        const float* __restrict__ b, TY* __restrict__ y,
                                                        float* __restrict__ mean, float* __restrict__ rstd, long rows,
                                                        int dim, float eps) {
  __shared__ float red[kBlock / 32];
  extern __shared__ __align__(16) float table[];   // SHIFT: w, then b, in the threads' columns: [NV * V / 4][thread] float4
  constexpr int kRows = kBlock / TPR;   // rows a block works on at a time
  constexpr int kTable = NV * V * kBlock;
  const int tid = threadIdx.x, t = tid % TPR;
  const long first = (long)blockIdx.x * kRows + tid / TPR;
  const long stride = (long)gridDim.x * kRows;
  const long total = rows * dim;
  const int o = SHIFT ? (int)((first * dim) % V) : 0;
  const float inv = 1.0f / (float)dim;
  if constexpr (SHIFT) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (t + i * TPR) * V - o + j;
        const int k = ((i * V + j) / 4 * kBlock + tid) * 4 + j % 4;
        table[k] = c >= 0 && c < dim ? __ldg(w + c) : 0.f;
        table[kTable + k] = c >= 0 && c < dim ? __ldg(b + c) : 0.f;
      }
  }
  for (long row = first; row < rows; row += stride) {
    float v[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (t + i * TPR) * V - o;
      const long at = row * dim + c0;
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      if (c0 < dim) {
        if (!SHIFT || at + V <= total) {
          ln_load<TX, V>(x + at, v[i]);
        } else {   // the last row's last vector ends with the operand
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (at + j < total) v[i][j] = DT<TX>::to(x[at + j]);
        }
        if (SHIFT && !ln_whole<V>(c0, dim)) {   // the neighbouring rows' values
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (c0 + j < 0 || c0 + j >= dim) v[i][j] = 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) s[0] += v[i][j];
    ln_row_sum<TPR, 1>(s, red);
    const float mu = s[0] * inv;
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (t + i * TPR) * V - o;
      if (c0 < dim) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] -= mu;
        if (SHIFT && !ln_whole<V>(c0, dim)) {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (c0 + j < 0 || c0 + j >= dim) v[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) q[0] = fmaf(v[i][j], v[i][j], q[0]);
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
      const int c0 = (t + i * TPR) * V - o;
      if (c0 < dim) {
        float ww[V], bb[V], out[V];
        if constexpr (SHIFT) {
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const float4 qw = *reinterpret_cast<const float4*>(table + ((i * V + j) / 4 * kBlock + tid) * 4);
            const float4 qb = *reinterpret_cast<const float4*>(table + kTable + ((i * V + j) / 4 * kBlock + tid) * 4);
            ww[j] = qw.x; ww[j + 1] = qw.y; ww[j + 2] = qw.z; ww[j + 3] = qw.w;
            bb[j] = qb.x; bb[j + 1] = qb.y; bb[j + 2] = qb.z; bb[j + 3] = qb.w;
          }
        } else {
          ln_load<float, V>(w + c0, ww);
          ln_load<float, V>(b + c0, bb);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = v[i][j] * rs * ww[j] + bb[j];
        if constexpr (SHIFT) ln_store_part<TY, V>(yr, c0, dim, out);
        else ln_store<TY, V>(yr + c0, out);
      }
    }
  }
}

// Rows wider than a block's registers, and operands that do not start on their
// vector: three sweeps over the row, the second and third out of L2.
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

constexpr int kMostBlocks = 152 * 8;
int blocks_of(long rows, int per_row) {
  const long need = (rows + per_row - 1) / per_row;
  return (int)(need < kMostBlocks ? need : kMostBlocks);
}

template <typename TX, typename TY, int V, int NV, int TPR, bool SHIFT>
cudaError_t launch_rows(const TX* x, const float* w, const float* b, TY* y, float* mean, float* rstd, long rows,
                        int dim, float eps, cudaStream_t s) {
  auto kern = ln_fwd_kernel<TX, TY, V, NV, TPR, SHIFT>;
  constexpr size_t kSmem = SHIFT ? sizeof(float) * 2 * NV * V * kBlock : 0;
  if constexpr (kSmem > 48 * 1024) {
    static DeviceOnce setup;
    const cudaError_t e = setup.run([&](int) {
      return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    });
    if (e != cudaSuccess) return e;
  }
  // a thread's rows have to be a multiple of V apart where its columns depend on them: 8 rows a block, or
  // a full grid of one-row blocks (a multiple of 8), or one row a block
  kern<<<blocks_of(rows, kBlock / TPR), kBlock, kSmem, s>>>(x, w, b, y, mean, rstd, rows, dim, eps);
  return cudaGetLastError();
}

template <typename TX, typename TY, int V, bool SHIFT>
cudaError_t fwd_v(const TX* x, const float* w, const float* b, TY* y, float* mean, float* rstd, long rows, int dim,
                  float eps, cudaStream_t s) {
  const int n = dim + (SHIFT ? V - 1 : 0);   // columns that the vectors cover
  if (n <= 256) return launch_rows<TX, TY, V, 8 / V, 32, SHIFT>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (n <= 512) return launch_rows<TX, TY, V, 16 / V, 32, SHIFT>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (n <= 1024) return launch_rows<TX, TY, V, 32 / V, 32, SHIFT>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (n <= 4096) return launch_rows<TX, TY, V, 16 / V, 256, SHIFT>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  return launch_rows<TX, TY, V, 32 / V, 256, SHIFT>(x, w, b, y, mean, rstd, rows, dim, eps, s);
}

constexpr int kLongest = 8192;   // columns that a block's registers hold

template <typename TX, typename TY>
cudaError_t fwd_t(const void* x_, const float* w, const float* b, void* y_, float* mean, float* rstd, long rows,
                  int dim, float eps, cudaStream_t s) {
  constexpr int V = sizeof(TX) == 4 ? 4 : 8;
  const TX* x = static_cast<const TX*>(x_);
  TY* y = static_cast<TY*>(y_);
  const bool vec = ln_aligned(x, V * sizeof(TX)) && ln_aligned(y, V * sizeof(TY));
  if (vec && dim % V == 0 && dim <= kLongest && ln_aligned(w, 16) && ln_aligned(b, 16))
    return fwd_v<TX, TY, V, false>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (vec && dim + V - 1 <= kLongest) return fwd_v<TX, TY, V, true>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  ln_fwd_wide_kernel<TX, TY><<<blocks_of(rows, 1), kBlock, 0, s>>>(x, w, b, y, mean, rstd, rows, dim, eps);
  return cudaGetLastError();
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
