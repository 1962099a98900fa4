// Layer norm backward.  With xh = (x - mean) rstd and c = dy * w, per row
//   dx = rstd (c - mean_j c - xh mean_j(c xh)) [+ res]
// and over the rows  dw = sum dy * xh,  db = sum dy.
//
// One pass over x, dy (and res): a row stays in registers between its two
// row sums and dx.  Each block walks a strip of rows and keeps the strip's dw
// and db sums in registers, so they cost no traffic until the strip ends; a
// second kernel adds the strips' sums in a fixed order (no atomics, so the
// result does not depend on scheduling).  Bound by HBM.
#include "layernorm_train.cuh"

namespace jepa {

namespace {

constexpr int kBlock = 256;

template <typename TX, typename TY, int V, int NV, int TPR, bool RES>
__global__ void __launch_bounds__(kBlock) ln_bwd_kernel(const TY* __restrict__ dy, const TX* __restrict__ x,
                                                        const float* __restrict__ w, const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, const TX* __restrict__ res,
                                                        TX* __restrict__ dx, float* __restrict__ part, long rows,
                                                        int dim) {
  extern __shared__ float sm[];   // [2 * 8] sums, then (one warp a row) [2 * dim] of a warp's dw, db
  constexpr int kRows = kBlock / TPR;
  const int t = threadIdx.x % TPR;
  const long stride = (long)gridDim.x * kRows;
  const float inv = 1.0f / (float)dim;
  float aw[NV][V], ab[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) aw[i][j] = ab[i][j] = 0.f;
  for (long row = (long)blockIdx.x * kRows + threadIdx.x / TPR; row < rows; row += stride) {
    const TX* xr = x + row * dim;
    const TY* gr = dy + row * dim;
    const float mu = __ldg(mean + row), rs = __ldg(rstd + row);
    float xv[NV][V], gv[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * TPR) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) xv[i][j] = gv[i][j] = 0.f;
      if (c < dim) {
        ln_load<TX, V>(xr + c, xv[i]);
        ln_load<TY, V>(gr + c, gv[i]);
      }
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * TPR) * V;
      if (c < dim) {
        float ww[V];
        ln_load<float, V>(w + c, ww);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (xv[i][j] - mu) * rs;
          xv[i][j] = xh;
          aw[i][j] = fmaf(gv[i][j], xh, aw[i][j]);
          ab[i][j] += gv[i][j];
          gv[i][j] *= ww[j];
          s[0] += gv[i][j];
          s[1] = fmaf(gv[i][j], xh, s[1]);
        }
      }
    }
    ln_row_sum<TPR, 2>(s, sm);
    const float m0 = s[0] * inv, m1 = s[1] * inv;
    TX* dr = dx + row * dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * TPR) * V;
      if (c < dim) {
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = rs * (gv[i][j] - m0 - xv[i][j] * m1);
        if constexpr (RES) {
          float r[V];
          ln_load<TX, V>(res + row * dim + c, r);
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] += r[j];
        }
        ln_store<TX, V>(dr + c, o);
      }
    }
  }
  // the block's dw and db: the warps add theirs one after another
  float* pw = part + (size_t)blockIdx.x * 2 * dim;
  if constexpr (TPR == 32) {
    float* acc = sm + 16;
    const int warp = threadIdx.x >> 5;
    for (int k = 0; k < kBlock / 32; ++k) {
      __syncthreads();
      if (warp == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * TPR) * V;
          if (c < dim) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              acc[c + j] = (k == 0 ? 0.f : acc[c + j]) + aw[i][j];
              acc[dim + c + j] = (k == 0 ? 0.f : acc[dim + c + j]) + ab[i][j];
            }
          }
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * dim; c += kBlock) pw[c] = acc[c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * TPR) * V;
      if (c < dim) {
        ln_store<float, V>(pw + c, aw[i]);
        if constexpr (V > 1) ln_store<float, V>(pw + dim + c, ab[i]);
        else pw[dim + c] = ab[i][0];
      }
    }
  }
}

// Rows wider than a block's registers: two sweeps over the row, the second
// out of L2; the strip's dw and db live in its slot of `part`.
template <typename TX, typename TY, bool RES>
__global__ void __launch_bounds__(kBlock) ln_bwd_wide_kernel(const TY* __restrict__ dy, const TX* __restrict__ x,
                                                             const float* __restrict__ w,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd,
                                                             const TX* __restrict__ res, TX* __restrict__ dx,
                                                             float* __restrict__ part, long rows, int dim) {
  __shared__ float red[2 * kBlock / 32];
  const float inv = 1.0f / (float)dim;
  float* pw = part + (size_t)blockIdx.x * 2 * dim;
  bool first = true;
  for (long row = blockIdx.x; row < rows; row += gridDim.x) {
    const TX* xr = x + row * dim;
    const TY* gr = dy + row * dim;
    const float mu = __ldg(mean + row), rs = __ldg(rstd + row);
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < dim; c += kBlock) {
      const float xh = (DT<TX>::to(xr[c]) - mu) * rs, g = DT<TY>::to(gr[c]);
      pw[c] = (first ? 0.f : pw[c]) + g * xh;
      pw[dim + c] = (first ? 0.f : pw[dim + c]) + g;
      const float gw = g * __ldg(w + c);
      s[0] += gw;
      s[1] = fmaf(gw, xh, s[1]);
    }
    ln_row_sum<kBlock, 2>(s, red);
    const float m0 = s[0] * inv, m1 = s[1] * inv;
    for (int c = threadIdx.x; c < dim; c += kBlock) {
      const float xh = (DT<TX>::to(xr[c]) - mu) * rs;
      float o = rs * (DT<TY>::to(gr[c]) * __ldg(w + c) - m0 - xh * m1);
      if (RES) o += DT<TX>::to(res[row * dim + c]);
      dx[row * dim + c] = DT<TX>::from(o);
    }
    first = false;
  }
}

// out[c] = sum over the strips of part[strip][c]; 8 threads a column, each
// over every eighth strip, joined in a fixed order.
__global__ void __launch_bounds__(kBlock) ln_bwd_sum_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                            float* __restrict__ db, int strips, int dim) {
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * dim)
    for (int k = g; k < strips; k += 8) s += part[(size_t)k * 2 * dim + c];
  sm[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < 2 * dim) {
    for (int k = 1; k < 8; ++k) s += sm[k][lane];
    float* out = c < dim ? dw : db;
    if (out != nullptr) out[c < dim ? c : c - dim] = s;
  }
}

int bwd_strips(long rows, int dim) {
  const int per = dim <= 1024 ? kBlock / 32 : 1;
  const long need = (rows + per - 1) / per;
  return (int)(need < kLnBwdStrips ? need : kLnBwdStrips);
}

template <typename TX, typename TY, int V, bool RES>
cudaError_t bwd_v(const TY* dy, const TX* x, const float* w, const float* mean, const float* rstd, const TX* res,
                  TX* dx, float* part, long rows, int dim, cudaStream_t s) {
  const int blocks = bwd_strips(rows, dim);
  const size_t smem = sizeof(float) * (16 + (dim <= 1024 ? 2 * dim : 0));
#define JEPA_LN_BWD(NVE, TPR) \
  ln_bwd_kernel<TX, TY, V, (NVE) / V, TPR, RES><<<blocks, kBlock, smem, s>>>(dy, x, w, mean, rstd, res, dx, part, rows, dim)
  if (dim <= 256) JEPA_LN_BWD(8, 32);
  else if (dim <= 512) JEPA_LN_BWD(16, 32);
  else if (dim <= 1024) JEPA_LN_BWD(32, 32);
  else if (dim <= 2048) JEPA_LN_BWD(8, 256);
  else if (dim <= 4096) JEPA_LN_BWD(16, 256);
  else if (dim <= 8192) JEPA_LN_BWD(32, 256);
  else ln_bwd_wide_kernel<TX, TY, RES><<<blocks, kBlock, 0, s>>>(dy, x, w, mean, rstd, res, dx, part, rows, dim);
#undef JEPA_LN_BWD
  return cudaGetLastError();
}

template <typename TX, typename TY>
cudaError_t bwd_t(const void* dy_, const void* x_, const float* w, const float* mean, const float* rstd,
                  const void* res_, void* dx_, float* part, long rows, int dim, cudaStream_t s) {
  constexpr int V = sizeof(TX) == 4 ? 4 : 8;
  const TX* x = static_cast<const TX*>(x_);
  const TY* dy = static_cast<const TY*>(dy_);
  const TX* res = static_cast<const TX*>(res_);
  TX* dx = static_cast<TX*>(dx_);
  const bool vec = dim % V == 0 && ln_aligned(x, V * sizeof(TX)) && ln_aligned(dy, V * sizeof(TY)) &&
                   ln_aligned(dx, V * sizeof(TX)) && ln_aligned(res, V * sizeof(TX)) && ln_aligned(w, 16) &&
                   ln_aligned(part, 16);
  if (vec)
    return res ? bwd_v<TX, TY, V, true>(dy, x, w, mean, rstd, res, dx, part, rows, dim, s)
               : bwd_v<TX, TY, V, false>(dy, x, w, mean, rstd, res, dx, part, rows, dim, s);
  return res ? bwd_v<TX, TY, 1, true>(dy, x, w, mean, rstd, res, dx, part, rows, dim, s)
             : bwd_v<TX, TY, 1, false>(dy, x, w, mean, rstd, res, dx, part, rows, dim, s);
}

}  // namespace

size_t layernorm_bwd_workspace(long rows, int dim) {
  return sizeof(float) * 2 * (size_t)dim * bwd_strips(rows, dim);
}

cudaError_t layernorm_bwd(int x_dtype, int y_dtype, const void* dy, const void* x, const float* w, const float* mean,
                          const float* rstd, const void* res, void* dx, float* dw, float* db, long rows, int dim,
                          float* ws, cudaStream_t s) {
  const int strips = bwd_strips(rows, dim);
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    if (x_dtype == DTYPE_F32) {
      if (y_dtype == DTYPE_F32) e = bwd_t<float, float>(dy, x, w, mean, rstd, res, dx, ws, rows, dim, s);
      else if (y_dtype == DTYPE_F16) e = bwd_t<float, __half>(dy, x, w, mean, rstd, res, dx, ws, rows, dim, s);
      else e = bwd_t<float, __nv_bfloat16>(dy, x, w, mean, rstd, res, dx, ws, rows, dim, s);
    } else if (x_dtype == DTYPE_F16) {
      e = bwd_t<__half, __half>(dy, x, w, mean, rstd, res, dx, ws, rows, dim, s);
    } else {
      e = bwd_t<__nv_bfloat16, __nv_bfloat16>(dy, x, w, mean, rstd, res, dx, ws, rows, dim, s);
    }
    if (e != cudaSuccess) return e;
  }
  if (dw == nullptr && db == nullptr) return cudaSuccess;
  ln_bwd_sum_kernel<<<(2 * dim + 31) / 32, kBlock, 0, s>>>(ws, dw, db, strips, dim);
  return cudaGetLastError();
}

}  // namespace jepa
