// Layer norm forward for training: y = (x - mean) * rstd * w + b over the last
// dimension, keeping mean and rstd of each row for the backward pass.
//
// mean = sum x / n, rstd = 1 / sqrt(sum (x - mean)^2 / n + eps): the centred
// variance, both sums in fp32 over a row that stays in registers, so x is read
// once and y written once.  Bound by HBM: 16384 x 1024, fp32 in and bf16 out,
// 17.8 us with its input from HBM (0.84 of the copy bandwidth; 14.2 where part of
// it is in L2); 73728 x 777 in bf16 55 us (0.61: shifted vectors cost
// instructions); 8192 x 2048 in bf16 17.9 us.
#include "layernorm_train.cuh"

namespace jepa {

namespace {

constexpr int kBlock = 256;

// Rows that are multiples of their vector: a warp a row, or a block.
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
        float ww[V], bb[V], out[V];
        ln_load<float, V>(w + c, ww);
        ln_load<float, V>(b + c, bb);
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = v[i][j] * rs * ww[j] + bb[j];
        ln_store<TY, V>(yr + c, out);
      }
    }
  }
}

// Rows that start anywhere (SHIFT): one block of 16 warps per SM, rows through
// an asynchronous ring as in the backward pass, w and b in the threads' columns
// in shared memory.
constexpr int kShiftThreads = 512;
constexpr int kMostSmem = 232448;
template <typename TX, int V, int NV, int TPR>
struct ShiftShape {
  static constexpr int kRows = kShiftThreads / TPR;
  using Table = LnTable<V, NV, TPR, kRows>;
  static constexpr int kRowVec = NV * V * sizeof(TX);
  static constexpr size_t kHead = 32 * sizeof(float);
  static constexpr int kFit = (int)((kMostSmem - kHead - 2 * Table::kBytes) / (kShiftThreads * kRowVec));
  static constexpr int kDepth = kFit > 4 ? 4 : kFit;
  static_assert(kDepth >= 1, "a row must fit");
  static constexpr size_t kRing = (size_t)kDepth * kShiftThreads * kRowVec;
  static constexpr size_t kSmem = kHead + kRing + 2 * Table::kBytes;
};

template <typename TX, typename TY, int V, int NV, int TPR>
__global__ void __launch_bounds__(kShiftThreads, 1)
    ln_fwd_shift_kernel(const TX* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
                        TY* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd, long rows, int dim,
                        float eps) {
  using S = ShiftShape<TX, V, NV, TPR>;
  constexpr int kBX = V * sizeof(TX);
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem);
  uint8_t* ring = smem + S::kHead;
  float* tw = reinterpret_cast<float*>(ring + S::kRing);
  float* tb = tw + S::Table::kBytes / sizeof(float);
  const int tid = threadIdx.x, t = tid % TPR;
  const long first = (long)blockIdx.x * S::kRows + tid / TPR;
  const long stride = (long)gridDim.x * S::kRows;
  const int o = (int)((first * dim) % V);
  const int head = t == 0 ? o : 0;   // elements of this thread's vector 0 that are the previous row's
  const float inv = 1.0f / (float)dim;
  S::Table::fill(tw, w, dim, o);
  S::Table::fill(tb, b, dim, o);
  __syncthreads();
  // this thread's first column, and how many columns follow from there
  const int col = t * V - o, left = dim - col;
  const TX* fx = x + first * dim + col;   // of the next row to fetch
  TY* out_row = y + first * dim + col;    // of the current row
  const long step = stride * dim;
  long next = first;
  auto fetch = [&](int d) {
    if (next < rows) {
      uint8_t* q = ring + (size_t)d * kShiftThreads * S::kRowVec + tid * kBX;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * TPR * V < left)   // the last vector ends with the row (zeros follow)
          ln_copy_async<kBX>(q + i * kShiftThreads * kBX, fx + i * TPR * V,
                             min(V, left - i * TPR * V) * (int)sizeof(TX));
      fx += step;
      next += stride;
    }
    ln_copy_commit();
  };
#pragma unroll
  for (int d = 0; d < S::kDepth; ++d) fetch(d);
  int d = 0;
  for (long row = first; row < rows; row += stride) {
    ln_copy_wait<S::kDepth - 1>();
    const uint8_t* slot = ring + (size_t)d * kShiftThreads * S::kRowVec;
    f2 v[NV][V / 2];
    f2 sa = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * TPR * V < left) {
        LnVec<TX, V> vx;
        vx.load(slot + tid * kBX + i * kShiftThreads * kBX);
        if (i == 0) vx.drop_head(head);
        vx.pairs(v[i]);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) sa = f2_add(sa, v[i][j]);
      }
    }
    fetch(d);   // the slot has been read
    if (++d == S::kDepth) d = 0;
    float s[1] = {f2_sum(sa)};
    ln_row_sum<TPR, 1>(s, red);
    const float mu = s[0] * inv;
    const f2 mu2 = f2_make(-mu, -mu);
    f2 qa = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * TPR * V < left) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[i][j] = f2_add(v[i][j], mu2);
        const int lo = i == 0 ? head : 0, hi = left - i * TPR * V;
        if (lo == 0 && hi >= V) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) qa = f2_fma(v[i][j], v[i][j], qa);
        } else {   // without the values that are not the row's
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            float a0, a1;
            f2_get(v[i][j], a0, a1);
            if (2 * j < lo || 2 * j >= hi) a0 = 0.f;
            if (2 * j + 1 < lo || 2 * j + 1 >= hi) a1 = 0.f;
            const f2 a = f2_make(a0, a1);
            qa = f2_fma(a, a, qa);
          }
        }
      }
    }
    float q[1] = {f2_sum(qa)};
    ln_row_sum<TPR, 1>(q, red);
    const float rs = 1.0f / sqrtf(q[0] * inv + eps);
    if (t == 0) {
      if (mean != nullptr) mean[row] = mu;
      if (rstd != nullptr) rstd[row] = rs;
    }
    const f2 rs2 = f2_make(rs, rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * TPR * V < left) {
        f2 ww[V / 2], out[V / 2];
        S::Table::load(tw, i, ww);
        S::Table::load(tb, i, out);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) out[j] = f2_fma(f2_mul(v[i][j], rs2), ww[j], out[j]);
        LnVec<TY, V> vo;
        vo.set(out);
        const int lo = i == 0 ? head : 0, hi = left - i * TPR * V;
        if (lo == 0 && hi >= V) vo.store(out_row + i * TPR * V);
        else ln_store_part<TY, V>(out_row + i * TPR * V, lo, hi, vo);   // shared with a neighbouring row
      }
    }
    out_row += step;
  }
  ln_copy_wait<0>();
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

template <typename TX, typename TY, int V>
cudaError_t fwd_rows(const TX* x, const float* w, const float* b, TY* y, float* mean, float* rstd, long rows, int dim,
                     float eps, cudaStream_t s) {
#define JEPA_LN_FWD(NVE, TPR)                                                                                   \
  ln_fwd_kernel<TX, TY, V, (NVE) / V, TPR><<<blocks_of(rows, kBlock / TPR), kBlock, 0, s>>>(x, w, b, y, mean, rstd, \
                                                                                            rows, dim, eps)
  if (dim <= 256) JEPA_LN_FWD(8, 32);
  else if (dim <= 512) JEPA_LN_FWD(16, 32);
  else if (dim <= 1024) JEPA_LN_FWD(32, 32);
  else if (dim <= 2048) JEPA_LN_FWD(32, 64);
  else if (dim <= 4096) JEPA_LN_FWD(32, 128);
  else JEPA_LN_FWD(32, 256);
#undef JEPA_LN_FWD
  return cudaGetLastError();
}

template <typename TX, typename TY, int V, int NV, int TPR>
cudaError_t launch_shift(const TX* x, const float* w, const float* b, TY* y, float* mean, float* rstd, long rows,
                         int dim, float eps, cudaStream_t s) {
  using S = ShiftShape<TX, V, NV, TPR>;
  auto kern = ln_fwd_shift_kernel<TX, TY, V, NV, TPR>;
  static DeviceOnce setup;
  const cudaError_t e = setup.run([&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  });
  if (e != cudaSuccess) return e;
  // a thread's rows are a multiple of 8 apart (152 blocks), or it has one row
  const long need = (rows + S::kRows - 1) / S::kRows;
  kern<<<(int)(need < 152 ? need : 152), kShiftThreads, S::kSmem, s>>>(x, w, b, y, mean, rstd, rows, dim, eps);
  return cudaGetLastError();
}

template <typename TX, typename TY, int V>
cudaError_t fwd_shift(const TX* x, const float* w, const float* b, TY* y, float* mean, float* rstd, long rows, int dim,
                      float eps, cudaStream_t s) {
  const int n = dim + V - 1;   // columns that the vectors cover
  if (n <= 256) return launch_shift<TX, TY, V, 8 / V, 32>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (n <= 512) return launch_shift<TX, TY, V, 16 / V, 32>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (n <= 1024) return launch_shift<TX, TY, V, 32 / V, 32>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (n <= 2048) return launch_shift<TX, TY, V, 32 / V, 64>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (n <= 4096) return launch_shift<TX, TY, V, 32 / V, 128>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  return launch_shift<TX, TY, V, 32 / V, 256>(x, w, b, y, mean, rstd, rows, dim, eps, s);
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
    return fwd_rows<TX, TY, V>(x, w, b, y, mean, rstd, rows, dim, eps, s);
  if (vec && dim + V - 1 <= kLongest) return fwd_shift<TX, TY, V>(x, w, b, y, mean, rstd, rows, dim, eps, s);
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
