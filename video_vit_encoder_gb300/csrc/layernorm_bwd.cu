// Layer norm backward.  With xh = (x - mean) rstd and c = dy * w, per row
//   dx = rstd (c - mean_j c - xh mean_j(c xh)) [+ res]
// and over the rows  dw = sum dy * xh,  db = sum dy.
//
// One pass over x, dy (and res): a row stays in registers between its two
// row sums and dx.  Each block (one per SM) walks rows and keeps its sums of
// dw and db in registers, so they cost no traffic until it ends; a second
// kernel adds the blocks' sums in a fixed order (no atomics, so the result
// does not depend on scheduling).  Bound by HBM.
//
// The accumulators leave room for 12 warps per SM, too few to hide the loads'
// latency, so rows come through shared memory: each thread copies its own
// vectors of its next rows asynchronously (no other thread reads them, so
// there is no barrier) while it works on the current one.
#include "layernorm_train.cuh"

namespace jepa {

namespace {

constexpr int kBlock = 256;
constexpr int kSmemRing = 160 * 1024;   // for the rows in flight

// The kernel's shape: TPR threads a row (32 or 256), blocks of 12 warps (one
// row each) or of 8 (one row), and the rows in flight per thread.
template <typename TX, typename TY, int V, int NV, int TPR>
struct BwdShape {
  static constexpr int kThreads = TPR == 32 ? 384 : 256;
  static constexpr int kRows = kThreads / TPR;
  static constexpr int kRowVec = NV * V * (2 * sizeof(TX) + sizeof(TY));   // x, res and dy of a thread's columns
  static constexpr int kFit = kSmemRing / (kThreads * kRowVec);
  static constexpr int kDepth = kFit < 1 ? 1 : (kFit > 4 ? 4 : kFit);
  static constexpr size_t kRing = (size_t)kDepth * kThreads * kRowVec;
  static constexpr size_t kTable = sizeof(float) * kThreads * NV * V;      // w in the threads' columns
  static constexpr size_t kSmem = 16 * sizeof(float) + kRing + kTable;
  static_assert(2 * kTable <= kRing + kTable, "the warps' dw and db reuse the ring");
  static_assert(kSmem <= 232448, "shared memory of one block");
};

template <typename TX, typename TY, int V, int NV, int TPR, bool SHIFT>
__global__ void __launch_bounds__(BwdShape<TX, TY, V, NV, TPR>::kThreads, 1)
    ln_bwd_kernel(const TY* __restrict__ dy, const TX* __restrict__ x, const float* __restrict__ w,
                  const float* __restrict__ mean, const float* __restrict__ rstd, const TX* __restrict__ res,
                  TX* __restrict__ dx, float* __restrict__ part_w, float* __restrict__ part_b, long rows, int dim) {
  using S = BwdShape<TX, TY, V, NV, TPR>;
  constexpr int kBX = V * sizeof(TX), kBY = V * sizeof(TY);
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem);                       // [16] row sums across warps
  uint8_t* ring = smem + 16 * sizeof(float);                         // [depth][x | res | dy][NV][thread]
  float* table = reinterpret_cast<float*>(ring + S::kRing);          // [NV * V / 4][thread] float4
  const int tid = threadIdx.x, t = tid % TPR;
  const long first = (long)blockIdx.x * S::kRows + tid / TPR;
  const long stride = (long)gridDim.x * S::kRows;
  const long total = rows * dim;
  const int o = SHIFT ? (int)((first * dim) % V) : 0;
  const float inv = 1.0f / (float)dim;

  if constexpr (SHIFT) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (t + i * TPR) * V - o + j;
        table[((i * V + j) / 4 * S::kThreads + tid) * 4 + j % 4] = c >= 0 && c < dim ? __ldg(w + c) : 0.f;
      }
  }

  // this thread's vectors of `row` into slot d of the ring
  auto fetch = [&](long row, int d) {
    if (row < rows) {
      uint8_t* slot = ring + (size_t)d * S::kThreads * S::kRowVec;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c0 = (t + i * TPR) * V - o;
        if (c0 < dim) {
          const long at = row * dim + c0;
          const long left = total - at;   // the last row's last vector ends with the operand
          const int n = SHIFT && left < V ? (int)left : V;
          uint8_t* q = slot + (size_t)(i * S::kThreads + tid) * kBX;
          ln_copy_async<kBX>(q, x + at, n * (int)sizeof(TX));
          if (res != nullptr)
            ln_copy_async<kBX>(q + (size_t)NV * S::kThreads * kBX, res + at, n * (int)sizeof(TX));
          ln_copy_async<kBY>(slot + (size_t)2 * NV * S::kThreads * kBX + (size_t)(i * S::kThreads + tid) * kBY, dy + at,
                             n * (int)sizeof(TY));
        }
      }
    }
    ln_copy_commit();
  };
#pragma unroll
  for (int d = 0; d < S::kDepth; ++d) fetch(first + d * stride, d);

  float aw[NV][V], ab[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) aw[i][j] = ab[i][j] = 0.f;

  int d = 0;
  for (long row = first; row < rows; row += stride) {
    const float mu = __ldg(mean + row), rs = __ldg(rstd + row);
    ln_copy_wait<S::kDepth - 1>();
    const uint8_t* slot = ring + (size_t)d * S::kThreads * S::kRowVec;
    float xv[NV][V], gv[NV][V];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (t + i * TPR) * V - o;
      if (c0 < dim) {
        ln_load<TX, V>(reinterpret_cast<const TX*>(slot + (size_t)(i * S::kThreads + tid) * kBX), xv[i]);
        ln_load<TY, V>(reinterpret_cast<const TY*>(slot + (size_t)2 * NV * S::kThreads * kBX +
                                                   (size_t)(i * S::kThreads + tid) * kBY),
                       gv[i]);
        if (SHIFT && !ln_whole<V>(c0, dim)) {
          // the neighbouring rows' values in a shared vector
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (c0 + j < 0 || c0 + j >= dim) {
              xv[i][j] = mu;
              gv[i][j] = 0.f;
            }
        }
        float ww[V];
        if constexpr (SHIFT) {
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const float4 q = *reinterpret_cast<const float4*>(table + ((i * V + j) / 4 * S::kThreads + tid) * 4);
            ww[j] = q.x; ww[j + 1] = q.y; ww[j + 2] = q.z; ww[j + 3] = q.w;
          }
        } else {
          ln_load<float, V>(w + c0, ww);
        }
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
    ln_row_sum<TPR, 2>(s, red);
    const float m0 = s[0] * inv, m1 = s[1] * inv;
    TX* dr = dx + row * dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (t + i * TPR) * V - o;
      if (c0 < dim) {
        float out[V];
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = rs * (gv[i][j] - m0 - xv[i][j] * m1);
        if (res != nullptr) {
          float r[V];
          ln_load<TX, V>(reinterpret_cast<const TX*>(slot + (size_t)((NV + i) * S::kThreads + tid) * kBX), r);
#pragma unroll
          for (int j = 0; j < V; ++j) out[j] += r[j];
        }
        if constexpr (SHIFT) ln_store_part<TX, V>(dr, c0, dim, out);
        else ln_store<TX, V>(dr + c0, out);
      }
    }
    fetch(row + S::kDepth * stride, d);   // the slot has been read
    if (++d == S::kDepth) d = 0;
  }
  ln_copy_wait<0>();

  float* pw = part_w + (size_t)blockIdx.x * 2 * dim;
  float* pb = part_b + (size_t)blockIdx.x * 2 * dim;
  if constexpr (TPR == 32) {
    // the warps' sums side by side in shared memory, then added in warp order
    __syncthreads();
    float* mine = reinterpret_cast<float*>(ring) + (size_t)(tid / 32) * 2 * dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = t * V + i * TPR * V - o;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c0 + j >= 0 && c0 + j < dim) {
          mine[c0 + j] = aw[i][j];
          mine[dim + c0 + j] = ab[i][j];
        }
    }
    __syncthreads();
    const float* all = reinterpret_cast<const float*>(ring);
    for (int c = tid; c < 2 * dim; c += S::kThreads) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < S::kRows; ++k) v += all[(size_t)k * 2 * dim + c];
      if (c < dim) pw[c] = v;
      else pb[c - dim] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = t * V + i * TPR * V - o;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c0 + j >= 0 && c0 + j < dim) {
          pw[c0 + j] = aw[i][j];
          pb[c0 + j] = ab[i][j];
        }
    }
  }
}

// Rows wider than a block's registers, and operands that do not start on their
// vector: two sweeps over the row, the second out of L2; the block's dw and db
// live in its slot of the workspace.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kBlock) ln_bwd_wide_kernel(const TY* __restrict__ dy, const TX* __restrict__ x,
                                                             const float* __restrict__ w,
                                                             const float* __restrict__ mean,
                                                             const float* __restrict__ rstd,
                                                             const TX* __restrict__ res, TX* __restrict__ dx,
                                                             float* __restrict__ part_w, float* __restrict__ part_b,
                                                             long rows, int dim) {
  __shared__ float red[2 * kBlock / 32];
  const float inv = 1.0f / (float)dim;
  float* pw = part_w + (size_t)blockIdx.x * 2 * dim;
  float* pb = part_b + (size_t)blockIdx.x * 2 * dim;
  bool first = true;
  for (long row = blockIdx.x; row < rows; row += gridDim.x) {
    const TX* xr = x + row * dim;
    const TY* gr = dy + row * dim;
    const float mu = __ldg(mean + row), rs = __ldg(rstd + row);
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < dim; c += kBlock) {
      const float xh = (DT<TX>::to(xr[c]) - mu) * rs, g = DT<TY>::to(gr[c]);
      pw[c] = (first ? 0.f : pw[c]) + g * xh;
      pb[c] = (first ? 0.f : pb[c]) + g;
      const float gw = g * __ldg(w + c);
      s[0] += gw;
      s[1] = fmaf(gw, xh, s[1]);
    }
    ln_row_sum<kBlock, 2>(s, red);
    const float m0 = s[0] * inv, m1 = s[1] * inv;
    for (int c = threadIdx.x; c < dim; c += kBlock) {
      const float xh = (DT<TX>::to(xr[c]) - mu) * rs;
      float o = rs * (DT<TY>::to(gr[c]) * __ldg(w + c) - m0 - xh * m1);
      if (res != nullptr) o += DT<TX>::to(res[row * dim + c]);
      dx[row * dim + c] = DT<TX>::from(o);
    }
    first = false;
  }
}

// out[c] = sum over the strips of part[strip][c]; 32 threads a column, each
// over every 32nd strip, joined in a fixed order.
__global__ void __launch_bounds__(1024) ln_bwd_sum_kernel(const float* __restrict__ part, float* __restrict__ dw,
                                                          float* __restrict__ db, int strips, int dim) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * dim) {
#pragma unroll 5
    for (int k = g; k < strips; k += 32) s += part[(size_t)k * 2 * dim + c];
  }
  sm[g][lane] = s;
  __syncthreads();
  s = ln_warp_sum(sm[lane][g]);   // warp g joins column g of the block
  const int cc = blockIdx.x * 32 + g;
  if (lane == 0 && cc < 2 * dim) {
    float* out = cc < dim ? dw : db;
    if (out != nullptr) out[cc < dim ? cc : cc - dim] = s;
  }
}

// How the rows are spread: over at most one block per SM (two for the wide
// kernel, whose blocks are small); one block writes dw and db itself.
constexpr int kBlocks = 152;
int bwd_strips_rows(long rows, int per, int most) {
  const long need = (rows + per - 1) / per;
  return (int)(need < most ? need : most);
}
constexpr int kLongest = 8192;   // columns that a block's registers hold

struct Args {
  const void *dy, *x, *res;
  const float *w, *mean, *rstd;
  void* dx;
  float *dw, *db, *ws;
  long rows;
  int dim;
};

// The partial sums' place: the workspace, or for a single strip the outputs.
void parts(const Args& a, int strips, float*& pw, float*& pb) {
  const bool direct = strips == 1 && a.dw != nullptr && a.db != nullptr;
  pw = direct ? a.dw : a.ws;
  pb = direct ? a.db : a.ws + a.dim;
}
cudaError_t join(const Args& a, int strips, cudaStream_t s) {
  if ((a.dw == nullptr && a.db == nullptr) || (strips == 1 && a.dw != nullptr && a.db != nullptr)) return cudaSuccess;
  ln_bwd_sum_kernel<<<(2 * a.dim + 31) / 32, 1024, 0, s>>>(a.ws, a.dw, a.db, strips, a.dim);
  return cudaGetLastError();
}

template <typename TX, typename TY, int V, int NV, int TPR, bool SHIFT>
cudaError_t launch_rows(const Args& a, cudaStream_t s) {
  using S = BwdShape<TX, TY, V, NV, TPR>;
  auto kern = ln_bwd_kernel<TX, TY, V, NV, TPR, SHIFT>;
  static DeviceOnce setup;
  cudaError_t e = setup.run([&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  });
  if (e != cudaSuccess) return e;
  const int strips = bwd_strips_rows(a.rows, S::kRows, kBlocks);
  float *pw, *pb;
  parts(a, strips, pw, pb);
  kern<<<strips, S::kThreads, S::kSmem, s>>>((const TY*)a.dy, (const TX*)a.x, a.w, a.mean, a.rstd, (const TX*)a.res,
                                             (TX*)a.dx, pw, pb, a.rows, a.dim);
  e = cudaGetLastError();
  return e == cudaSuccess ? join(a, strips, s) : e;
}

template <typename TX, typename TY, int V, bool SHIFT>
cudaError_t launch_width(const Args& a, cudaStream_t s) {
  const int n = a.dim + (SHIFT ? V - 1 : 0);   // columns that the vectors cover
  if (n <= 256) return launch_rows<TX, TY, V, 8 / V, 32, SHIFT>(a, s);
  if (n <= 512) return launch_rows<TX, TY, V, 16 / V, 32, SHIFT>(a, s);
  if (n <= 1024) return launch_rows<TX, TY, V, 32 / V, 32, SHIFT>(a, s);
  if (n <= 4096) return launch_rows<TX, TY, V, 16 / V, 256, SHIFT>(a, s);
  return launch_rows<TX, TY, V, 32 / V, 256, SHIFT>(a, s);
}

template <typename TX, typename TY>
cudaError_t bwd_t(const Args& a, cudaStream_t s) {
  constexpr int V = sizeof(TX) == 4 ? 4 : 8;
  const bool vec = ln_aligned(a.x, V * sizeof(TX)) && ln_aligned(a.dy, V * sizeof(TY)) &&
                   ln_aligned(a.dx, V * sizeof(TX)) && ln_aligned(a.res, V * sizeof(TX));
  if (vec && a.dim % V == 0 && a.dim <= kLongest && ln_aligned(a.w, 16)) return launch_width<TX, TY, V, false>(a, s);
  if (vec && a.dim + V - 1 <= kLongest) return launch_width<TX, TY, V, true>(a, s);
  const int strips = bwd_strips_rows(a.rows, 1, 2 * kBlocks);
  float *pw, *pb;
  parts(a, strips, pw, pb);
  ln_bwd_wide_kernel<TX, TY><<<strips, kBlock, 0, s>>>((const TY*)a.dy, (const TX*)a.x, a.w, a.mean, a.rstd,
                                                       (const TX*)a.res, (TX*)a.dx, pw, pb, a.rows, a.dim);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? join(a, strips, s) : e;
}

}  // namespace

size_t layernorm_bwd_workspace(long rows, int dim) {
  return sizeof(float) * 2 * (size_t)dim * bwd_strips_rows(rows, 1, 2 * kBlocks);
}

cudaError_t layernorm_bwd(int x_dtype, int y_dtype, const void* dy, const void* x, const float* w, const float* mean,
                          const float* rstd, const void* res, void* dx, float* dw, float* db, long rows, int dim,
                          float* ws, cudaStream_t s) {
  if (rows == 0) {
    cudaError_t e = dw != nullptr ? cudaMemsetAsync(dw, 0, sizeof(float) * (size_t)dim, s) : cudaSuccess;
    if (e == cudaSuccess && db != nullptr) e = cudaMemsetAsync(db, 0, sizeof(float) * (size_t)dim, s);
    return e;
  }
  const Args a{dy, x, res, w, mean, rstd, dx, dw, db, ws, rows, dim};
  if (x_dtype == DTYPE_F32) {
    if (y_dtype == DTYPE_F32) return bwd_t<float, float>(a, s);
    if (y_dtype == DTYPE_F16) return bwd_t<float, __half>(a, s);
    return bwd_t<float, __nv_bfloat16>(a, s);
  }
  if (x_dtype == DTYPE_F16) return bwd_t<__half, __half>(a, s);
  return bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace jepa
