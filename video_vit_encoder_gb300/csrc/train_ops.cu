// The training operators on the CUDA cores: the path of fp32, and of 16-bit
// operands whose rows do not start on 16 bytes.
//
// Each works over pieces of its wide dimension (the vocabulary, the hidden
// width): the piece's products go to an fp32 workspace, a row-wise kernel
// turns them into what the piece contributes, and further products reduce
// that.  The workspace holds one piece, never the whole [rows, width] matrix.
// The products (gemm_any.cu) take nearly all the time, so the kernels here
// are plain single passes.
#include "train_tc.h"

namespace jepa {

namespace {

constexpr int kBlock = 256;
constexpr float kLog2e = 1.4426950408889634f;

size_t larger(size_t a, size_t b) { return a > b ? a : b; }
size_t align256(size_t n) { return (n + 255) & ~size_t(255); }
size_t elem(int dtype) { return dtype == DTYPE_F32 ? 4 : 2; }
unsigned blocks_for(long n, int block) { return (unsigned)((n + block - 1) / block); }

AnyMat rows_k(const void* p, int dtype, long ld) { return AnyMat{p, dtype, ld, 1}; }  // p is [r, k]
AnyMat k_rows(const void* p, int dtype, long ld) { return AnyMat{p, dtype, 1, ld}; }  // p is [k, r]

// Columns of the wide dimension (of `total`) per piece: a multiple of 128 of
// which `bufs` fp32 arrays of M rows stay within 64 MB (they then live in L2
// between the kernels that write and read them), but at least 1024 columns,
// so that each product still fills the machine.
int piece_cols(int M, int total, int bufs) {
  const size_t per = sizeof(float) * (size_t)bufs * (M > 0 ? M : 1);
  size_t c = ((size_t)64 << 20) / per / 128 * 128;
  if (c < 1024) c = 1024;
  const size_t all = ((size_t)total + 127) / 128 * 128;
  return (int)(c < all ? c : all);
}

// ----------------------------------------------------------------------------- column sums
// out[c] = sum over the rows of a[r, c]: 32 columns a block, 8 threads a
// column, each over every eighth row, joined in a fixed order.
template <typename T>
__global__ void __launch_bounds__(kBlock) col_sum_kernel(const T* __restrict__ a, long ld, int M, int n,
                                                         float* __restrict__ out) {
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < n)
    for (int r = g; r < M; r += 8) s += DT<T>::to(a[(long)r * ld + c]);
  sm[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < n) {
    for (int k = 1; k < 8; ++k) s += sm[k][lane];
    out[c] = s;
  }
}
cudaError_t col_sum(const void* a, int dtype, long ld, int M, int n, float* out, cudaStream_t s) {
  const unsigned b = blocks_for(n, 32);
  if (dtype == DTYPE_F32) col_sum_kernel<float><<<b, kBlock, 0, s>>>((const float*)a, ld, M, n, out);
  else if (dtype == DTYPE_F16) col_sum_kernel<__half><<<b, kBlock, 0, s>>>((const __half*)a, ld, M, n, out);
  else col_sum_kernel<__nv_bfloat16><<<b, kBlock, 0, s>>>((const __nv_bfloat16*)a, ld, M, n, out);
  return cudaGetLastError();
}

template <typename T>
__global__ void cast_kernel(const float* __restrict__ a, T* __restrict__ out, long n) {
  const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) out[i] = DT<T>::from(a[i]);
}
cudaError_t cast_to(const float* a, int dtype, void* out, long n, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  if (dtype == DTYPE_F16) cast_kernel<__half><<<blocks_for(n, kBlock), kBlock, 0, s>>>(a, (__half*)out, n);
  else cast_kernel<__nv_bfloat16><<<blocks_for(n, kBlock), kBlock, 0, s>>>(a, (__nv_bfloat16*)out, n);
  return cudaGetLastError();
}

// ----------------------------------------------------------------------------- softmax cross entropy
// Label of a row: -1 for a row that takes no part (ignored, or bad).
__device__ __forceinline__ long row_label(long label, long ignore_index, int V) {
  return label == ignore_index || label < 0 || label >= V ? -1 : label;
}

// Running statistics of a row over the pieces seen so far: the max m of its
// logits, sum of exp(z - m), sum of z, and the label's logit.
struct CeState {
  float m, s, sum, zy;
};

// Joins (m, s) with (m2, s2); a side that has seen nothing but -inf has s = 0.
__device__ __forceinline__ void ce_join(float& m, float& s, float m2, float s2) {
  const float mm = fmaxf(m, m2);
  // exp(-inf - -inf) would be NaN: nothing has been summed on that side
  const float f1 = m == -INFINITY ? 0.f : exp2f((m - mm) * kLog2e);
  const float f2 = m2 == -INFINITY ? 0.f : exp2f((m2 - mm) * kLog2e);
  s = (m == -INFINITY ? 0.f : s * f1) + (m2 == -INFINITY ? 0.f : s2 * f2);
  m = mm;
}

// One block a row: adds the piece's logits z[row, 0:n) (columns v0..) to the state.
__global__ void __launch_bounds__(kBlock) ce_piece_kernel(const float* __restrict__ z, long ld, int n, int v0, int V,
                                                          const int64_t* __restrict__ labels, long ignore_index,
                                                          CeState* __restrict__ state, int first) {
  __shared__ float sm[3][kBlock / 32];
  const long row = blockIdx.x;
  const float* zr = z + row * ld;
  float m = -INFINITY, s = 0.f, sum = 0.f;
  bool nan = false;
  for (int c = threadIdx.x; c < n; c += kBlock) {
    const float v = zr[c];
    nan |= v != v;
    sum += v;
    m = fmaxf(m, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sm[0][warp] = m;
  __syncthreads();
  for (int k = 0; k < kBlock / 32; ++k) m = fmaxf(m, sm[0][k]);
  if (m != -INFINITY)
    for (int c = threadIdx.x; c < n; c += kBlock) s += exp2f((zr[c] - m) * kLog2e);
  if (nan) s = NAN;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  if (lane == 0) {
    sm[1][warp] = s;
    sm[2][warp] = sum;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    s = sum = 0.f;
    for (int k = 0; k < kBlock / 32; ++k) {
      s += sm[1][k];
      sum += sm[2][k];
    }
    if (s != s) m = NAN;
    CeState st = first ? CeState{-INFINITY, 0.f, 0.f, 0.f} : state[row];
    if (m != m || st.m != st.m) {
      st.m = NAN;
    } else {
      ce_join(st.m, st.s, m, s);
    }
    st.sum += sum;
    const long y = row_label(labels[row], ignore_index, V);
    if (y >= v0 && y < (long)v0 + n) st.zy = zr[y - v0];
    state[row] = st;
  }
}

// loss = lse - (1 - e) z_y - e mean(z); 0 for an ignored row, NaN (and the
// status bit) for a label outside [0, V).
__global__ void ce_finish_kernel(const CeState* __restrict__ state, const int64_t* __restrict__ labels, int M, int V,
                                 long ignore_index, float smoothing, float* __restrict__ loss,
                                 float* __restrict__ lse_out, int* status) {
  const int row = blockIdx.x * blockDim.x + threadIdx.x;
  if (row >= M) return;
  const CeState st = state[row];
  const float lse = st.m == -INFINITY ? -INFINITY : st.m + logf(st.s);
  const long label = labels[row];
  float l;
  if (label == ignore_index) {
    l = 0.f;
  } else if (label < 0 || label >= V) {
    l = NAN;
    atomicOr(status, DEV_BAD_INDEX);
  } else {
    l = lse - (1.0f - smoothing) * st.zy;
    if (smoothing > 0.f) l -= smoothing * (st.sum / (float)V);
  }
  if (loss != nullptr) loss[row] = l;
  if (lse_out != nullptr) lse_out[row] = lse;
}

// z -> dz in place: dz = dloss (exp(z - lse) - (1 - e) [v == y] - e / V); rows
// that take no part get zeros.
__global__ void __launch_bounds__(kBlock) ce_grad_kernel(float* __restrict__ z, long ld, int n, int v0, int V,
                                                         const int64_t* __restrict__ labels, long ignore_index,
                                                         const float* __restrict__ lse,
                                                         const float* __restrict__ dloss, float smoothing,
                                                         int* status) {
  const long row = blockIdx.x;
  float* zr = z + row * ld;
  const long label = labels[row];
  const long y = row_label(label, ignore_index, V);
  if (y < 0) {
    if (threadIdx.x == 0 && label != ignore_index) atomicOr(status, DEV_BAD_INDEX);
    for (int c = threadIdx.x; c < n; c += kBlock) zr[c] = 0.f;
    return;
  }
  const float l = lse[row], g = dloss[row], uni = smoothing / (float)V;
  for (int c = threadIdx.x; c < n; c += kBlock) {
    float d = exp2f((zr[c] - l) * kLog2e) - uni;
    if (v0 + c == y) d -= 1.0f - smoothing;
    zr[c] = d * g;
  }
}

// ----------------------------------------------------------------------------- gate
__device__ __forceinline__ void gate_value(int act, float g, float& a, float& da) {
  if (act == ACT_SILU) {
    const float s = 1.0f / (1.0f + __expf(-g));
    a = g * s;
    da = s * (1.0f + g * (1.0f - s));
  } else {
    const float cdf = 0.5f * (1.0f + erff(g * 0.70710678118654752f));
    a = g * cdf;
    da = cdf + g * 0.3989422804014327f * __expf(-0.5f * g * g);
  }
}

template <typename T>
__global__ void gate_fwd_kernel(const float* __restrict__ g, const float* __restrict__ u, long ld, int M, int n, int act,
                                T* __restrict__ h, long ldh) {
  const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long)M * n) return;
  const long r = i / n, c = i - r * n;
  float a, da;
  gate_value(act, g[r * ld + c], a, da);
  h[r * ldh + c] = DT<T>::from(a * u[r * ld + c]);
}

// g, u -> dg, du in place.
template <typename T>
__global__ void gate_bwd_kernel(float* __restrict__ g, float* __restrict__ u, long ld, int M, int n, int act,
                                const T* __restrict__ dh, long ldh) {
  const long i = (long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (long)M * n) return;
  const long r = i / n, c = i - r * n;
  float a, da;
  gate_value(act, g[r * ld + c], a, da);
  const float d = DT<T>::to(dh[r * ldh + c]);
  g[r * ld + c] = d * u[r * ld + c] * da;
  u[r * ld + c] = d * a;
}

#define JEPA_TRY_CUDA(expr)                 \
  do {                                      \
    const cudaError_t e_ = (expr);          \
    if (e_ != cudaSuccess) return e_;       \
  } while (0)

cudaError_t zero(void* p, size_t bytes, cudaStream_t s) {
  return p == nullptr || bytes == 0 ? cudaSuccess : cudaMemsetAsync(p, 0, bytes, s);
}

}  // namespace

// ----------------------------------------------------------------------------- softmax cross entropy
// Workspace: the rows' state (forward), the piece's logits, and (backward,
// 16-bit) the fp32 sum of dx over the pieces.
size_t linear_ce_workspace(int M, int D, int V, int dtype, bool backward) {
  const size_t z = align256(sizeof(float) * (size_t)M * piece_cols(M, V, 1));
  size_t b = backward ? z + (dtype == DTYPE_F32 ? 0 : align256(sizeof(float) * (size_t)M * D))
                      : align256(sizeof(CeState) * (size_t)M) + z;
  return dtype != DTYPE_F32 && D % 8 == 0 ? larger(b, linear_ce_tc_workspace(M, D, V, backward)) : b;
}

cudaError_t linear_ce_fwd(const CeArgs& a, float* loss, float* lse, void* ws, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  if (linear_ce_tc_ok(a, nullptr, nullptr)) return linear_ce_fwd_tc(a, loss, lse, ws, s);
  CeState* state = static_cast<CeState*>(ws);
  float* z = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align256(sizeof(CeState) * (size_t)a.M));
  const int pc = piece_cols(a.M, a.V, 1);
  const AnyMat x = rows_k(a.x, a.dtype, a.D);
  for (int v0 = 0; v0 < a.V; v0 += pc) {
    const int n = a.V - v0 < pc ? a.V - v0 : pc;
    const AnyMat w = rows_k(static_cast<const uint8_t*>(a.w) + elem(a.dtype) * (size_t)v0 * a.D, a.dtype, a.D);
    JEPA_TRY_CUDA(gemm_any(x, w, z, DTYPE_F32, pc, a.M, n, a.D, a.bias ? a.bias + v0 : nullptr, false, s));
    ce_piece_kernel<<<a.M, kBlock, 0, s>>>(z, pc, n, v0, a.V, a.labels, a.ignore_index, state, v0 == 0);
    JEPA_TRY_CUDA(cudaGetLastError());
  }
  ce_finish_kernel<<<blocks_for(a.M, kBlock), kBlock, 0, s>>>(state, a.labels, a.M, a.V, a.ignore_index, a.smoothing,
                                                              loss, lse, a.status);
  return cudaGetLastError();
}

cudaError_t linear_ce_bwd(const CeArgs& a, const float* lse, const float* dloss, void* dx, void* dw, float* dbias,
                          void* ws, cudaStream_t s) {
  const size_t es = elem(a.dtype);
  if (a.M == 0) {
    JEPA_TRY_CUDA(zero(dw, es * (size_t)a.V * a.D, s));
    return zero(dbias, sizeof(float) * (size_t)a.V, s);
  }
  if (linear_ce_tc_ok(a, dx, dw)) return linear_ce_bwd_tc(a, lse, dloss, dx, dw, dbias, ws, s);
  const int pc = piece_cols(a.M, a.V, 1);
  float* z = static_cast<float*>(ws);
  float* dxa = a.dtype == DTYPE_F32
                   ? static_cast<float*>(dx)
                   : reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align256(sizeof(float) * (size_t)a.M * pc));
  const AnyMat x = rows_k(a.x, a.dtype, a.D);
  for (int v0 = 0; v0 < a.V; v0 += pc) {
    const int n = a.V - v0 < pc ? a.V - v0 : pc;
    const uint8_t* wp = static_cast<const uint8_t*>(a.w) + es * (size_t)v0 * a.D;
    JEPA_TRY_CUDA(gemm_any(x, rows_k(wp, a.dtype, a.D), z, DTYPE_F32, pc, a.M, n, a.D, a.bias ? a.bias + v0 : nullptr,
                           false, s));
    ce_grad_kernel<<<a.M, kBlock, 0, s>>>(z, pc, n, v0, a.V, a.labels, a.ignore_index, lse, dloss, a.smoothing,
                                          a.status);
    JEPA_TRY_CUDA(cudaGetLastError());
    if (dx != nullptr)
      JEPA_TRY_CUDA(gemm_any(rows_k(z, DTYPE_F32, pc), k_rows(wp, a.dtype, a.D), dxa, DTYPE_F32, a.D, a.M, a.D, n,
                             nullptr, v0 != 0, s));
    if (dw != nullptr)
      JEPA_TRY_CUDA(gemm_any(k_rows(z, DTYPE_F32, pc), k_rows(a.x, a.dtype, a.D),
                             static_cast<uint8_t*>(dw) + es * (size_t)v0 * a.D, a.dtype, a.D, n, a.D, a.M, nullptr,
                             false, s));
    if (dbias != nullptr) JEPA_TRY_CUDA(col_sum(z, DTYPE_F32, pc, a.M, n, dbias + v0, s));
  }
  if (dx != nullptr && a.dtype != DTYPE_F32) JEPA_TRY_CUDA(cast_to(dxa, a.dtype, dx, (long)a.M * a.D, s));
  return cudaSuccess;
}

// ----------------------------------------------------------------------------- gated feed-forward
// Workspace: the piece's two projections, and (backward, 16-bit) the fp32 sum
// of dx over the pieces.
size_t gated_ffn_workspace(int M, int D, int F, int dtype, bool backward) {
  size_t b = 2 * align256(sizeof(float) * (size_t)M * piece_cols(M, F, 2));
  if (backward && dtype != DTYPE_F32) b += align256(sizeof(float) * (size_t)M * D);
  return dtype != DTYPE_F32 && D % 8 == 0 && F % 8 == 0 ? larger(b, gated_ffn_tc_workspace(M, D, F, backward)) : b;
}

namespace {

struct FfnPiece {
  float *g, *u;
  int pc;
};
FfnPiece ffn_buffers(const FfnArgs& a, void* ws) {
  FfnPiece p;
  p.pc = piece_cols(a.M, a.F, 2);
  p.g = static_cast<float*>(ws);
  p.u = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align256(sizeof(float) * (size_t)a.M * p.pc));
  return p;
}
cudaError_t ffn_project(const FfnArgs& a, const FfnPiece& p, int f0, int n, cudaStream_t s) {
  const size_t off = elem(a.dtype) * (size_t)f0 * a.D;
  const AnyMat x = rows_k(a.x, a.dtype, a.D);
  JEPA_TRY_CUDA(gemm_any(x, rows_k(static_cast<const uint8_t*>(a.wg) + off, a.dtype, a.D), p.g, DTYPE_F32, p.pc, a.M, n,
                         a.D, a.bg ? a.bg + f0 : nullptr, false, s));
  return gemm_any(x, rows_k(static_cast<const uint8_t*>(a.wu) + off, a.dtype, a.D), p.u, DTYPE_F32, p.pc, a.M, n, a.D,
                  a.bu ? a.bu + f0 : nullptr, false, s);
}

}  // namespace

cudaError_t gated_ffn_fwd(const FfnArgs& a, void* h, void* ws, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  if (gated_ffn_tc_ok(a, h, nullptr, nullptr, nullptr)) return gated_ffn_fwd_tc(a, h, s);
  const FfnPiece p = ffn_buffers(a, ws);
  for (int f0 = 0; f0 < a.F; f0 += p.pc) {
    const int n = a.F - f0 < p.pc ? a.F - f0 : p.pc;
    JEPA_TRY_CUDA(ffn_project(a, p, f0, n, s));
    const unsigned b = blocks_for((long)a.M * n, kBlock);
    if (a.dtype == DTYPE_F32)
      gate_fwd_kernel<float><<<b, kBlock, 0, s>>>(p.g, p.u, p.pc, a.M, n, a.act, (float*)h + f0, a.F);
    else if (a.dtype == DTYPE_F16)
      gate_fwd_kernel<__half><<<b, kBlock, 0, s>>>(p.g, p.u, p.pc, a.M, n, a.act, (__half*)h + f0, a.F);
    else
      gate_fwd_kernel<__nv_bfloat16><<<b, kBlock, 0, s>>>(p.g, p.u, p.pc, a.M, n, a.act, (__nv_bfloat16*)h + f0, a.F);
    JEPA_TRY_CUDA(cudaGetLastError());
  }
  return cudaSuccess;
}

cudaError_t gated_ffn_bwd(const FfnArgs& a, const void* dh, void* dx, void* dwg, void* dwu, float* dbg, float* dbu,
                          void* ws, cudaStream_t s) {
  const size_t es = elem(a.dtype);
  if (a.M == 0) {
    JEPA_TRY_CUDA(zero(dwg, es * (size_t)a.F * a.D, s));
    JEPA_TRY_CUDA(zero(dwu, es * (size_t)a.F * a.D, s));
    JEPA_TRY_CUDA(zero(dbg, sizeof(float) * (size_t)a.F, s));
    return zero(dbu, sizeof(float) * (size_t)a.F, s);
  }
  if (gated_ffn_tc_ok(a, dh, dx, dwg, dwu)) return gated_ffn_bwd_tc(a, dh, dx, dwg, dwu, dbg, dbu, ws, s);
  const FfnPiece p = ffn_buffers(a, ws);
  float* dxa = a.dtype == DTYPE_F32
                   ? static_cast<float*>(dx)
                   : reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 2 * align256(sizeof(float) * (size_t)a.M * p.pc));
  for (int f0 = 0; f0 < a.F; f0 += p.pc) {
    const int n = a.F - f0 < p.pc ? a.F - f0 : p.pc;
    JEPA_TRY_CUDA(ffn_project(a, p, f0, n, s));
    const unsigned b = blocks_for((long)a.M * n, kBlock);
    if (a.dtype == DTYPE_F32)
      gate_bwd_kernel<float><<<b, kBlock, 0, s>>>(p.g, p.u, p.pc, a.M, n, a.act, (const float*)dh + f0, a.F);
    else if (a.dtype == DTYPE_F16)
      gate_bwd_kernel<__half><<<b, kBlock, 0, s>>>(p.g, p.u, p.pc, a.M, n, a.act, (const __half*)dh + f0, a.F);
    else
      gate_bwd_kernel<__nv_bfloat16><<<b, kBlock, 0, s>>>(p.g, p.u, p.pc, a.M, n, a.act, (const __nv_bfloat16*)dh + f0, a.F);
    JEPA_TRY_CUDA(cudaGetLastError());
    const size_t off = es * (size_t)f0 * a.D;
    for (int k = 0; k < 2; ++k) {
      const float* d = k == 0 ? p.g : p.u;
      const uint8_t* w = static_cast<const uint8_t*>(k == 0 ? a.wg : a.wu) + off;
      void* dw = k == 0 ? dwg : dwu;
      float* db = k == 0 ? dbg : dbu;
      if (dx != nullptr)
        JEPA_TRY_CUDA(gemm_any(rows_k(d, DTYPE_F32, p.pc), k_rows(w, a.dtype, a.D), dxa, DTYPE_F32, a.D, a.M, a.D, n,
                               nullptr, f0 != 0 || k != 0, s));
      if (dw != nullptr)
        JEPA_TRY_CUDA(gemm_any(k_rows(d, DTYPE_F32, p.pc), k_rows(a.x, a.dtype, a.D), static_cast<uint8_t*>(dw) + off,
                               a.dtype, a.D, n, a.D, a.M, nullptr, false, s));
      if (db != nullptr) JEPA_TRY_CUDA(col_sum(d, DTYPE_F32, p.pc, a.M, n, db + f0, s));
    }
  }
  if (dx != nullptr && a.dtype != DTYPE_F32) JEPA_TRY_CUDA(cast_to(dxa, a.dtype, dx, (long)a.M * a.D, s));
  return cudaSuccess;
}

// ----------------------------------------------------------------------------- linear layer backward
size_t linear_bwd_workspace(int M, int N, int K, int dtype) {
  return dtype != DTYPE_F32 && N % 8 == 0 && K % 8 == 0 ? linear_bwd_tc_workspace(M, N, K) : 0;
}

cudaError_t linear_bwd(int dtype, const void* dout, const void* A, const void* W, void* dA, void* dW, float* dbias,
                       int M, int N, int K, void* ws, int* status, int num_sms, cudaStream_t s) {
  if (M == 0) {
    JEPA_TRY_CUDA(zero(dW, elem(dtype) * (size_t)N * K, s));
    return zero(dbias, sizeof(float) * (size_t)N, s);
  }
  if (linear_bwd_tc_ok(dtype, dout, A, W, dA, dW, N, K))
    return linear_bwd_tc(dtype, dout, A, W, dA, dW, dbias, M, N, K, ws, status, num_sms, s);
  if (dA != nullptr)
    JEPA_TRY_CUDA(gemm_any(rows_k(dout, dtype, N), k_rows(W, dtype, K), dA, dtype, K, M, K, N, nullptr, false, s));
  if (dW != nullptr)
    JEPA_TRY_CUDA(gemm_any(k_rows(dout, dtype, N), k_rows(A, dtype, K), dW, dtype, K, N, K, M, nullptr, false, s));
  if (dbias != nullptr) JEPA_TRY_CUDA(col_sum(dout, dtype, N, M, N, dbias, s));
  return cudaSuccess;
}

}  // namespace jepa
