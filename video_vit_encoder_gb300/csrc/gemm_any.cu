// General matrix product on the CUDA cores, fp32 accumulation (FFMA, no TF32):
// C[m, n] (+)= sum_k A(m, k) B(n, k) (+ bias[n]), each operand contiguous along
// either of its two dimensions, in fp32 or a 16-bit type.
//
// The path of the training operators in fp32, and in 16-bit types where rows do
// not start on 16 bytes (the tensor-core path reads tiles with TMA).  128 x 128
// outputs per 256-thread block, 8 x 8 per thread as packed f32x2 products, K in
// slices of 16 staged through two shared-memory buffers while the next slice
// is loaded into registers.  Bound by the FFMA rate.
#include "train.h"

namespace jepa {

namespace {

constexpr int BM = 128, BN = 128, BK = 16, kThreads = 256;
constexpr int kPad = 4;

__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t dup2(float a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
  return r;
}

// Four consecutive elements from p, of which the first `n` exist.
template <typename T>
__device__ __forceinline__ void load4(const T* p, int n, bool vec, float (&v)[4]) {
  if (vec && n >= 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      T h[4];
      memcpy(h, &q, 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = DT<T>::to(h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? DT<T>::to(p[i]) : 0.f;
  }
}

// This thread's 8 elements of the 128 x 16 slice at (r0, k0), as two groups of
// four along the contiguous dimension.
template <typename T, bool KMAJ>
__device__ __forceinline__ void load_slice(const T* p, long ld, int r0, int k0, int R, int K, bool vec,
                                           float (&v)[2][4]) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (KMAJ) {
      const int r = r0 + (tid >> 2) + 64 * h, k = k0 + (tid & 3) * 4;
      const int n = r < R ? K - k : 0;
      load4<T>(p + (n > 0 ? (long)r * ld + k : 0), n, vec, v[h]);
    } else {
      const int k = k0 + (tid >> 5) + 8 * h, r = r0 + (tid & 31) * 4;
      const int n = k < K ? R - r : 0;
      load4<T>(p + (n > 0 ? (long)k * ld + r : 0), n, vec, v[h]);
    }
  }
}
template <bool KMAJ>
__device__ __forceinline__ void store_slice(float (*s)[BM + kPad], const float (&v)[2][4]) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (KMAJ) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[(tid & 3) * 4 + i][(tid >> 2) + 64 * h] = v[h][i];
    } else {
      *reinterpret_cast<float4*>(&s[(tid >> 5) + 8 * h][(tid & 31) * 4]) =
          make_float4(v[h][0], v[h][1], v[h][2], v[h][3]);
    }
  }
}

template <typename TA, typename TB, typename TC, bool AK, bool BKM>
__global__ void __launch_bounds__(kThreads, 2)
    gemm_any_kernel(const TA* __restrict__ A, long lda, const TB* __restrict__ B, long ldb, TC* __restrict__ C, long ldc,
                    int M, int N, int K, const float* __restrict__ bias, int accumulate, int avec, int bvec) {
  __shared__ __align__(16) float As[2][BK][BM + kPad];
  __shared__ __align__(16) float Bs[2][BK][BN + kPad];
  const int tiles_n = (N + BN - 1) / BN;
  const int m0 = (int)(blockIdx.x / tiles_n) * BM, n0 = (int)(blockIdx.x % tiles_n) * BN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  uint64_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
  float ra[2][4], rb[2][4];
  load_slice<TA, AK>(A, lda, m0, 0, M, K, avec, ra);
  load_slice<TB, BKM>(B, ldb, n0, 0, N, K, bvec, rb);
  store_slice<AK>(As[0], ra);
  store_slice<BKM>(Bs[0], rb);
  __syncthreads();
  int buf = 0;
  for (int k0 = 0; k0 < K; k0 += BK) {
    const bool more = k0 + BK < K;
    if (more) {
      load_slice<TA, AK>(A, lda, m0, k0 + BK, M, K, avec, ra);
      load_slice<TB, BKM>(B, ldb, n0, k0 + BK, N, K, bvec, rb);
    }
#pragma unroll
    for (int kk = 0; kk < BK; ++kk) {
      const float4 a0 = *reinterpret_cast<const float4*>(&As[buf][kk][ty * 4]);
      const float4 a1 = *reinterpret_cast<const float4*>(&As[buf][kk][64 + ty * 4]);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(&Bs[buf][kk][tx * 4]);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(&Bs[buf][kk][64 + tx * 4]);
      const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      const uint64_t b[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t aa = dup2(a[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) fma2(acc[i][j], aa, b[j]);
      }
    }
    if (more) {
      store_slice<AK>(As[buf ^ 1], ra);
      store_slice<BKM>(Bs[buf ^ 1], rb);
      __syncthreads();
      buf ^= 1;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + (i < 4 ? ty * 4 + i : 64 + ty * 4 + i - 4);
    if (m >= M) continue;
    TC* row = C + (long)m * ldc;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + (j < 2 ? tx * 4 + 2 * j : 64 + tx * 4 + 2 * (j - 2));
      float v[2];
      memcpy(v, &acc[i][j], 8);
#pragma unroll
      for (int l = 0; l < 2; ++l)
        if (n + l < N) {
          float o = v[l];
          if (bias != nullptr) o += __ldg(bias + n + l);
          if constexpr (sizeof(TC) == 4) {
            if (accumulate) o += row[n + l];
          }
          row[n + l] = DT<TC>::from(o);
        }
    }
  }
}

// Whether four consecutive elements of every row start on their own size.
bool vec4_ok(const void* p, long ld, size_t elem) {
  return (reinterpret_cast<uintptr_t>(p) % (4 * elem)) == 0 && ld % 4 == 0;
}

template <typename TA, typename TB, typename TC>
cudaError_t any_t(const AnyMat& A, const AnyMat& B, void* C, long ldc, int M, int N, int K, const float* bias,
                  bool accumulate, cudaStream_t s) {
  const bool ak = A.ks == 1, bk = B.ks == 1;
  const long lda = ak ? A.rs : A.ks, ldb = bk ? B.rs : B.ks;
  const int av = vec4_ok(A.p, lda, sizeof(TA)), bv = vec4_ok(B.p, ldb, sizeof(TB));
  const TA* a = static_cast<const TA*>(A.p);
  const TB* b = static_cast<const TB*>(B.p);
  TC* c = static_cast<TC*>(C);
  const long blocks = (long)((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  if (blocks > 0x7fffffffl) return cudaErrorInvalidValue;
  const dim3 g((unsigned)blocks);
  if (ak && bk)
    gemm_any_kernel<TA, TB, TC, true, true><<<g, kThreads, 0, s>>>(a, lda, b, ldb, c, ldc, M, N, K, bias, accumulate, av, bv);
  else if (ak)
    gemm_any_kernel<TA, TB, TC, true, false><<<g, kThreads, 0, s>>>(a, lda, b, ldb, c, ldc, M, N, K, bias, accumulate, av, bv);
  else if (bk)
    gemm_any_kernel<TA, TB, TC, false, true><<<g, kThreads, 0, s>>>(a, lda, b, ldb, c, ldc, M, N, K, bias, accumulate, av, bv);
  else
    gemm_any_kernel<TA, TB, TC, false, false><<<g, kThreads, 0, s>>>(a, lda, b, ldb, c, ldc, M, N, K, bias, accumulate, av, bv);
  return cudaGetLastError();
}

// T: the operator's type.  A and B are T, or A is an fp32 intermediate of it.
template <typename T>
cudaError_t any_dtype(const AnyMat& A, const AnyMat& B, void* C, int c_dtype, long ldc, int M, int N, int K,
                      const float* bias, bool accumulate, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (A.dtype == DTYPE_F32)
      return c_dtype == DTYPE_F32 ? any_t<float, T, float>(A, B, C, ldc, M, N, K, bias, accumulate, s)
                                  : any_t<float, T, T>(A, B, C, ldc, M, N, K, bias, false, s);
    if (c_dtype != DTYPE_F32) return any_t<T, T, T>(A, B, C, ldc, M, N, K, bias, false, s);
  }
  return any_t<T, T, float>(A, B, C, ldc, M, N, K, bias, accumulate, s);
}

}  // namespace

cudaError_t gemm_any(const AnyMat& A, const AnyMat& B, void* C, int c_dtype, long ldc, int M, int N, int K,
                     const float* bias, bool accumulate, cudaStream_t s) {
  if (M == 0 || N == 0) return cudaSuccess;
  if (accumulate && c_dtype != DTYPE_F32) return cudaErrorInvalidValue;
  switch (B.dtype) {
    case DTYPE_F32: return any_dtype<float>(A, B, C, c_dtype, ldc, M, N, K, bias, accumulate, s);
    case DTYPE_F16: return any_dtype<__half>(A, B, C, c_dtype, ldc, M, N, K, bias, accumulate, s);
    case DTYPE_BF16: return any_dtype<__nv_bfloat16>(A, B, C, c_dtype, ldc, M, N, K, bias, accumulate, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace jepa
