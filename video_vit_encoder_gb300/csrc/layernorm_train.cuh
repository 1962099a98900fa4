// Row access shared by the layer norm's forward and backward kernels.
//
// A row of `dim` values is held in registers by TPR threads (one warp, or a
// whole block), each owning NV vectors of V consecutive columns (16 bytes of
// the widest operand).  Where dim is a multiple of V, vector i of thread t
// starts at column (t + i * TPR) * V.  Where it is not, rows start at any
// element, so the vectors are laid on the aligned memory under the row: they
// start at column (t + i * TPR) * V - o with o = (row * dim) mod V, and the
// first and last one share their memory with the neighbouring rows.  A
// thread's rows are a multiple of V apart, so o, and with it the columns a
// thread owns, are the same for all its rows.  Operands that do not start on
// their vector take V = 1.
#pragma once
#include "train.h"

namespace jepa {

template <typename T, int V>
__device__ __forceinline__ void ln_load(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = DT<T>::to(*p);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 q = reinterpret_cast<const float4*>(p)[i];
      v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
    }
  } else {
    uint32_t u[V / 2];
    if constexpr (V == 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      u[0] = q.x; u[1] = q.y; u[2] = q.z; u[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      u[0] = q.x; u[1] = q.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      T h[2];
      memcpy(h, &u[i], 4);
      v[2 * i] = DT<T>::to(h[0]);
      v[2 * i + 1] = DT<T>::to(h[1]);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void ln_store(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = DT<T>::from(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  }
}

__device__ __forceinline__ float ln_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of N values over the TPR threads of a row; every thread gets them.
// With TPR > 32 the row is the block's: red holds N x (TPR / 32) floats and
// every thread of the block calls this.
template <int TPR, int N>
__device__ __forceinline__ void ln_row_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = ln_warp_sum(v[j]);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();   // the previous sum has been read
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < N; ++j) red[j * W + warp] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) s += red[j * W + i];
      v[j] = s;
    }
  }
}

// Shared memory is filled with the vector at p, of which the first `bytes`
// bytes exist (the rest become zeros).
template <int N>
__device__ __forceinline__ void ln_copy_async(void* dst, const void* p, int bytes) {
  static_assert(N == 8 || N == 16, "vector size");
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(p), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ln_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ln_copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Whether a vector whose first column is c0 lies inside the row as a whole.
template <int V>
__device__ __forceinline__ bool ln_whole(int c0, int dim) {
  return c0 >= 0 && c0 + V <= dim;
}
// Stores the part of a vector that lies inside the row.
template <typename T, int V>
__device__ __forceinline__ void ln_store_part(T* row, int c0, int dim, const float (&v)[V]) {
  if (ln_whole<V>(c0, dim)) {
    ln_store<T, V>(row + c0, v);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c0 + j >= 0 && c0 + j < dim) row[c0 + j] = DT<T>::from(v[j]);
  }
}

inline bool ln_aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline size_t ln_size(int dtype) { return dtype == DTYPE_F32 ? 4 : 2; }

}  // namespace jepa
