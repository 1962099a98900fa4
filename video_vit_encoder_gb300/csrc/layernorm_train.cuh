// Row access shared by the layer norm's forward and backward kernels.
//
// A row of `dim` values is the work of TPR threads (one warp to a block), each
// owning NV vectors of V consecutive columns (16 bytes of the widest operand).
// Where dim is a multiple of V, vector i of thread t starts at column
// (t + i * TPR) * V.  Where it is not (SHIFT), rows start at any element, so
// the vectors are laid on the aligned memory under the row: they start at
// column (t + i * TPR) * V - o with o = (row * dim) mod V, and the first and
// last one share their memory with the neighbouring rows.  A thread's rows are
// a multiple of V apart, so o, and with it the columns a thread owns, are the
// same for all its rows.  Operands that do not start on their vector, and rows
// of more than 8192 columns, have kernels of their own.
#pragma once
#include "train.h"

namespace jepa {

// V values from or to 16 bytes or a multiple of them; 16-bit results of four
// fp32 values take 8.
template <typename T, int V>
__device__ __forceinline__ void ln_load(const T* p, float (&v)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 q = reinterpret_cast<const float4*>(p)[i];
      v[4 * i] = q.x; v[4 * i + 1] = q.y; v[4 * i + 2] = q.z; v[4 * i + 3] = q.w;
    }
  } else {
    static_assert(V == 8, "16 bytes");
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T h[2];
      memcpy(h, &u[i], 4);
      v[2 * i] = DT<T>::to(h[0]);
      v[2 * i + 1] = DT<T>::to(h[1]);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void ln_store(T* p, const float (&v)[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  } else {
    static_assert(V == 4, "8 bytes");
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  }
}

// Two neighbouring fp32 values in one register pair; the rows' arithmetic is
// packed, because it is instruction issue that bounds it.
using f2 = uint64_t;
__device__ __forceinline__ f2 f2_make(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(f2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
  float a, b;
  f2_get(v, a, b);
  return a + b;
}

// The 32-bit words of a vector of V values, and their values in pairs.
template <typename T, int V>
struct LnVec {
  static constexpr int kWords = V * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (kWords == 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x; w[1] = q.y;
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (kWords == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  // Zeros in place of the first n values.
  __device__ __forceinline__ void drop_head(int n) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      if constexpr (sizeof(T) == 4) w[k] = k < n ? 0u : w[k];
      else w[k] &= 2 * k + 1 < n ? 0u : (2 * k < n ? 0xffff0000u : 0xffffffffu);
    }
  }
  __device__ __forceinline__ void pairs(f2 (&v)[V / 2]) const {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      if constexpr (sizeof(T) == 4) {
        asm("mov.b64 %0, {%1, %2};" : "=l"(v[k]) : "r"(w[2 * k]), "r"(w[2 * k + 1]));
      } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        asm("mov.b64 %0, {%1, %2};" : "=l"(v[k]) : "r"(w[k] << 16), "r"(w[k] & 0xffff0000u));
      } else {
        T h[2];
        memcpy(h, &w[k], 4);
        v[k] = f2_make(DT<T>::to(h[0]), DT<T>::to(h[1]));
      }
    }
  }
  __device__ __forceinline__ void set(const f2 (&v)[V / 2]) {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      float a, b;
      f2_get(v[k], a, b);
      if constexpr (sizeof(T) == 4) {
        w[2 * k] = __float_as_uint(a);
        w[2 * k + 1] = __float_as_uint(b);
      } else {
        w[k] = pack2<T>(a, b);
      }
    }
  }
};
// Four to eight consecutive floats in pairs.
template <int V>
__device__ __forceinline__ void ln_floats(const float* p, f2 (&v)[V / 2]) {
#pragma unroll
  for (int j = 0; j < V / 4; ++j) {
    const ulonglong2 q = reinterpret_cast<const ulonglong2*>(p)[j];
    v[2 * j] = q.x;
    v[2 * j + 1] = q.y;
  }
}

__device__ __forceinline__ float ln_warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of N values over the TPR threads of a row; every thread gets them.
// With TPR > 32 red holds N x (TPR / 32) floats for each group of TPR threads
// of the block, and the group's warps meet at a barrier of their own.
template <int TPR, int N>
__device__ __forceinline__ void ln_row_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = ln_warp_sum(v[j]);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int group = threadIdx.x / TPR, warp = (threadIdx.x % TPR) >> 5, lane = threadIdx.x & 31;
    red += group * N * W;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");   // the previous sum has been read
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < N; ++j) red[j * W + warp] = v[j];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
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

// A vector of float parameters per column, in the columns that a thread's
// vectors cover, shared by the groups of a block whose o is the same (they are
// V apart): [class][NV * V / 4][thread of the row] float4.
template <int V, int NV, int TPR, int GROUPS>
struct LnTable {
  static constexpr int kClasses = GROUPS < V ? GROUPS : V;
  static constexpr size_t kBytes = sizeof(float) * kClasses * TPR * NV * V;
  // Filled by the first groups of the block; the block meets before it is read.
  static __device__ __forceinline__ void fill(float* table, const float* src, int dim, int o) {
    const int g = threadIdx.x / TPR, t = threadIdx.x % TPR;
    if (g < kClasses) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (t + i * TPR) * V - o + j;
          table[((g * (NV * V / 4) + (i * V + j) / 4) * TPR + t) * 4 + j % 4] = c >= 0 && c < dim ? __ldg(src + c) : 0.f;
        }
    }
  }
  static __device__ __forceinline__ void load(const float* table, int i, f2 (&v)[V / 2]) {
    const int g = threadIdx.x / TPR % kClasses, t = threadIdx.x % TPR;
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const ulonglong2 q =
          *reinterpret_cast<const ulonglong2*>(table + ((g * (NV * V / 4) + (i * V + j) / 4) * TPR + t) * 4);
      v[j / 2] = q.x;
      v[j / 2 + 1] = q.y;
    }
  }
};

// Stores values lo .. hi - 1 of a vector.
template <typename T, int V>
__device__ __forceinline__ void ln_store_part(T* p, int lo, int hi, const LnVec<T, V>& v) {
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (j >= lo && j < hi) {
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<uint32_t*>(p)[j] = v.w[j];
      } else {
        reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(v.w[j / 2] >> (16 * (j & 1)));
      }
    }
}

inline bool ln_aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
inline size_t ln_size(int dtype) { return dtype == DTYPE_F32 ? 4 : 2; }

}  // namespace jepa
