// The forward passes of the gated feed-forward and of the cross entropy for a
// few rows of x (single tokens, one pooled row per clip).
//
// With M <= 16 rows the weights are all the traffic and a 256-row tile is
// mostly padding: bound by HBM where the weights are large, by latency where
// they are not.  A block of eight warps computes 16 weight rows (of each
// matrix) against all of x; the warps take every eighth piece of K, so that a
// block has its whole share of the weights in flight at once, and add their
// sums through shared memory in warp order.
//
// 16-bit: products m16n8k16 with the weights as the 16 rows and x as the 8
// columns, fp32 sums.  The order of K inside a product is free as long as both
// operands use the same one, so every thread loads 16 contiguous bytes of its
// row, which are two products' worth.  The products truncate their sums like
// tcgen05.mma (gemm_train.cuh), so each 32 of a warp are added up apart.  fp32:
// eight weight rows and all of x per thread in FFMA, each thread four of K at a
// time.
//
// Gated feed-forward, 8 rows, 1024 -> 4096, bf16: 16.8 MB of weights, 5.7 us with
// the weights from HBM, 4.2 from L2 (tiles of 256 rows: 16.5).  Cross entropy, 8
// rows, 1024 -> 174, fp32: 7.0 us with its joining kernel (tiles: 41); 16 rows,
// 1024 -> 131072, bf16: 70 us (17 rows, on tiles: 96).
#include "gemm_train.cuh"

namespace jepa {

namespace {

constexpr int kWarps = 8, kBlock = 32 * kWarps;
constexpr int kRows = 16;   // weight rows of a block
constexpr int kChunk = 4096;   // of K, a warp's share of it 32 steps: then its sums are taken out and added with rounding

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Streaming: the weights are read once.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 q;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

// This warp's share of the sums of weight rows r0 .. r0 + 15 of NM matrices
// against x, into sums[mat][16][8 * NT] (its own part of shared memory).  Rows
// past `rows` and x rows past M repeat the last one; their sums go nowhere.
template <typename T, int NM, int NT>
__device__ __forceinline__ void dot_rows(const T* const (&w)[NM], const T* x, int rows, int M, int D, int r0, int warp,
                                         int lane, float* sums) {
  if constexpr (sizeof(T) == 2) {
    const int g = lane >> 2, q = lane & 3;
    const T* a[NM][2];
#pragma unroll
    for (int k = 0; k < NM; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) a[k][h] = w[k] + (size_t)min(r0 + g + 8 * h, rows - 1) * D;
    const T* b[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) b[n] = x + (size_t)min(n * 8 + g, M - 1) * D;
    float c[NM][NT][4] = {};
#pragma unroll 1
    for (int k1 = warp * 64; k1 < D; k1 += kChunk) {
      const int end = min(D, k1 + kChunk);
      float t[NM][NT][4] = {};
#pragma unroll 2
      for (int k0 = k1; k0 < end; k0 += kWarps * 64) {
        uint4 av[NM][2][2], bv[NT][2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int k = k0 + p * 32 + q * 8;
          const bool in = k < D;   // D is a multiple of 8
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) av[m][h][p] = in ? load_once(a[m][h] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            bv[n][p] = in ? __ldg(reinterpret_cast<const uint4*>(b[n] + k)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16816<T>(t[m][n], av[m][0][p].x, av[m][1][p].x, av[m][0][p].y, av[m][1][p].y, bv[n][p].x, bv[n][p].y);
              mma16816<T>(t[m][n], av[m][0][p].z, av[m][1][p].z, av[m][0][p].w, av[m][1][p].w, bv[n][p].z, bv[n][p].w);
            }
      }
#pragma unroll
      for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[m][n][i] += t[m][n][i];
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float2*>(sums + (m * kRows + g + 8 * h) * (8 * NT) + n * 8 + 2 * q) =
              make_float2(c[m][n][2 * h], c[m][n][2 * h + 1]);
  } else {
    // eight weight rows against eight rows of x at a time; the weights' second time comes from L2
#pragma unroll 1
    for (int part = 0; part < 2 * NM * NT; ++part) {
      const int m = part / (2 * NT), h = part & 1, n0 = part / 2 % NT * 8;
      const float* a[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) a[r] = (NM == 1 || m == 0 ? w[0] : w[NM - 1]) + (size_t)min(r0 + 8 * h + r, rows - 1) * D;
      float c[64] = {};   // [weight row][x row]
      for (int k = warp * 128 + lane * 4; k < D; k += kWarps * 128) {   // D is a multiple of 4
        float4 av[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint4 u = load_once(a[r] + k);
          memcpy(&av[r], &u, 16);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float4 b = __ldg(reinterpret_cast<const float4*>(x + (size_t)min(n0 + n, M - 1) * D + k));
#pragma unroll
          for (int r = 0; r < 8; ++r)
            c[r * 8 + n] = fmaf(av[r].x, b.x, fmaf(av[r].y, b.y, fmaf(av[r].z, b.z, fmaf(av[r].w, b.w, c[r * 8 + n]))));
        }
      }
      // lanes to sums: each step halves the values a lane carries; lane l ends with values 2 l and 2 l + 1
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < 2 * o; ++i) {
          const float send = up ? c[i] : c[i + 2 * o];
          const float keep = up ? c[i + 2 * o] : c[i];
          c[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      *reinterpret_cast<float2*>(sums + (m * kRows + 8 * h + lane / 4) * (8 * NT) + n0 + 2 * (lane & 3)) = make_float2(c[0], c[1]);
    }
  }
}

// Sum of one (matrix, weight row, x row) over the warps.
template <int NM, int NT>
__device__ __forceinline__ float join(const float* sums, int m, int r, int n) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) s += sums[((k * NM + m) * kRows + r) * (8 * NT) + n];
  return s;
}

template <typename T, int NT, int ACT>
__global__ void __launch_bounds__(kBlock) few_gate_kernel(const T* __restrict__ x, const T* __restrict__ wg,
                                                          const T* __restrict__ wu, const float* __restrict__ bg,
                                                          const float* __restrict__ bu, T* __restrict__ h, int M, int D,
                                                          int F) {
  __shared__ float sums[kWarps * 2 * kRows * 8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * kRows;
  const T* const w[2] = {wg, wu};
  dot_rows<T, 2, NT>(w, x, F, M, D, r0, warp, lane, sums + warp * 2 * kRows * 8 * NT);
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * 8 * NT; i += kBlock) {
    const int r = i % kRows, n = i / kRows, f = r0 + r;
    if (f < F && n < M) {
      float g = join<2, NT>(sums, 0, r, n), u = join<2, NT>(sums, 1, r, n);
      if (bg != nullptr) g += __ldg(bg + f);
      if (bu != nullptr) u += __ldg(bu + f);
      float a, da;
      tg::gate<ACT, false>(g, a, da);
      h[(size_t)n * F + f] = DT<T>::from(a * u);
    }
  }
}

// Each block walks groups of 16 classes and carries the statistics of every
// row of x: thread n < M those of row n.
template <typename T, int NT>
__global__ void __launch_bounds__(kBlock) few_ce_kernel(const T* __restrict__ x, const T* __restrict__ w,
                                                        const float* __restrict__ bias,
                                                        const int64_t* __restrict__ labels, int M, int D, int V,
                                                        float2* __restrict__ part_ms, float* __restrict__ part_sum,
                                                        float* __restrict__ zy) {
  __shared__ float sums[kWarps * kRows * 8 * NT];
  __shared__ float z[kRows][8 * NT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tg::RowStats st{-INFINITY, 0.f, 0.f};
  const long label = threadIdx.x < M ? labels[threadIdx.x] : -1;
  const T* const ws[1] = {w};
  const int groups = (V + kRows - 1) / kRows;
  for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const int r0 = grp * kRows;
    dot_rows<T, 1, NT>(ws, x, V, M, D, r0, warp, lane, sums + warp * kRows * 8 * NT);
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * 8 * NT; i += kBlock) {
      const int r = i % kRows, n = i / kRows;
      float v = join<1, NT>(sums, 0, r, n);
      if (bias != nullptr && r0 + r < V) v += __ldg(bias + r0 + r);
      z[r][n] = v;
    }
    __syncthreads();
    if (threadIdx.x < M) {
      const int n = threadIdx.x, left = min(kRows, V - r0);
      float m = st.m;
      for (int r = 0; r < left; ++r) m = fmaxf(m, z[r][n] * tg::kLog2e);
      const float ref = m == -INFINITY ? 0.f : m;   // nothing but -inf so far: every power is 0
      float s = st.s * tg::ex2(st.m - ref);
      for (int r = 0; r < left; ++r) {
        s += tg::ex2(fmaf(z[r][n], tg::kLog2e, -ref));
        st.sum += z[r][n];
      }
      st.m = m;
      st.s = s;
      if (label >= r0 && label < r0 + left) zy[n] = z[label - r0][n];
    }
    // z is written again after the next group's first barrier
  }
  if (threadIdx.x < M) {
    const size_t i = (size_t)blockIdx.x * M + threadIdx.x;
    part_ms[i] = make_float2(st.m, st.s);
    if (part_sum != nullptr) part_sum[i] = st.sum;
  }
}

int ce_blocks(int V) {
  const int groups = (V + kRows - 1) / kRows;
  return groups < 4 * 152 ? groups : 4 * 152;
}

template <typename T, int NT>
cudaError_t gate_t(const FfnArgs& a, void* h, cudaStream_t s) {
  const unsigned blocks = (unsigned)((a.F + kRows - 1) / kRows);
  if (a.act == ACT_SILU)
    few_gate_kernel<T, NT, ACT_SILU><<<blocks, kBlock, 0, s>>>((const T*)a.x, (const T*)a.wg, (const T*)a.wu, a.bg, a.bu,
                                                               (T*)h, a.M, a.D, a.F);
  else
    few_gate_kernel<T, NT, ACT_GELU><<<blocks, kBlock, 0, s>>>((const T*)a.x, (const T*)a.wg, (const T*)a.wu, a.bg, a.bu,
                                                               (T*)h, a.M, a.D, a.F);
  return cudaGetLastError();
}
template <typename T, int NT>
cudaError_t ce_t(const CeArgs& a, float2* ms, float* sums, float* zy, cudaStream_t s) {
  few_ce_kernel<T, NT><<<ce_blocks(a.V), kBlock, 0, s>>>((const T*)a.x, (const T*)a.w, a.bias, a.labels, a.M, a.D, a.V, ms,
                                                         sums, zy);
  return cudaGetLastError();
}

}  // namespace

bool few_rows_ok(int dtype, int M, int D) {
  return M <= 16 && D % (dtype == DTYPE_F32 ? 4 : 8) == 0;
}
cudaError_t few_rows_gate(const FfnArgs& a, void* h, cudaStream_t s) {
  if (a.dtype == DTYPE_F32) return a.M <= 8 ? gate_t<float, 1>(a, h, s) : gate_t<float, 2>(a, h, s);
  if (a.dtype == DTYPE_F16) return a.M <= 8 ? gate_t<__half, 1>(a, h, s) : gate_t<__half, 2>(a, h, s);
  return a.M <= 8 ? gate_t<__nv_bfloat16, 1>(a, h, s) : gate_t<__nv_bfloat16, 2>(a, h, s);
}
int few_rows_ce_parts(int V) { return ce_blocks(V); }
cudaError_t few_rows_ce(const CeArgs& a, float2* ms, float* sums, float* zy, cudaStream_t s) {
  if (a.dtype == DTYPE_F32) return a.M <= 8 ? ce_t<float, 1>(a, ms, sums, zy, s) : ce_t<float, 2>(a, ms, sums, zy, s);
  if (a.dtype == DTYPE_F16) return a.M <= 8 ? ce_t<__half, 1>(a, ms, sums, zy, s) : ce_t<__half, 2>(a, ms, sums, zy, s);
  return a.M <= 8 ? ce_t<__nv_bfloat16, 1>(a, ms, sums, zy, s) : ce_t<__nv_bfloat16, 2>(a, ms, sums, zy, s);
}

}  // namespace jepa
