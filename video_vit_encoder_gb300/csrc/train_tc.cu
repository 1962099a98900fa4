// The training operators on the tensor cores: which products they launch, in
// which pieces, and the small kernels between them.
#include "gemm_train.cuh"
#include "train_tc.h"

namespace jepa {

namespace tg {
cudaError_t gemm_bf16(bool amn, bool bmn, int epi, const Params& p, int num_sms, cudaStream_t s);
cudaError_t gemm_f16(bool amn, bool bmn, int epi, const Params& p, int num_sms, cudaStream_t s);
}  // namespace tg

namespace {

using tg::Params;

constexpr int kBlock = 256;
constexpr int kPairs = 76;   // CTA pairs of 152 SMs: the plans (and workspaces) assume it, the launch asks the device

#define JEPA_TRY_CUDA(expr)                 \
  do {                                      \
    const cudaError_t e_ = (expr);          \
    if (e_ != cudaSuccess) return e_;       \
  } while (0)

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }
int ceil_div(long a, long b) { return (int)((a + b - 1) / b); }
unsigned blocks_for(long n, int block) { return (unsigned)((n + block - 1) / block); }

// ----------------------------------------------------------------------------- operands and plans
// [rows, k] with k contiguous: boxes of 64 k x 128 rows.
cudaError_t map_k(CUtensorMap* m, const void* p, long rows, long k, long ld) {
  return make_tmap_2d(m, p, 2, k, rows, ld * 2, tg::kBK, tg::kBM);
}
// [k, rows] with rows contiguous: boxes of 64 rows x 64 k.
cudaError_t map_mn(CUtensorMap* m, const void* p, long rows, long k, long ld) {
  return make_tmap_2d(m, p, 2, rows, k, ld * 2, 64, tg::kBK);
}
// 16-bit output [rows, cols]; fp32 slabs.
cudaError_t map_out(CUtensorMap* m, void* p, long rows, long cols, long ld) {
  return make_tmap_2d(m, p, 2, cols, rows, ld * 2, 64, 32);
}
cudaError_t map_slab(CUtensorMap* m, void* p, long rows, long cols) {
  return make_tmap_2d(m, p, 4, cols, rows, cols * 4, 32, 32);
}

Params base_params(int M, int N, int cols_per_tile, int* status) {
  Params p{};
  p.M = M;
  p.N = N;
  p.num_m = ceil_div(M, 2 * tg::kBM);
  p.num_n = ceil_div(N, cols_per_tile);
  p.run = p.nseg = p.nz = p.splits = 1;
  p.status = status;
  return p;
}
void set_k(Params& p, long k_per_seg, int nseg, int splits) {
  p.kb_seg = ceil_div(k_per_seg, tg::kBK);
  p.nseg = nseg;
  const int total = p.kb_seg * nseg;
  p.kb_split = ceil_div(total, splits);
  p.splits = ceil_div(total, p.kb_split);
}

// K splits of a product of nz outputs M x N over kb blocks, from the time of
// the schedule: rounds of the 76 pairs, each a unit's blocks (0.27 us a block)
// plus about 6 blocks' time to fill and drain, and, when split, writing the
// fp32 slabs and adding them (5 TB/s, and a launch of about 8 blocks' time).
int plan_splits(long M, long N, int nz, int kb) {
  const long tiles = (long)ceil_div(M, 256) * ceil_div(N, 256) * nz;
  int best = 1;
  double best_t = 1e300;
  for (int s = 1; s <= 16 && (s == 1 || kb / s >= 4); ++s) {
    const int per = ceil_div(kb, s);
    const int real = ceil_div(kb, per);
    double t = (double)ceil_div(tiles * real, kPairs) * (per + 6);
    if (real > 1) t += 8.0 + 2.0 * real * nz * (double)M * N * 4.0 / 5e6 / 0.27;
    if (t < best_t) {
      best_t = t;
      best = real;
    }
  }
  return best;
}
size_t slab_bytes(int splits, long M, long N) { return align256((size_t)splits * ceil_div(M, 256) * 256 * N * 4); }

cudaError_t gemm(int dtype, bool amn, bool bmn, int epi, const Params& p, int num_sms, cudaStream_t s) {
  return dtype == DTYPE_BF16 ? tg::gemm_bf16(amn, bmn, epi, p, num_sms, s) : tg::gemm_f16(amn, bmn, epi, p, num_sms, s);
}

// ----------------------------------------------------------------------------- small kernels
// out[i] = scale * sum over the slabs, in slab order; 8 values a thread.
template <typename T>
__global__ void __launch_bounds__(kBlock) slab_sum_kernel(const float* __restrict__ slab, long stride, int n_slabs,
                                                          T* __restrict__ out, long n8,
                                                          const float* __restrict__ scale) {
  const long i = (long)blockIdx.x * kBlock + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  const float4* a = reinterpret_cast<const float4*>(slab) + 2 * i;
  float4 x = __ldg(a), y = __ldg(a + 1);
  v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  for (int k = 1; k < n_slabs; ++k) {
    a += stride / 4;
    x = __ldg(a);
    y = __ldg(a + 1);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w; v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
  const float sc = scale != nullptr ? __ldg(scale) : 1.f;
  reinterpret_cast<uint4*>(out)[i] = make_uint4(pack2<T>(v[0] * sc, v[1] * sc), pack2<T>(v[2] * sc, v[3] * sc),
                                                pack2<T>(v[4] * sc, v[5] * sc), pack2<T>(v[6] * sc, v[7] * sc));
}
cudaError_t slab_sum(int dtype, const float* slab, long rows_padded, int n_slabs, void* out, long M, long N,
                     const float* scale, cudaStream_t s) {
  const long n8 = M * N / 8;
  const unsigned b = blocks_for(n8, kBlock);
  if (dtype == DTYPE_BF16)
    slab_sum_kernel<__nv_bfloat16><<<b, kBlock, 0, s>>>(slab, rows_padded * N, n_slabs, (__nv_bfloat16*)out, n8, scale);
  else
    slab_sum_kernel<__half><<<b, kBlock, 0, s>>>(slab, rows_padded * N, n_slabs, (__half*)out, n8, scale);
  return cudaGetLastError();
}

// out[c] = sum over r of a[r, c]: 32 columns a block, 8 threads a column, each
// over every eighth row, joined in a fixed order.
__global__ void __launch_bounds__(kBlock) part_sum_kernel(const float* __restrict__ a, long ld, int rows, int n,
                                                          float* __restrict__ out) {
  __shared__ float sm[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < n) {
#pragma unroll 4
    for (int r = g; r < rows; r += 8) s += a[(long)r * ld + c];
  }
  sm[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < n) {
    for (int k = 1; k < 8; ++k) s += sm[k][lane];
    out[c] = s;
  }
}
cudaError_t part_sum(const float* a, long ld, int rows, int n, float* out, cudaStream_t s) {
  part_sum_kernel<<<blocks_for(n, 32), kBlock, 0, s>>>(a, ld, rows, n, out);
  return cudaGetLastError();
}

// Column sums of a 16-bit [M, N] matrix with rows of 16 bytes: block (256
// columns, strip of rows), 8 columns a thread, 8 rows at a time.
template <typename T>
__global__ void __launch_bounds__(kBlock) col_strip_kernel(const T* __restrict__ a, int M, int N, int rows_per,
                                                           float* __restrict__ part) {
  __shared__ float sm[8][256 + 8];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + lane * 8;
  const int r0 = blockIdx.y * rows_per, r1 = min(M, r0 + rows_per);
  float v[8] = {};
  if (c < N) {
#pragma unroll 4
    for (int r = r0 + g; r < r1; r += 8) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(a + (size_t)r * N + c));
      T h[8];
      memcpy(h, &q, 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += DT<T>::to(h[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sm[g][lane * 8 + i] = v[i];
  __syncthreads();
  const int cc = blockIdx.x * 256 + threadIdx.x;
  if (cc < N) {
    float s = 0.f;
    for (int k = 0; k < 8; ++k) s += sm[k][threadIdx.x];
    part[(size_t)blockIdx.y * N + cc] = s;
  }
}
int col_strips(int M, int N) {
  const int want = ceil_div(4 * 152, ceil_div(N, 256)), most = ceil_div(M, 64);
  return want < most ? want : most;
}

// Joins the (max, sum of 2^(z - max)) of a row's parts; 32 rows a block, the
// block's 8 warps take every eighth part.
struct Ms {
  float m, s, sum;
};
__device__ __forceinline__ void ms_join(Ms& a, float m, float s, float sum) {
  const float mm = fmaxf(a.m, m);
  const float ref = mm == -INFINITY ? 0.f : mm;   // a side that has seen only -inf has 2^-inf = 0
  a.s = a.s * tg::ex2(a.m - ref) + s * tg::ex2(m - ref);
  a.m = mm;
  a.sum += sum;
}
__global__ void __launch_bounds__(kBlock) ce_join_kernel(const float2* __restrict__ ms, const float* __restrict__ sums,
                                                         const float* __restrict__ zy, int parts, int M, int V,
                                                         const int64_t* __restrict__ labels, long ignore_index,
                                                         float smoothing, float* __restrict__ loss,
                                                         float* __restrict__ lse_out, int* status) {
  __shared__ Ms sm[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  Ms a{-INFINITY, 0.f, 0.f};
  if (row < M) {
#pragma unroll 4
    for (int k = g; k < parts; k += 8) {
      const float2 q = __ldg(ms + (size_t)k * M + row);
      ms_join(a, q.x, q.y, sums != nullptr ? __ldg(sums + (size_t)k * M + row) : 0.f);
    }
  }
  sm[g][lane] = a;
  __syncthreads();
  if (g != 0 || row >= M) return;
  for (int k = 1; k < 8; ++k) ms_join(a, sm[k][lane].m, sm[k][lane].s, sm[k][lane].sum);
  // lse = ln(2^m s)
  const float lse = (a.m + log2f(a.s)) * 0.69314718055994531f;
  const long label = labels[row];
  float l;
  if (label == ignore_index) {
    l = 0.f;
  } else if (label < 0 || label >= V) {
    l = NAN;
    atomicOr(status, DEV_BAD_INDEX);
  } else {
    l = lse - (1.0f - smoothing) * zy[row];
    if (smoothing > 0.f) l -= smoothing * (a.sum / (float)V);
  }
  if (loss != nullptr) loss[row] = l;
  lse_out[row] = lse;
}

// scale[0] = 2^k with max |dloss| 2^k in (2^13, 2^14], scale[1] = 2^-k, so that
// |dz| 2^k stays below fp16's largest value and small probabilities stay
// normal numbers; 1 when the max is 0 or not finite.
__global__ void __launch_bounds__(1024) dz_scale_kernel(const float* __restrict__ dloss, int M, float* scale) {
  __shared__ float sm[32];
  float m = 0.f;
  for (int i = threadIdx.x; i < M; i += 1024) {
    const float a = fabsf(dloss[i]);
    m = a > m ? a : m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < 32; ++k) m = fmaxf(m, sm[k]);
    int k = 0;
    if (m > 0.f && m < INFINITY) {
      int e;
      frexpf(m, &e);           // m = f 2^e, f in [1/2, 1)
      k = 14 - e;
      k = k > 100 ? 100 : (k < -100 ? -100 : k);
    }
    scale[0] = ldexpf(1.f, k);
    scale[1] = ldexpf(1.f, -k);
  }
}

bool tc_matrix(const void* p, long width) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && width % 8 == 0; }

// A workspace cut into 256-byte aligned buffers.
struct Carver {
  uint8_t* p;
  size_t used = 0;
  template <typename U>
  U* take(size_t bytes) {
    U* r = reinterpret_cast<U*>(p + used);
    used += align256(bytes);
    return r;
  }
};

}  // namespace

// ----------------------------------------------------------------------------- softmax cross entropy
namespace {

// Column tiles per unit of the forward pass: at least 8 units a pair, at most 16 tiles.
int ce_run(int M, int V) {
  const long tiles = (long)ceil_div(M, 256) * ceil_div(V, 256);
  const long r = tiles / (kPairs * 8);
  return (int)(r < 1 ? 1 : (r > 16 ? 16 : r));
}
int ce_parts(int M, int V) { return 2 * ceil_div(ceil_div(V, 256), ce_run(M, V)); }

// The backward pass goes over the vocabulary in pieces whose dz takes at most
// 256 MB, all of the same width up to rounding to 256.
struct CePlan {
  int piece, pieces, dx_splits, dw_splits;
};
CePlan ce_plan(int M, int D, int V) {
  CePlan c;
  long most = ((long)256 << 20) / (2 * (long)M) / 256 * 256;
  if (most < 4096) most = 4096;
  c.pieces = ceil_div(V, most);
  c.piece = ceil_div(ceil_div(V, c.pieces), 256) * 256;
  c.pieces = ceil_div(V, c.piece);
  c.dx_splits = plan_splits(M, D, 1, ceil_div(V < c.piece ? V : c.piece, tg::kBK));
  c.dw_splits = plan_splits(V < c.piece ? V : c.piece, D, 1, ceil_div(M, tg::kBK));
  return c;
}
bool ce_dx_direct(const CePlan& c) { return c.pieces == 1 && c.dx_splits == 1; }

}  // namespace

bool linear_ce_tc_ok(const CeArgs& a, const void* dx, const void* dw) {
  return a.dtype != DTYPE_F32 && tc_matrix(a.x, a.D) && tc_matrix(a.w, a.D) && tc_matrix(dx, a.D) && tc_matrix(dw, a.D);
}

size_t linear_ce_tc_workspace(int M, int D, int V, bool backward) {
  if (M == 0) return 0;
  if (!backward) {
    const size_t n = (size_t)ce_parts(M, V) * M;
    return align256(n * 8) + align256(n * 4) + align256((size_t)M * 4);
  }
  const CePlan c = ce_plan(M, D, V);
  size_t b = 256 + align256((size_t)M * c.piece * 2) + align256((size_t)ceil_div(M, 32) * c.piece * 4);
  if (!ce_dx_direct(c)) b += slab_bytes(c.dx_splits, M, D);
  if (c.dw_splits > 1) b += slab_bytes(c.dw_splits, c.piece, D);
  return b;
}

cudaError_t linear_ce_fwd_tc(const CeArgs& a, float* loss, float* lse, void* ws, cudaStream_t s) {
  const int parts = ce_parts(a.M, a.V);
  const size_t n = (size_t)parts * a.M;
  Carver cv{static_cast<uint8_t*>(ws)};
  Params p = base_params(a.M, a.V, tg::kBN, a.status);
  p.run = ce_run(a.M, a.V);
  set_k(p, a.D, 1, 1);
  JEPA_TRY_CUDA(map_k(&p.a[0], a.x, a.M, a.D, a.D));
  JEPA_TRY_CUDA(map_k(&p.b[0], a.w, a.V, a.D, a.D));
  p.ep.bias = a.bias;
  p.ep.labels = a.labels;
  p.ep.V = a.V;
  p.ep.part_ms = cv.take<float2>(n * 8);
  float* sums = cv.take<float>(n * 4);
  p.ep.part_sum = a.smoothing > 0.f ? sums : nullptr;
  p.ep.zy = cv.take<float>((size_t)a.M * 4);
  JEPA_TRY_CUDA(gemm(a.dtype, false, false, tg::CE_FWD, p, a.num_sms, s));
  ce_join_kernel<<<blocks_for(a.M, 32), kBlock, 0, s>>>(p.ep.part_ms, p.ep.part_sum, p.ep.zy, parts, a.M, a.V, a.labels,
                                                        a.ignore_index, a.smoothing, loss, lse, a.status);
  return cudaGetLastError();
}

cudaError_t linear_ce_bwd_tc(const CeArgs& a, const float* lse, const float* dloss, void* dx, void* dw, float* dbias,
                             void* ws, cudaStream_t s) {
  const CePlan c = ce_plan(a.M, a.D, a.V);
  Carver cv{static_cast<uint8_t*>(ws)};
  float* scale = cv.take<float>(8);
  uint8_t* dz = cv.take<uint8_t>((size_t)a.M * c.piece * 2);
  float* colp = cv.take<float>((size_t)ceil_div(a.M, 32) * c.piece * 4);
  float* dxs = ce_dx_direct(c) ? nullptr : cv.take<float>(slab_bytes(c.dx_splits, a.M, a.D));
  float* dws = c.dw_splits > 1 ? cv.take<float>(slab_bytes(c.dw_splits, c.piece, a.D)) : nullptr;
  const float* unscale = nullptr;
  if (a.dtype == DTYPE_F16) {
    dz_scale_kernel<<<1, 1024, 0, s>>>(dloss, a.M, scale);
    JEPA_TRY_CUDA(cudaGetLastError());
    unscale = scale + 1;
  }
  const long mp = (long)ceil_div(a.M, 256) * 256;
  int dx_slabs = 1;
  for (int v0 = 0; v0 < a.V; v0 += c.piece) {
    const int n = a.V - v0 < c.piece ? a.V - v0 : c.piece;
    const uint8_t* w = static_cast<const uint8_t*>(a.w) + 2 * (size_t)v0 * a.D;
    {
      Params p = base_params(a.M, n, tg::kBN, a.status);
      set_k(p, a.D, 1, 1);
      JEPA_TRY_CUDA(map_k(&p.a[0], a.x, a.M, a.D, a.D));
      JEPA_TRY_CUDA(map_k(&p.b[0], w, n, a.D, a.D));
      JEPA_TRY_CUDA(map_out(&p.c[0], dz, a.M, c.piece, c.piece));
      p.ep.bias = a.bias != nullptr ? a.bias + v0 : nullptr;
      p.ep.labels = a.labels;
      p.ep.ignore_index = a.ignore_index;
      p.ep.lse = lse;
      p.ep.dloss = dloss;
      p.ep.dz_scale = unscale != nullptr ? scale : nullptr;
      p.ep.smoothing = a.smoothing;
      p.ep.v0 = v0;
      p.ep.V = a.V;
      p.ep.col_part = dbias != nullptr ? colp : nullptr;
      p.ep.ld_col = c.piece;
      JEPA_TRY_CUDA(gemm(a.dtype, false, false, tg::CE_BWD, p, a.num_sms, s));
    }
    if (dbias != nullptr) JEPA_TRY_CUDA(part_sum(colp, c.piece, ceil_div(a.M, 32), n, dbias + v0, s));
    if (dx != nullptr) {
      Params p = base_params(a.M, a.D, tg::kBN, a.status);
      set_k(p, n, 1, c.dx_splits);
      JEPA_TRY_CUDA(map_k(&p.a[0], dz, a.M, n, c.piece));
      JEPA_TRY_CUDA(map_mn(&p.b[0], w, a.D, n, a.D));
      if (dxs == nullptr) {
        JEPA_TRY_CUDA(map_out(&p.c[0], dx, a.M, a.D, a.D));
        p.ep.scale = unscale;
        JEPA_TRY_CUDA(gemm(a.dtype, false, true, tg::STORE, p, a.num_sms, s));
      } else {
        // the first piece has the most splits: a narrower last piece adds into the first slabs
        if (v0 == 0) dx_slabs = p.splits;
        JEPA_TRY_CUDA(map_slab(&p.c[0], dxs, mp * c.dx_splits, a.D));
        p.slab_rows = (int)mp;
        JEPA_TRY_CUDA(gemm(a.dtype, false, true, v0 == 0 ? tg::F32 : tg::F32_ADD, p, a.num_sms, s));
      }
    }
    if (dw != nullptr) {
      uint8_t* out = static_cast<uint8_t*>(dw) + 2 * (size_t)v0 * a.D;
      Params p = base_params(n, a.D, tg::kBN, a.status);
      set_k(p, a.M, 1, c.dw_splits);
      JEPA_TRY_CUDA(map_mn(&p.a[0], dz, n, a.M, c.piece));
      JEPA_TRY_CUDA(map_mn(&p.b[0], a.x, a.D, a.M, a.D));
      if (dws == nullptr) {
        JEPA_TRY_CUDA(map_out(&p.c[0], out, n, a.D, a.D));
        p.ep.scale = unscale;
        JEPA_TRY_CUDA(gemm(a.dtype, true, true, tg::STORE, p, a.num_sms, s));
      } else {
        const long np = (long)ceil_div(n, 256) * 256;
        JEPA_TRY_CUDA(map_slab(&p.c[0], dws, np * p.splits, a.D));
        p.slab_rows = (int)np;
        JEPA_TRY_CUDA(gemm(a.dtype, true, true, tg::F32, p, a.num_sms, s));
        JEPA_TRY_CUDA(slab_sum(a.dtype, dws, np, p.splits, out, n, a.D, unscale, s));
      }
    }
  }
  if (dx != nullptr && dxs != nullptr) JEPA_TRY_CUDA(slab_sum(a.dtype, dxs, mp, dx_slabs, dx, a.M, a.D, unscale, s));
  return cudaSuccess;
}

// ----------------------------------------------------------------------------- gated feed-forward
bool gated_ffn_tc_ok(const FfnArgs& a, const void* h, const void* dx, const void* dwg, const void* dwu) {
  return a.dtype != DTYPE_F32 && tc_matrix(a.x, a.D) && tc_matrix(a.wg, a.D) && tc_matrix(a.wu, a.D) &&
         tc_matrix(h, a.F) && tc_matrix(dx, a.D) && tc_matrix(dwg, a.D) && tc_matrix(dwu, a.D);
}

namespace {

struct FfnPlan {
  int fp;   // row length of dg and du
  int dx_splits, dw_splits;
};
FfnPlan ffn_plan(int M, int D, int F) {
  FfnPlan f;
  f.fp = ceil_div(F, 64) * 64;
  f.dx_splits = plan_splits(M, D, 1, 2 * ceil_div(F, tg::kBK));
  f.dw_splits = plan_splits(F, D, 2, ceil_div(M, tg::kBK));
  return f;
}
cudaError_t ffn_params(const FfnArgs& a, Params& p) {
  p = base_params(a.M, a.F, tg::kBN / 2, a.status);
  set_k(p, a.D, 1, 1);
  JEPA_TRY_CUDA(map_k(&p.a[0], a.x, a.M, a.D, a.D));
  JEPA_TRY_CUDA(map_k(&p.b[0], a.wg, a.F, a.D, a.D));
  JEPA_TRY_CUDA(map_k(&p.b[1], a.wu, a.F, a.D, a.D));
  p.ep.bias = a.bg;
  p.ep.bias2 = a.bu;
  p.ep.act = a.act;
  return cudaSuccess;
}

}  // namespace

size_t gated_ffn_tc_workspace(int M, int D, int F, bool backward) {
  if (M == 0 || !backward) return 0;
  const FfnPlan f = ffn_plan(M, D, F);
  size_t b = 2 * align256((size_t)M * f.fp * 2) + 2 * align256((size_t)ceil_div(M, 32) * f.fp * 4);
  if (f.dx_splits > 1) b += slab_bytes(f.dx_splits, M, D);
  if (f.dw_splits > 1) b += 2 * slab_bytes(f.dw_splits, F, D);
  return b;
}

cudaError_t gated_ffn_fwd_tc(const FfnArgs& a, void* h, cudaStream_t s) {
  Params p;
  JEPA_TRY_CUDA(ffn_params(a, p));
  JEPA_TRY_CUDA(map_out(&p.c[0], h, a.M, a.F, a.F));
  return gemm(a.dtype, false, false, tg::GATE_FWD, p, a.num_sms, s);
}

cudaError_t gated_ffn_bwd_tc(const FfnArgs& a, const void* dh, void* dx, void* dwg, void* dwu, float* dbg, float* dbu,
                             void* ws, cudaStream_t s) {
  const FfnPlan f = ffn_plan(a.M, a.D, a.F);
  Carver cv{static_cast<uint8_t*>(ws)};
  uint8_t* d[2];
  float* colp[2];
  for (int k = 0; k < 2; ++k) d[k] = cv.take<uint8_t>((size_t)a.M * f.fp * 2);
  for (int k = 0; k < 2; ++k) colp[k] = cv.take<float>((size_t)ceil_div(a.M, 32) * f.fp * 4);
  float* dxs = f.dx_splits > 1 ? cv.take<float>(slab_bytes(f.dx_splits, a.M, a.D)) : nullptr;
  float* dws[2] = {nullptr, nullptr};
  if (f.dw_splits > 1)
    for (int k = 0; k < 2; ++k) dws[k] = cv.take<float>(slab_bytes(f.dw_splits, a.F, a.D));
  {
    Params p;
    JEPA_TRY_CUDA(ffn_params(a, p));
    for (int k = 0; k < 2; ++k) JEPA_TRY_CUDA(map_out(&p.c[k], d[k], a.M, f.fp, f.fp));
    p.ep.dh = dh;
    p.ep.col_part = dbg != nullptr ? colp[0] : nullptr;
    p.ep.col_part2 = dbu != nullptr ? colp[1] : nullptr;
    p.ep.ld_col = f.fp;
    JEPA_TRY_CUDA(gemm(a.dtype, false, false, tg::GATE_BWD, p, a.num_sms, s));
  }
  if (dbg != nullptr) JEPA_TRY_CUDA(part_sum(colp[0], f.fp, ceil_div(a.M, 32), a.F, dbg, s));
  if (dbu != nullptr) JEPA_TRY_CUDA(part_sum(colp[1], f.fp, ceil_div(a.M, 32), a.F, dbu, s));
  if (dx != nullptr) {
    Params p = base_params(a.M, a.D, tg::kBN, a.status);
    set_k(p, a.F, 2, f.dx_splits);
    for (int k = 0; k < 2; ++k) {
      JEPA_TRY_CUDA(map_k(&p.a[k], d[k], a.M, a.F, f.fp));
      JEPA_TRY_CUDA(map_mn(&p.b[k], k == 0 ? a.wg : a.wu, a.D, a.F, a.D));
    }
    if (dxs == nullptr) {
      JEPA_TRY_CUDA(map_out(&p.c[0], dx, a.M, a.D, a.D));
      JEPA_TRY_CUDA(gemm(a.dtype, false, true, tg::STORE, p, a.num_sms, s));
    } else {
      const long mp = (long)ceil_div(a.M, 256) * 256;
      JEPA_TRY_CUDA(map_slab(&p.c[0], dxs, mp * p.splits, a.D));
      p.slab_rows = (int)mp;
      JEPA_TRY_CUDA(gemm(a.dtype, false, true, tg::F32, p, a.num_sms, s));
      JEPA_TRY_CUDA(slab_sum(a.dtype, dxs, mp, p.splits, dx, a.M, a.D, nullptr, s));
    }
  }
  void* dw[2] = {dwg, dwu};
  if (dwg == nullptr && dwu == nullptr) return cudaSuccess;
  // both weight gradients are one launch; asked for alone, each is its own
  Params p = base_params(a.F, a.D, tg::kBN, a.status);
  set_k(p, a.M, 1, f.dw_splits);
  JEPA_TRY_CUDA(map_mn(&p.b[0], a.x, a.D, a.M, a.D));
  const long np = (long)ceil_div(a.F, 256) * 256;
  int nz = 0;
  for (int k = 0; k < 2; ++k) {
    if (dw[k] == nullptr) continue;
    JEPA_TRY_CUDA(map_mn(&p.a[nz], d[k], a.F, a.M, f.fp));
    if (dws[0] == nullptr) JEPA_TRY_CUDA(map_out(&p.c[nz], dw[k], a.F, a.D, a.D));
    else JEPA_TRY_CUDA(map_slab(&p.c[nz], dws[k], np * p.splits, a.D));
    ++nz;
  }
  p.nz = nz;
  p.slab_rows = (int)np;
  JEPA_TRY_CUDA(gemm(a.dtype, true, true, dws[0] == nullptr ? tg::STORE : tg::F32, p, a.num_sms, s));
  if (dws[0] != nullptr)
    for (int k = 0; k < 2; ++k)
      if (dw[k] != nullptr) JEPA_TRY_CUDA(slab_sum(a.dtype, dws[k], np, p.splits, dw[k], a.F, a.D, nullptr, s));
  return cudaSuccess;
}

// ----------------------------------------------------------------------------- linear layer backward
bool linear_bwd_tc_ok(int dtype, const void* dout, const void* A, const void* W, const void* dA, const void* dW, int N,
                      int K) {
  return dtype != DTYPE_F32 && tc_matrix(dout, N) && tc_matrix(A, K) && tc_matrix(W, K) && tc_matrix(dA, K) &&
         tc_matrix(dW, K);
}
size_t linear_bwd_tc_workspace(int M, int N, int K) {
  if (M == 0) return 0;
  const int sa = plan_splits(M, K, 1, ceil_div(N, tg::kBK)), sw = plan_splits(N, K, 1, ceil_div(M, tg::kBK));
  const size_t a = sa > 1 ? slab_bytes(sa, M, K) : 0, w = sw > 1 ? slab_bytes(sw, N, K) : 0;
  return (a > w ? a : w) + align256((size_t)col_strips(M, N) * N * 4);
}
cudaError_t linear_bwd_tc(int dtype, const void* dout, const void* A, const void* W, void* dA, void* dW, float* dbias,
                          int M, int N, int K, void* ws, int* status, int num_sms, cudaStream_t s) {
  const int sa = plan_splits(M, K, 1, ceil_div(N, tg::kBK)), sw = plan_splits(N, K, 1, ceil_div(M, tg::kBK));
  Carver cv{static_cast<uint8_t*>(ws)};
  float* colp = cv.take<float>((size_t)col_strips(M, N) * N * 4);
  float* slab = cv.take<float>(0);
  for (int k = 0; k < 2; ++k) {
    // dA = dout W, then dW = dout^T A; the slabs of one are free when the other starts
    void* out = k == 0 ? dA : dW;
    if (out == nullptr) continue;
    const int rows = k == 0 ? M : N, red = k == 0 ? N : M, splits = k == 0 ? sa : sw;
    Params p = base_params(rows, K, tg::kBN, status);
    set_k(p, red, 1, splits);
    JEPA_TRY_CUDA(k == 0 ? map_k(&p.a[0], dout, M, N, N) : map_mn(&p.a[0], dout, N, M, N));
    JEPA_TRY_CUDA(map_mn(&p.b[0], k == 0 ? W : A, K, red, K));
    if (splits == 1) {
      JEPA_TRY_CUDA(map_out(&p.c[0], out, rows, K, K));
      JEPA_TRY_CUDA(gemm(dtype, k != 0, true, tg::STORE, p, num_sms, s));
    } else {
      const long rp = (long)ceil_div(rows, 256) * 256;
      JEPA_TRY_CUDA(map_slab(&p.c[0], slab, rp * p.splits, K));
      p.slab_rows = (int)rp;
      JEPA_TRY_CUDA(gemm(dtype, k != 0, true, tg::F32, p, num_sms, s));
      JEPA_TRY_CUDA(slab_sum(dtype, slab, rp, p.splits, out, rows, K, nullptr, s));
    }
  }
  if (dbias != nullptr) {
    const int strips = col_strips(M, N), per = ceil_div(M, strips);
    const dim3 g(ceil_div(N, 256), strips);
    if (dtype == DTYPE_BF16)
      col_strip_kernel<__nv_bfloat16><<<g, kBlock, 0, s>>>((const __nv_bfloat16*)dout, M, N, per, colp);
    else
      col_strip_kernel<__half><<<g, kBlock, 0, s>>>((const __half*)dout, M, N, per, colp);
    JEPA_TRY_CUDA(cudaGetLastError());
    JEPA_TRY_CUDA(part_sum(colp, N, strips, N, dbias, s));
  }
  return cudaSuccess;
}

}  // namespace jepa
