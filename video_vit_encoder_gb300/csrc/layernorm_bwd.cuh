// Layer norm backward.  With xh = (x - mean) rstd and c = dy * w, per row
//   dx = rstd (c - mean_j c - xh mean_j(c xh)) [+ res]
// and over the rows  dw = sum dy * xh,  db = sum dy.
//
// One pass over x, dy (and res): a row stays on the SM between its two row sums
// and dx.  Each block (one per SM) walks rows and keeps its sums of
// dw and db in registers, so they cost no traffic until it ends; a second
// kernel adds the blocks' sums in a fixed order (no atomics, so the result
// does not depend on scheduling).  Bound by HBM.
//
// Rows come through shared memory: each thread copies its own vectors of its
// next rows asynchronously (no other thread reads them, so there is no
// barrier) and reads them twice, once for the row sums and once for dx.  Only
// the dw and db sums stay in registers, which leaves room for 16 warps per SM
// to hide the latency of the row sums.
#pragma once
#include "layernorm_train.cuh"

namespace jepa {

namespace {

constexpr int kMostSmem = 232448;

// The kernel's shape: TPR threads a row, groups of TPR threads up to 16 warps,
// and the rows in flight per thread.  SHIFT takes as many groups as leave two
// rows in flight each (8192 x 7001 in fp32 with a residual 174 us, with 16
// warps 224; 8192 x 4093 in bf16 78 and 84); without its table and masks 16
// warps with fewer rows in flight are faster (16384 x 1536 in fp32 57 us
// against 64, 8192 x 4096 with a 16-bit dy 90 against 99).
template <typename TX, typename TY, int V, int NV, int TPR, bool SHIFT, bool RES>
struct BwdShape {
  static constexpr int kRowVec = NV * V * ((RES ? 2 : 1) * sizeof(TX) + sizeof(TY));   // a thread's columns of x, res, dy
  static constexpr size_t kHead = 32 * sizeof(float);
  static constexpr int kMostGroups = 512 / TPR;
  static constexpr size_t kRowTable = sizeof(float) * TPR * NV * V;   // w as it is, where columns do not shift
  static constexpr size_t kLargestTable = SHIFT ? LnTable<V, NV, TPR, kMostGroups>::kBytes : kRowTable;
  static constexpr int kSlots = (int)((kMostSmem - kHead - kLargestTable) / (TPR * kRowVec));
  static constexpr int kHalf = kSlots / 2 > 0 ? kSlots / 2 : 1;
  static constexpr int kRows = SHIFT && kHalf < kMostGroups ? kHalf : kMostGroups;
  static constexpr int kThreads = kRows * TPR;
  using Table = LnTable<V, NV, TPR, kRows>;
  // w comes from shared memory, or where that does not fit beside a row from global memory
  static constexpr size_t kWanted = SHIFT ? Table::kBytes : kRowTable;
  static constexpr bool kTable = kHead + (size_t)kThreads * kRowVec + kWanted <= kMostSmem;
  static constexpr size_t kTableBytes = kTable ? kWanted : 0;
  static constexpr int kFit = (int)((kMostSmem - kHead - kTableBytes) / (kThreads * kRowVec));
  static constexpr int kDepth = kFit > 4 ? 4 : kFit;
  static_assert(kDepth >= 1, "a row must fit");
  static constexpr size_t kRing = (size_t)kDepth * kThreads * kRowVec;
  static constexpr size_t kSums = 2 * sizeof(float) * kThreads * NV * V;   // at the end: the groups' dw and db
  static constexpr size_t kSmem = kHead + (kRing + kTableBytes > kSums ? kRing + kTableBytes : kSums);
  static_assert(kSmem <= kMostSmem, "shared memory of one block");
};

template <typename TX, typename TY, int V, int NV, int TPR, bool SHIFT, bool RES>
__global__ void __launch_bounds__(BwdShape<TX, TY, V, NV, TPR, SHIFT, RES>::kThreads, 1)
    ln_bwd_kernel(const TY* __restrict__ dy, const TX* __restrict__ x, const float* __restrict__ w,
                  const float* __restrict__ mean, const float* __restrict__ rstd, const TX* __restrict__ res,
                  TX* __restrict__ dx, float* __restrict__ part_w, float* __restrict__ part_b, long rows, int dim) {
  using S = BwdShape<TX, TY, V, NV, TPR, SHIFT, RES>;
  constexpr int kThreads = S::kThreads;
  constexpr int kBX = V * sizeof(TX), kBY = V * sizeof(TY);
  constexpr size_t kOffY = (size_t)(RES ? 2 : 1) * NV * kThreads * kBX;   // of dy in a slot
  extern __shared__ __align__(16) uint8_t smem[];
  float* red = reinterpret_cast<float*>(smem);                       // [32] row sums across warps
  uint8_t* ring = smem + S::kHead;                                   // [depth][x | res | dy][NV][thread]
  float* table = reinterpret_cast<float*>(ring + S::kRing);
  const int tid = threadIdx.x, t = tid % TPR;
  const long first = (long)blockIdx.x * S::kRows + tid / TPR;
  const long stride = (long)gridDim.x * S::kRows;
  const int o = SHIFT ? (int)((first * dim) % V) : 0;
  const int head = SHIFT && t == 0 ? o : 0;   // elements of this thread's vector 0 that are the previous row's
  const float inv = 1.0f / (float)dim;
  if constexpr (S::kTable) {
    if constexpr (SHIFT) S::Table::fill(table, w, dim, o);
    else
      for (int c = tid; c < dim; c += kThreads) table[c] = __ldg(w + c);
    __syncthreads();
  }

  // this thread's vectors of `row` into slot d of the ring; the last vector ends with the row (zeros follow)
  auto fetch = [&](long row, int d) {
    if (row < rows) {
      uint8_t* slot = ring + (size_t)d * kThreads * S::kRowVec;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c0 = (t + i * TPR) * V - o;
        if (c0 < dim) {
          const long at = row * dim + c0;
          const int n = SHIFT ? min(V, dim - c0) : V;
          uint8_t* q = slot + (size_t)(i * kThreads + tid) * kBX;
          ln_copy_async<kBX>(q, x + at, n * (int)sizeof(TX));
          if constexpr (RES) ln_copy_async<kBX>(q + (size_t)NV * kThreads * kBX, res + at, n * (int)sizeof(TX));
          ln_copy_async<kBY>(slot + kOffY + (size_t)(i * kThreads + tid) * kBY, dy + at, n * (int)sizeof(TY));
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
  float mu = 0.f, rs = 0.f;
  if (first < rows) {
    mu = __ldg(mean + first);
    rs = __ldg(rstd + first);
  }
  for (long row = first; row < rows; row += stride) {
    float mu_next = 0.f, rs_next = 0.f;
    if (row + stride < rows) {
      mu_next = __ldg(mean + row + stride);
      rs_next = __ldg(rstd + row + stride);
    }
    ln_copy_wait<S::kDepth - 1>();
    const uint8_t* slot = ring + (size_t)d * kThreads * S::kRowVec;
    // vector i: x - mean in xv, dy in gv and w in ww; the previous row's values and the zeros after the row meet w = 0
    // and dy = 0
    auto load = [&](int i, int c0, float (&xv)[V], float (&gv)[V], float (&ww)[V]) {
      ln_load<TX, V>(reinterpret_cast<const TX*>(slot + (size_t)(i * kThreads + tid) * kBX), xv);
      ln_load<TY, V>(reinterpret_cast<const TY*>(slot + kOffY + (size_t)(i * kThreads + tid) * kBY), gv);
      if (SHIFT && i == 0) {
#pragma unroll
        for (int j = 0; j < V - 1; ++j) {
          xv[j] = j < head ? 0.f : xv[j];
          gv[j] = j < head ? 0.f : gv[j];
        }
      }
#pragma unroll
      for (int j = 0; j < V; j += 2) add2f(xv[j], xv[j + 1], -mu, -mu);
      if constexpr (SHIFT && !S::kTable) {
#pragma unroll
        for (int j = 0; j < V; ++j) ww[j] = c0 + j >= 0 && c0 + j < dim ? __ldg(w + c0 + j) : 0.f;
      } else if constexpr (SHIFT) {
        S::Table::load(table, i, ww);
      } else {
        ln_load<float, V>((S::kTable ? table : w) + c0, ww);
      }
    };
    float sa[2] = {0.f, 0.f}, sb[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (t + i * TPR) * V - o;
      if (c0 < dim) {
        float xv[V], gv[V], ww[V];
        load(i, c0, xv, gv, ww);
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          ln_mul2(xv[j], xv[j + 1], rs, rs);
          ln_fma2(aw[i][j], aw[i][j + 1], gv[j], gv[j + 1], xv[j], xv[j + 1]);
          add2f(ab[i][j], ab[i][j + 1], gv[j], gv[j + 1]);
          ln_mul2(gv[j], gv[j + 1], ww[j], ww[j + 1]);
          add2f(sa[0], sa[1], gv[j], gv[j + 1]);
          ln_fma2(sb[0], sb[1], gv[j], gv[j + 1], xv[j], xv[j + 1]);
        }
      }
    }
    float s[2] = {sa[0] + sa[1], sb[0] + sb[1]};
    ln_row_sum<TPR, 2>(s, red);
    // dx = rs c - rs m0 - (rs m1 rs) (x - mean)
    const float k0 = -rs * (s[0] * inv), k1 = -rs * (s[1] * inv) * rs;
    TX* dr = dx + row * dim;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c0 = (t + i * TPR) * V - o;
      if (c0 < dim) {
        float xv[V], gv[V], ww[V];
        load(i, c0, xv, gv, ww);
        float out[V];
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          ln_mul2(gv[j], gv[j + 1], ww[j], ww[j + 1]);
          out[j] = out[j + 1] = k0;
          ln_fma2(out[j], out[j + 1], xv[j], xv[j + 1], k1, k1);
          ln_fma2(out[j], out[j + 1], gv[j], gv[j + 1], rs, rs);
        }
        if constexpr (RES) {
          float r[V];
          ln_load<TX, V>(reinterpret_cast<const TX*>(slot + (size_t)((NV + i) * kThreads + tid) * kBX), r);
#pragma unroll
          for (int j = 0; j < V; j += 2) add2f(out[j], out[j + 1], r[j], r[j + 1]);
        }
        if constexpr (SHIFT) ln_store_part<TX, V>(dr, c0, dim, out);
        else ln_store<TX, V>(dr + c0, out);
      }
    }
    fetch(row + S::kDepth * stride, d);   // the slot has been read
    if (++d == S::kDepth) d = 0;
    mu = mu_next;
    rs = rs_next;
  }
  ln_copy_wait<0>();

  // the groups' sums side by side in shared memory, then added in their order
  float* pw = part_w + (size_t)blockIdx.x * 2 * dim;
  float* pb = part_b + (size_t)blockIdx.x * 2 * dim;
  __syncthreads();
  float* mine = reinterpret_cast<float*>(ring) + (size_t)(tid / TPR) * 2 * dim;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c0 = (t + i * TPR) * V - o;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (c0 + j >= 0 && c0 + j < dim) {
        mine[c0 + j] = aw[i][j];
        mine[dim + c0 + j] = ab[i][j];
      }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(ring);
  for (int c = tid; c < 2 * dim; c += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < S::kRows; ++k) v += all[(size_t)k * 2 * dim + c];
    if (c < dim) pw[c] = v;
    else pb[c - dim] = v;
  }
}

constexpr int kBlock = 256;

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

using Args = LnBwdArgs;

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

template <typename TX, typename TY, int V, int NV, int TPR, bool SHIFT, bool RES>
cudaError_t launch_rows(const Args& a, cudaStream_t s) {
  using S = BwdShape<TX, TY, V, NV, TPR, SHIFT, RES>;
  auto kern = ln_bwd_kernel<TX, TY, V, NV, TPR, SHIFT, RES>;
  static DeviceOnce setup;
  cudaError_t e = setup.run([&](int) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
  });
  if (e != cudaSuccess) return e;
  // a thread's rows are a multiple of 8 apart (152 blocks), or it has one row
  const int strips = bwd_strips_rows(a.rows, S::kRows, kBlocks);
  float *pw, *pb;
  parts(a, strips, pw, pb);
  kern<<<strips, S::kThreads, S::kSmem, s>>>((const TY*)a.dy, (const TX*)a.x, a.w, a.mean, a.rstd, (const TX*)a.res,
                                          (TX*)a.dx, pw, pb, a.rows, a.dim);
  e = cudaGetLastError();
  return e == cudaSuccess ? join(a, strips, s) : e;
}

// The fewest threads a row whose registers hold 32 columns each of dw and db.
template <typename TX, typename TY, int V, bool SHIFT, bool RES>
cudaError_t launch_width(const Args& a, cudaStream_t s) {
  const int n = a.dim + (SHIFT ? V - 1 : 0);   // columns that the vectors cover
  if (n <= 256) return launch_rows<TX, TY, V, 8 / V, 32, SHIFT, RES>(a, s);
  if (n <= 512) return launch_rows<TX, TY, V, 16 / V, 32, SHIFT, RES>(a, s);
  if (n <= 1024) return launch_rows<TX, TY, V, 32 / V, 32, SHIFT, RES>(a, s);
  if (n <= 2048) return launch_rows<TX, TY, V, 32 / V, 64, SHIFT, RES>(a, s);
  if (n <= 4096) return launch_rows<TX, TY, V, 32 / V, 128, SHIFT, RES>(a, s);
  return launch_rows<TX, TY, V, 32 / V, 256, SHIFT, RES>(a, s);
}

template <typename TX, typename TY>
cudaError_t bwd_t(const Args& a, cudaStream_t s) {
  constexpr int V = sizeof(TX) == 4 ? 4 : 8;
  const bool vec = ln_aligned(a.x, V * sizeof(TX)) && ln_aligned(a.dy, V * sizeof(TY)) &&
                   ln_aligned(a.dx, V * sizeof(TX)) && ln_aligned(a.res, V * sizeof(TX));
  if (vec && a.dim % V == 0 && a.dim <= kLongest && ln_aligned(a.w, 16))
    return a.res != nullptr ? launch_width<TX, TY, V, false, true>(a, s) : launch_width<TX, TY, V, false, false>(a, s);
  if (vec && a.dim + V - 1 <= kLongest)
    return a.res != nullptr ? launch_width<TX, TY, V, true, true>(a, s) : launch_width<TX, TY, V, true, false>(a, s);
  const int strips = bwd_strips_rows(a.rows, 1, 2 * kBlocks);
  float *pw, *pb;
  parts(a, strips, pw, pb);
  ln_bwd_wide_kernel<TX, TY><<<strips, kBlock, 0, s>>>((const TY*)a.dy, (const TX*)a.x, a.w, a.mean, a.rstd,
                                                       (const TX*)a.res, (TX*)a.dx, pw, pb, a.rows, a.dim);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? join(a, strips, s) : e;
}

}  // namespace

// The backward pass for one pair of types, rows > 0.
#define JEPA_LN_BWD_INSTANCE(TX, TY, NAME) \
  cudaError_t NAME(const LnBwdArgs& a, cudaStream_t s) { return bwd_t<TX, TY>(a, s); }

}  // namespace jepa
