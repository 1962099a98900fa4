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
// barrier) while 16 warps per SM work on the current ones.
#pragma once
#include "layernorm_train.cuh"

namespace jepa {

namespace {

constexpr int kMostSmem = 232448;

// The kernel's shape: TPR threads a row, groups of TPR threads up to 16 warps,
// and the rows in flight per thread.  SHIFT takes as many groups as leave two
// rows in flight each (8192 x 7001 in fp32 with a residual 177 us, with 16
// warps 224; 8192 x 4093 in bf16 78 and 84); without its table and masks 16
// warps with fewer rows in flight are faster (16384 x 1536 in fp32 56 us
// against 64).  16384 x 1024 in fp32 with a 16-bit dy and a residual: 41.9 us,
// 0.83 of the copy bandwidth; 73728 x 777 in bf16 70.6 us, 0.72 of it (SHIFT's
// masks and w's table add instructions).
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

  // this thread's first column, and how many columns follow from there
  const int col = t * V - o, left = dim - col;
  const TX* fx = x + first * dim + col;      // of the next row to fetch
  const TY* fg = dy + first * dim + col;
  const TX* fr = RES ? res + first * dim + col : nullptr;
  TX* out_row = dx + first * dim + col;      // of the current row
  const long step = stride * dim;
  // this thread's vectors of the next row into slot d of the ring; the last vector ends with the row (zeros follow)
  long next = first;
  auto fetch = [&](int d) {
    if (next < rows) {
      uint8_t* q = ring + (size_t)d * kThreads * S::kRowVec + tid * kBX;
      uint8_t* qy = ring + (size_t)d * kThreads * S::kRowVec + kOffY + tid * kBY;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i * TPR * V < left) {
          const int n = SHIFT ? min(V, left - i * TPR * V) : V;
          ln_copy_async<kBX>(q + i * kThreads * kBX, fx + i * TPR * V, n * (int)sizeof(TX));
          if constexpr (RES)
            ln_copy_async<kBX>(q + (NV + i) * kThreads * kBX, fr + i * TPR * V, n * (int)sizeof(TX));
          ln_copy_async<kBY>(qy + i * kThreads * kBY, fg + i * TPR * V, n * (int)sizeof(TY));
        }
      }
      fx += step;
      fg += step;
      if constexpr (RES) fr += step;
      next += stride;
    }
    ln_copy_commit();
  };
#pragma unroll
  for (int d = 0; d < S::kDepth; ++d) fetch(d);

  f2 aw[NV][V / 2], ab[NV][V / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V / 2; ++j) aw[i][j] = ab[i][j] = 0ull;

  int d = 0;
  // mean and rstd of 32 rows, one a lane, and of the next 32 (loaded for one row ahead, and handed on in registers, their
  // latency was most of a narrow row's time: 73728 x 768 in bf16 80 us instead of 63)
  const int lane = tid & 31;
  auto stat = [&](const float* p, long from) {
    const long r = from + lane * stride;
    return r < rows ? __ldg(p + r) : 0.f;
  };
  float mean_c = stat(mean, first), rstd_c = stat(rstd, first);
  float mean_n = stat(mean, first + 32 * stride), rstd_n = stat(rstd, first + 32 * stride);
  int k = 0;
  for (long row = first; row < rows; row += stride) {
    if (k == 32) {
      k = 0;
      mean_c = mean_n;
      rstd_c = rstd_n;
      mean_n = stat(mean, row + 32 * stride);
      rstd_n = stat(rstd, row + 32 * stride);
    }
    const float mu = __shfl_sync(0xffffffffu, mean_c, k), rs = __shfl_sync(0xffffffffu, rstd_c, k);
    ++k;
    ln_copy_wait<S::kDepth - 1>();
    const uint8_t* slot = ring + (size_t)d * kThreads * S::kRowVec;
    const f2 mu2 = f2_make(-mu, -mu), rs2 = f2_make(rs, rs);
    // x - mean in xv and c = dy w in gv; the previous row's values and the zeros after the row meet w = 0 and dy = 0
    f2 xv[NV][V / 2], gv[NV][V / 2];
    f2 sa = 0ull, sb = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * TPR * V < left) {
        LnVec<TX, V> vx;
        LnVec<TY, V> vg;
        vx.load(slot + tid * kBX + i * kThreads * kBX);
        vg.load(slot + kOffY + tid * kBY + i * kThreads * kBY);
        if (SHIFT && i == 0) {
          vx.drop_head(head);
          vg.drop_head(head);
        }
        vx.pairs(xv[i]);
        vg.pairs(gv[i]);
        f2 ww[V / 2];
        if constexpr (SHIFT && !S::kTable) {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const int c = col + i * TPR * V + j;
            ww[j / 2] = f2_make(c >= 0 && c < dim ? __ldg(w + c) : 0.f, c + 1 >= 0 && c + 1 < dim ? __ldg(w + c + 1) : 0.f);
          }
        } else if constexpr (SHIFT) {
          S::Table::load(table, i, ww);
        } else {
          ln_floats<V>((S::kTable ? table : w) + col + i * TPR * V, ww);
        }
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          xv[i][j] = f2_add(xv[i][j], mu2);
          const f2 xh = f2_mul(xv[i][j], rs2);
          aw[i][j] = f2_fma(gv[i][j], xh, aw[i][j]);
          ab[i][j] = f2_add(ab[i][j], gv[i][j]);
          gv[i][j] = f2_mul(gv[i][j], ww[j]);
          sa = f2_add(sa, gv[i][j]);
          sb = f2_fma(gv[i][j], xh, sb);
        }
      }
    }
    if constexpr (!RES) fetch(d);   // the slot has been read
    float s[2] = {f2_sum(sa), f2_sum(sb)};
    ln_row_sum<TPR, 2>(s, red);
    // dx = rs c - rs m0 - (rs m1 rs) (x - mean)
    const float k0 = -rs * (s[0] * inv), k1 = -rs * (s[1] * inv) * rs;
    const f2 k02 = f2_make(k0, k0), k12 = f2_make(k1, k1);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * TPR * V < left) {
        f2 out[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) out[j] = f2_fma(gv[i][j], rs2, f2_fma(xv[i][j], k12, k02));
        if constexpr (RES) {
          LnVec<TX, V> vr;
          f2 r[V / 2];
          vr.load(slot + tid * kBX + (NV + i) * kThreads * kBX);
          vr.pairs(r);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) out[j] = f2_add(out[j], r[j]);
        }
        LnVec<TX, V> vo;
        vo.set(out);
        TX* to = out_row + i * TPR * V;
        if (!SHIFT || ((i > 0 || head == 0) && i * TPR * V + V <= left)) vo.store(to);
        else ln_store_part<TX, V>(to, i == 0 ? head : 0, left - i * TPR * V, vo);   // shared with a neighbouring row
      }
    }
    if constexpr (RES) fetch(d);   // the slot has been read
    if (++d == S::kDepth) d = 0;
    out_row += step;
  }
  ln_copy_wait<0>();

  // the groups' sums side by side in shared memory, then added in their order
  float* pw = part_w + (size_t)blockIdx.x * 2 * dim;
  float* pb = part_b + (size_t)blockIdx.x * 2 * dim;
  __syncthreads();
  float* mine = reinterpret_cast<float*>(ring) + (size_t)(tid / TPR) * 2 * dim;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const int c = col + i * TPR * V + 2 * j;
      float w0, w1, b0, b1;
      f2_get(aw[i][j], w0, w1);
      f2_get(ab[i][j], b0, b1);
      if (c >= 0 && c < dim) {
        mine[c] = w0;
        mine[dim + c] = b0;
      }
      if (c + 1 >= 0 && c + 1 < dim) {
        mine[c + 1] = w1;
        mine[dim + c + 1] = b1;
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

// The fewest threads a row that hold at most 16 columns each: x - mean, c and the
// sums of dw and db of 16 columns fit in the registers that 16 warps have.
template <typename TX, typename TY, int V, bool SHIFT, bool RES>
cudaError_t launch_width(const Args& a, cudaStream_t s) {
  const int n = a.dim + (SHIFT ? V - 1 : 0);   // columns that the vectors cover
  if (n <= 256) return launch_rows<TX, TY, V, 8 / V, 32, SHIFT, RES>(a, s);
  if (n <= 512) return launch_rows<TX, TY, V, 16 / V, 32, SHIFT, RES>(a, s);
  if (n <= 1024) return launch_rows<TX, TY, V, 16 / V, 64, SHIFT, RES>(a, s);
  if (n <= 2048) return launch_rows<TX, TY, V, 16 / V, 128, SHIFT, RES>(a, s);
  if (n <= 4096) return launch_rows<TX, TY, V, 16 / V, 256, SHIFT, RES>(a, s);
  return launch_rows<TX, TY, V, 16 / V, 512, SHIFT, RES>(a, s);
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
