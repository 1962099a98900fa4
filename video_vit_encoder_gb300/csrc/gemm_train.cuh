// Tensor-core products of the training operators (sm_103a): persistent CTA
// pairs computing 256 x 256 tiles of C = A B^T with fused epilogues.
//
// Both operands are 16-bit and either contiguous along K (rows of a forward
// product) or along their other dimension (the transposed operands of a
// backward product: dW = dOut^T A reduces over rows).  Either way a stage is
// 64 deep in K and TMA writes it in the 128-byte swizzle that tcgen05.mma
// reads directly, so no transposed copy is ever made:
//   K-major:  one box of 128 rows x 64 k (128 bytes a row);
//   MN-major: two boxes of 64 k x 64 rows, each 64 k-lines of 128 bytes.
//
// Work units are runs of tiles: the cross entropy carries its row statistics
// over a run of column tiles, everything else has runs of one.  K may consist
// of two segments with their own operands (dx = dg Wg + du Wu is one product),
// and may be split between units, each writing its own fp32 slab, which a
// second kernel adds in a fixed order.
//
// Warp roles (320 threads): warp 0 loads, warp 1 issues the MMAs (the even
// CTA's, for the pair), warps 2-9 run the epilogue, two warps per 32 TMEM
// lanes, each half the tile's columns.  Two accumulators of 256 columns fill
// tensor memory, so a tile's epilogue overlaps the next tile's main loop.
#pragma once
#include "train.h"

namespace jepa {
namespace tg {

constexpr int kBM = 128;        // rows per CTA, 256 per pair
constexpr int kBN = 256;        // columns per pair tile
constexpr int kBK = 64;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kStages = 6;
constexpr int kGroupM = 8;      // row tiles that share a sweep over the columns (operand reuse in L2)

constexpr uint32_t kABytes = kBM * kBK * 2;
constexpr uint32_t kBBytes = (kBN / 2) * kBK * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr uint32_t kEpiStage = 4096;   // per epilogue warp: 32 rows x 128 bytes
constexpr uint32_t kEpiOffset = kStages * kStageBytes;
constexpr uint32_t kBarOffset = kEpiOffset + kEpiWarps * kEpiStage;
constexpr size_t kSmemBytes = 1024 + kBarOffset + 256;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

enum Epi : int {
  STORE = 0,     // C (T) = acc * scale
  F32 = 1,       // slab (fp32) = acc
  F32_ADD = 2,   // slab (fp32) += acc
  CE_FWD = 3,    // row statistics of z = acc + bias
  CE_BWD = 4,    // dz (T) from z = acc + bias
  GATE_FWD = 5,  // h (T); columns 0-127 of the tile are gates, 128-255 the same columns' ups
  GATE_BWD = 6   // dg, du (T)
};

struct EpiArgs {
  const float* scale;      // STORE: factor on the device, or null
  const float* bias;       // CE: [N], GATE: gate's [N]
  const float* bias2;      // GATE: up's [N]
  // cross entropy (columns are v0 .. v0 + N of V)
  const int64_t* labels;
  long ignore_index;
  const float* lse;
  const float* dloss;
  const float* dz_scale;   // CE_BWD: power of two on the device, or null
  float smoothing;
  int v0, V;
  float2* part_ms;         // CE_FWD: [parts][M] (max, sum) in base 2
  float* part_sum;         // CE_FWD: [parts][M] sum of z, or null
  float* zy;               // CE_FWD: [M] the label's logit
  float* col_part;         // CE_BWD, GATE_BWD: [ceil(M/32)][ld_col] column sums of 32 rows, or null
  float* col_part2;
  int ld_col;
  const void* dh;          // GATE_BWD: T [M, N]
  int act;
};

struct Params {
  CUtensorMap a[2], b[2], c[2];
  int M, N;              // extents of the output
  int num_m, num_n;      // pair tiles
  int run;               // column tiles per unit
  int kb_seg, nseg;      // K blocks per segment, segments
  int nz;                // products that share B (a[z], c[z])
  int splits, kb_split;  // K splits, blocks per split
  int slab_rows;         // rows of a slab (F32, F32_ADD)
  EpiArgs ep;
  int* status;
};

// One unit: row tile m, columns tiles n0 .. n0 + nr, product z, K blocks kb0 .. kb1.
struct Unit {
  int m, n0, nr, run_index, z, split, kb0, kb1;
};
__host__ __device__ __forceinline__ int unit_count(const Params& p) {
  return p.num_m * ((p.num_n + p.run - 1) / p.run) * p.nz * p.splits;
}
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  Unit t;
  const int runs = (p.num_n + p.run - 1) / p.run;
  const int tiles = p.num_m * runs;
  const int q = u / tiles;
  const int r = u - q * tiles;
  t.split = q / p.nz;
  t.z = q - t.split * p.nz;
  const int group = kGroupM * runs;
  const int gi = r / group, w = r - gi * group;
  const int gm = min(p.num_m - gi * kGroupM, kGroupM);
  t.run_index = w / gm;
  t.m = gi * kGroupM + (w - t.run_index * gm);
  t.n0 = t.run_index * p.run;
  t.nr = min(p.run, p.num_n - t.n0);
  t.kb0 = t.split * p.kb_split;
  t.kb1 = min(t.kb0 + p.kb_split, p.kb_seg * p.nseg);
  return t;
}

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle: 64
// rows (128 bytes) by 8 k per 1024-byte atom, atoms stacked along k (stride
// byte offset 1024); the next 64 rows are the next box, 8192 bytes on
// (leading byte offset).  16 k further is 2048 bytes.
__device__ __forceinline__ uint64_t smem_desc_mnmajor(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(8192 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// Sum over the warp's 32 lanes of v[j] for each j: lane j returns column j's.
// Each step halves the columns a lane still carries; the order is fixed.
__device__ __forceinline__ float warp_col_sum32(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o];
      const float keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

// This warp's staged 32 x 128-byte block, written by `put` (which stores lane's
// row), goes out with one TMA store; the buffer's previous store has been read.
template <typename Put>
__device__ __forceinline__ void stage_store(const CUtensorMap* c, uint8_t* buf, int lane, int x, int y, bool add,
                                            Put&& put) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
  uint8_t* row = buf + lane * 128;
#pragma unroll
  for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(row + ((k ^ (lane & 7)) << 4)) = put(k);
  fence_proxy_async_shared();
  __syncwarp();
  if (lane == 0) {
    if (add) tma_reduce_add_2d(c, buf, x, y);
    else tma_store_2d(c, buf, x, y);
    bulk_commit_group();
  }
}

__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Gate and its slope.  silu: a = g s, a' = s (1 + g (1 - s)) with s = 1 / (1 +
// 2^(-g log2 e)); gelu: a = g Phi(g), a' = Phi(g) + g phi(g).
template <int ACT, bool GRAD>
__device__ __forceinline__ void gate(float g, float& a, float& da) {
  if constexpr (ACT == ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + ex2(-g * kLog2e));
    a = g * s;
    if constexpr (GRAD) da = s * fmaf(g, 1.0f - s, 1.0f);
  } else {
    const float cdf = fmaf(0.5f, erff(g * 0.70710678118654752f), 0.5f);
    a = g * cdf;
    if constexpr (GRAD) da = fmaf(g * 0.3989422804014327f, ex2(g * g * (-0.5f * kLog2e)), cdf);
  }
}

// Statistics a thread carries over a run of the cross entropy: its row's max
// and sum of powers in base 2 (z log2 e), and the sum of z.
struct RowStats {
  float m, s, sum;
};

template <bool SUM>
__device__ __forceinline__ void ce_fwd_tile(const Params& p, uint32_t taddr, int row, int col0, int lane, int label,
                                            RowStats& st) {
  const EpiArgs& ep = p.ep;
#pragma unroll 1
  for (int c = 0; c < kBN / 64; ++c) {
    const int col = col0 + c * 32;
    if (col >= p.N) break;
    // lane j holds column j's bias in base 2, -inf past the vocabulary (whose accumulators are 0)
    const float b = col + lane < p.N ? (ep.bias != nullptr ? __ldg(ep.bias + col + lane) : 0.f) : -INFINITY;
    float v[32];
    tmem_ld32f(taddr + c * 32, v);
    const bool plain = ep.bias == nullptr && col + 32 <= p.N;
    const int ly = label - col;
    if (ly >= 0 && ly < 32) {
      float zy = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) zy = j == ly ? v[j] : zy;
      ep.zy[row] = zy + (ep.bias != nullptr ? __ldg(ep.bias + label) : 0.f);
    }
    if constexpr (SUM) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float bj = __shfl_sync(0xffffffffu, b, j);
        s += col + j < p.N ? v[j] + bj : 0.f;
      }
      st.sum += s;
    }
    if (plain) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= kLog2e;
    } else {
      const float b2 = b * kLog2e;
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = fmaf(v[j], kLog2e, __shfl_sync(0xffffffffu, b2, j));
    }
    float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
    for (int j = 4; j < 32; j += 4) {
      m0 = fmaxf(m0, v[j]); m1 = fmaxf(m1, v[j + 1]); m2 = fmaxf(m2, v[j + 2]); m3 = fmaxf(m3, v[j + 3]);
    }
    const float m = fmaxf(st.m, fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)));
    const float ref = m == -INFINITY ? 0.f : m;   // nothing but -inf so far: every power is 0
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      s0 += ex2(v[j] - ref); s1 += ex2(v[j + 1] - ref); s2 += ex2(v[j + 2] - ref); s3 += ex2(v[j + 3] - ref);
    }
    st.s = fmaf(st.s, ex2(st.m - ref), (s0 + s1) + (s2 + s3));
    st.m = m;
  }
}

template <typename T>
__device__ __forceinline__ void ce_bwd_tile(const Params& p, uint32_t taddr, int row, int col0, uint8_t* buf, int lane) {
  const EpiArgs& ep = p.ep;
  // a row that takes no part (past M, ignored, bad label) gets zeros
  bool part = false;
  int label = -1;       // the label's column of this piece, if it lies in it
  float l2 = 0.f, g = 0.f;
  if (row < p.M) {
    const long y = ep.labels[row];
    part = y != ep.ignore_index && y >= 0 && y < ep.V;
    if (part) {
      label = (int)y - ep.v0;
      l2 = ep.lse[row] * kLog2e;
      g = ep.dloss[row];
    } else if (y != ep.ignore_index && col0 == 0) {
      atomicOr(p.status, DEV_BAD_INDEX);
    }
  }
  const float uni = ep.smoothing / (float)ep.V, hit = 1.0f - ep.smoothing;
  const float zs = ep.dz_scale != nullptr ? __ldg(ep.dz_scale) : 1.0f;
#pragma unroll 1
  for (int c = 0; c < kBN / 128; ++c) {
    const int col = col0 + c * 64;
    if (col >= p.N) break;
    uint32_t w[32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cc = col + h * 32;
      float v[32];
      tmem_ld32f(taddr + c * 64 + h * 32, v);
      if (ep.bias == nullptr && cc + 32 <= p.N) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = ex2(fmaf(v[j], kLog2e, -l2));
      } else {
        const float b2 = (cc + lane < p.N ? (ep.bias != nullptr ? __ldg(ep.bias + cc + lane) : 0.f) : -INFINITY) * kLog2e;
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = ex2(fmaf(v[j], kLog2e, __shfl_sync(0xffffffffu, b2, j)) - l2);
      }
      if (ep.smoothing > 0.f) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] -= uni;
      }
      const int ly = label - cc;
      if (part && ly >= 0 && ly < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = j == ly ? v[j] - hit : v[j];
      }
      if (part) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= g;
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) w[h * 16 + j] = pack2<T>(v[2 * j] * zs, v[2 * j + 1] * zs);
      if (ep.col_part != nullptr) {
        const float s = warp_col_sum32(v, lane);
        if (cc + lane < p.N && row - lane < p.M) ep.col_part[(size_t)(row >> 5) * ep.ld_col + cc + lane] = s;
      }
    }
    stage_store(&p.c[0], buf, lane, col, row - lane, false,
                [&](int k) { return make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]); });
  }
}

// 64 output columns col .. col + 63 from the gates at tg and the ups at tu.
template <typename T, int ACT, bool BWD>
__device__ __forceinline__ void gate_tile(const Params& p, uint32_t tg, uint32_t tu, int row, int col, uint8_t* buf,
                                          int lane) {
  const EpiArgs& ep = p.ep;
  uint32_t wg[32], wu[BWD ? 32 : 1];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int cc = col + h * 32;
    float g[32], u[32];
    uint4 d[BWD ? 4 : 1];
    if constexpr (BWD) {
      // rows are multiples of 16 bytes: an 8-column piece is inside or outside as a whole
      const T* dh = static_cast<const T*>(ep.dh) + (size_t)row * p.N + cc;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = row < p.M && cc + 8 * i < p.N ? __ldg(reinterpret_cast<const uint4*>(dh) + i) : make_uint4(0, 0, 0, 0);
    }
    tmem_ld32f(tg + h * 32, g);
    tmem_ld32f(tu + h * 32, u);
    if (ep.bias != nullptr) {
      const float b = cc + lane < p.N ? __ldg(ep.bias + cc + lane) : 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) g[j] += __shfl_sync(0xffffffffu, b, j);
    }
    if (ep.bias2 != nullptr) {
      const float b = cc + lane < p.N ? __ldg(ep.bias2 + cc + lane) : 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j) u[j] += __shfl_sync(0xffffffffu, b, j);
    }
    if constexpr (!BWD) {
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        float a0, a1, da;
        gate<ACT, false>(g[j], a0, da);
        gate<ACT, false>(g[j + 1], a1, da);
        wg[h * 16 + j / 2] = pack2<T>(a0 * u[j], a1 * u[j + 1]);
      }
    } else {
      const uint32_t* dw = reinterpret_cast<const uint32_t*>(d);
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        T t[2];
        memcpy(t, &dw[j / 2], 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a, da;
          gate<ACT, true>(g[j + i], a, da);
          const float dd = DT<T>::to(t[i]);
          g[j + i] = dd * u[j + i] * da;
          u[j + i] = dd * a;
        }
        wg[h * 16 + j / 2] = pack2<T>(g[j], g[j + 1]);
        wu[h * 16 + j / 2] = pack2<T>(u[j], u[j + 1]);
      }
      const bool put = cc + lane < p.N && row - lane < p.M;
      if (ep.col_part != nullptr) {
        const float s = warp_col_sum32(g, lane);
        if (put) ep.col_part[(size_t)(row >> 5) * ep.ld_col + cc + lane] = s;
      }
      if (ep.col_part2 != nullptr) {
        const float s = warp_col_sum32(u, lane);
        if (put) ep.col_part2[(size_t)(row >> 5) * ep.ld_col + cc + lane] = s;
      }
    }
  }
  if (col >= p.N) return;
  stage_store(&p.c[0], buf, lane, col, row - lane, false,
              [&](int k) { return make_uint4(wg[4 * k], wg[4 * k + 1], wg[4 * k + 2], wg[4 * k + 3]); });
  if constexpr (BWD)
    stage_store(&p.c[1], buf, lane, col, row - lane, false,
                [&](int k) { return make_uint4(wu[4 * k], wu[4 * k + 1], wu[4 * k + 2], wu[4 * k + 3]); });
}

template <typename T>
__device__ __forceinline__ void store_tile(const Params& p, const CUtensorMap* c, uint32_t taddr, int row0, int col0,
                                           uint8_t* buf, int lane) {
  const float sc = p.ep.scale != nullptr ? __ldg(p.ep.scale) : 1.0f;
#pragma unroll 1
  for (int c0 = 0; c0 < kBN / 2; c0 += 64) {
    if (col0 + c0 >= p.N) break;
    uint32_t w[32];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      tmem_ld32f(taddr + c0 + h * 32, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) w[h * 16 + j] = pack2<T>(v[2 * j] * sc, v[2 * j + 1] * sc);
    }
    stage_store(c, buf, lane, col0 + c0, row0, false,
                [&](int k) { return make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]); });
  }
}

__device__ __forceinline__ void slab_tile(const Params& p, const CUtensorMap* c, uint32_t taddr, int row0, int col0,
                                          uint8_t* buf, int lane, bool add) {
#pragma unroll 1
  for (int c0 = 0; c0 < kBN / 2; c0 += 32) {
    if (col0 + c0 >= p.N) break;
    uint32_t w[32];
    tmem_ld32(taddr + c0, w);
    tmem_wait_ld();
    stage_store(c, buf, lane, col0 + c0, row0, add,
                [&](int k) { return make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]); });
  }
}

template <typename T, bool AMN, bool BMN, int EPI>
__global__ void __launch_bounds__(kThreads, 1) train_gemm_kernel(const __grid_constant__ Params p) {
  constexpr bool kGate = EPI == GATE_FWD || EPI == GATE_BWD;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kABytes;
  uint8_t* sEpi = smem + kEpiOffset;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOffset);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;
  const int num_units = unit_count(p);
  const int first = (int)cluster_id_x(), stride = (int)cluster_count_x();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);    // the even CTA's producer arrives; bytes of both CTAs complete it
      mbar_init(&empty[s], 1);   // released by the MMA commit
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);   // one arrival per epilogue warp of both CTAs
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.a[0]);
    tma_prefetch_desc(&p.b[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers and tensor memory exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), 0);
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      bool stop = false;
      for (int u = first; u < num_units && !stop; u += stride) {
        const Unit t = unit_of(p, u);
        const int ra = (t.m * 2 + rank) * kBM;
        for (int r = 0; r < t.nr && !stop; ++r) {
          const int rb = kGate ? (t.n0 + r) * (kBN / 2) : (t.n0 + r) * kBN + rank * (kBN / 2);
          for (int kb = t.kb0; kb < t.kb1; ++kb) {
            if (*abort_flag || !mbar_wait(&empty[stage], phase ^ 1)) {
              atomicOr(p.status, DEV_TIMEOUT);
              *abort_flag = 1;
              stop = true;
              break;
            }
            const int seg = kb >= p.kb_seg ? 1 : 0;
            const int k = (kb - seg * p.kb_seg) * kBK;
            const CUtensorMap* ma = &p.a[seg + t.z];
            const CUtensorMap* mb = &p.b[kGate ? rank : seg];
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
            const uint32_t bar = full0 + 8 * stage;
            uint8_t* da = sA + stage * kABytes;
            uint8_t* db = sB + stage * kBBytes;
            if constexpr (AMN) {
              tma_load_2d_pair(da, ma, bar, ra, k);
              tma_load_2d_pair(da + 8192, ma, bar, ra + 64, k);
            } else {
              tma_load_2d_pair(da, ma, bar, k, ra);
            }
            if constexpr (BMN) {
              tma_load_2d_pair(db, mb, bar, rb, k);
              tma_load_2d_pair(db + 8192, mb, bar, rb + 64, k);
            } else {
              tma_load_2d_pair(db, mb, bar, k, rb);
            }
            ++issued;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
      // Every copy issued must land before the CTAs exit.  The even CTA's
      // barriers count the bytes of both CTAs of the pair.
      if (leader) {
        const long pending = issued < kStages ? issued : kStages;
        for (long i = 0; i < pending; ++i) {
          if (--stage < 0) {
            stage = kStages - 1;
            phase ^= 1;
          }
          mbar_wait(&full[stage], phase);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (the even CTA)
    if (leader) {
      constexpr uint32_t idesc =
          idesc_f16<T, 2 * kBM, kBN>() | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      bool ok = true;
      for (int u = first; u < num_units && ok; u += stride) {
        const Unit t = unit_of(p, u);
        for (int r = 0; r < t.nr && ok; ++r, ++acc) {
          if (__any_sync(0xffffffffu, *abort_flag)) {
            ok = false;
            break;
          }
          const int buf = acc & 1;
          if (!__all_sync(0xffffffffu, mbar_wait(&tempty[buf], ((acc >> 1) & 1) ^ 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + buf * kBN;
          for (int kb = t.kb0; kb < t.kb1; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t aa = smem_u32(sA + stage * kABytes), bb = smem_u32(sB + stage * kBBytes);
            const uint64_t da = AMN ? smem_desc_mnmajor(aa) : smem_desc_kmajor<128>(aa);
            const uint64_t db = BMN ? smem_desc_mnmajor(bb) : smem_desc_kmajor<128>(bb);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
              umma_f16_ss_pair_warp(d, da + k * (AMN ? 128 : 2), db + k * (BMN ? 128 : 2), idesc,
                                    kb != t.kb0 || k != 0);
            umma_commit_pair_warp(&empty[stage], (uint16_t)0x3);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          umma_commit_pair_warp(&tfull[buf], (uint16_t)0x3);
        }
      }
      if (!ok && lane == 0) {
        atomicOr(p.status, DEV_TIMEOUT);
        *abort_flag = 1;
      }
      umma_commit_pair_warp(mma_done, (uint16_t)0x1);   // no MMA may still run when tensor memory is released
      mbar_wait(mma_done, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    uint8_t* buf_s = sEpi + (warp - 2) * kEpiStage;
    int acc = 0;
    bool stop = false;
    for (int u = first; u < num_units && !stop; u += stride) {
      const Unit t = unit_of(p, u);
      const int row = (t.m * 2 + rank) * kBM + quarter * 32 + lane;
      RowStats st{-INFINITY, 0.f, 0.f};
      int label = -1;
      if constexpr (EPI == CE_FWD) {
        if (row < p.M) {
          const long y = p.ep.labels[row];
          label = y >= 0 && y < p.ep.V ? (int)y : -1;
        }
      }
      for (int r = 0; r < t.nr; ++r, ++acc) {
        const int buf = acc & 1;
        const bool ok = mbar_wait(&tfull[buf], (acc >> 1) & 1);
        // tcgen05.ld is warp-collective: the stop decision is warp-uniform
        if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
          if (lane == 0) atomicOr(p.status, DEV_TIMEOUT);
          *abort_flag = 1;
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t tl = tmem_base + ((uint32_t)(quarter * 32) << 16) + buf * kBN;
        const int col = (t.n0 + r) * kBN + half * (kBN / 2);
        if constexpr (EPI == STORE) {
          store_tile<T>(p, &p.c[t.z], tl + half * (kBN / 2), row - lane, col, buf_s, lane);
        } else if constexpr (EPI == F32 || EPI == F32_ADD) {
          slab_tile(p, &p.c[t.z], tl + half * (kBN / 2), row - lane + t.split * p.slab_rows, col, buf_s, lane,
                    EPI == F32_ADD);
        } else if constexpr (EPI == CE_FWD) {
          if (p.ep.part_sum != nullptr) ce_fwd_tile<true>(p, tl + half * (kBN / 2), row, col, lane, label, st);
          else ce_fwd_tile<false>(p, tl + half * (kBN / 2), row, col, lane, label, st);
        } else if constexpr (EPI == CE_BWD) {
          ce_bwd_tile<T>(p, tl + half * (kBN / 2), row, col, buf_s, lane);
        } else {
          const int oc = (t.n0 + r) * (kBN / 2) + half * 64;
          const uint32_t tg = tl + half * 64, tu = tg + kBN / 2;
          if (p.ep.act == ACT_SILU) gate_tile<T, ACT_SILU, EPI == GATE_BWD>(p, tg, tu, row, oc, buf_s, lane);
          else gate_tile<T, ACT_GELU, EPI == GATE_BWD>(p, tg, tu, row, oc, buf_s, lane);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * buf);
      }
      if constexpr (EPI == CE_FWD) {
        if (!stop && row < p.M) {
          const size_t i = (size_t)(t.run_index * 2 + half) * p.M + row;
          p.ep.part_ms[i] = make_float2(st.m, st.s);
          if (p.ep.part_sum != nullptr) p.ep.part_sum[i] = st.sum;
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // the tile stores have completed
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the pair's MMAs and epilogues are done; no signal targets an exited CTA
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Launches over the resident CTA pairs of the current device.
template <typename T, bool AMN, bool BMN, int EPI>
cudaError_t launch(const Params& p, int num_sms, cudaStream_t s) {
  auto kern = train_gemm_kernel<T, AMN, BMN, EPI>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static DeviceOnce setup;
  static int resident_on[kMaxDevices];
  int dev = 0;
  cudaError_t e = setup.run([&](int d) -> cudaError_t {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (r != cudaSuccess) return r;
    int resident = num_sms / 2, n = 0;
    cudaLaunchConfig_t probe = cfg;
    probe.gridDim = dim3(2 * (num_sms / 2));
    if (cudaOccupancyMaxActiveClusters(&n, kern, &probe) == cudaSuccess && n >= 1) resident = n;
    resident_on[d] = resident;
    return cudaSuccess;
  }, &dev);
  if (e != cudaSuccess) return e;
  const long units = (long)p.num_m * ((p.num_n + p.run - 1) / p.run) * p.nz * p.splits;
  if (units < 1 || units > 0x7fffffffl - 4096) return cudaErrorInvalidValue;
  const int clusters = units < resident_on[dev] ? (int)units : resident_on[dev];
  cfg.gridDim = dim3(2 * clusters);
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace tg
}  // namespace jepa

// The instantiations for one type; each type has its own translation unit.
#define JEPA_TRAIN_GEMM_INSTANCES(T, NAME)                                                                  \
  namespace jepa {                                                                                          \
  namespace tg {                                                                                            \
  cudaError_t NAME(bool amn, bool bmn, int epi, const Params& p, int num_sms, cudaStream_t s) {             \
    if (!amn && !bmn) {                                                                                     \
      if (epi == CE_FWD) return launch<T, false, false, CE_FWD>(p, num_sms, s);                             \
      if (epi == CE_BWD) return launch<T, false, false, CE_BWD>(p, num_sms, s);                             \
      if (epi == GATE_FWD) return launch<T, false, false, GATE_FWD>(p, num_sms, s);                         \
      if (epi == GATE_BWD) return launch<T, false, false, GATE_BWD>(p, num_sms, s);                         \
    } else if (!amn) {                                                                                      \
      if (epi == STORE) return launch<T, false, true, STORE>(p, num_sms, s);                                \
      if (epi == F32) return launch<T, false, true, F32>(p, num_sms, s);                                    \
      if (epi == F32_ADD) return launch<T, false, true, F32_ADD>(p, num_sms, s);                            \
    } else if (bmn) {                                                                                       \
      if (epi == STORE) return launch<T, true, true, STORE>(p, num_sms, s);                                 \
      if (epi == F32) return launch<T, true, true, F32>(p, num_sms, s);                                     \
    }                                                                                                       \
    return cudaErrorInvalidValue;                                                                           \
  }                                                                                                         \
  }                                                                                                         \
  }
