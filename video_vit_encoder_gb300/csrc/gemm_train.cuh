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
// fp32 operands (SPLIT) come as three bf16 planes x = x0 + x1 + x2, each the
// rounding of what the ones before leave, 24 bits and more together.  Of the
// nine products of planes the six with i + j <= 2 are taken; the others are
// below 2^-24 of the first.  That is 6 times the work of a bf16 product and
// still several times the FFMA rate.
//
// The tensor core truncates its fp32 accumulator at every step of 16 k: after n
// steps a sum has lost about n 2^-25 of itself (measured: logits over 1024 k
// 1.5e-6 too small).  Epilogues whose results are fp32 therefore take the
// accumulator out every kb_chunk blocks and add the pieces in registers, with
// rounding; SPLIT does so every block, with the products of the small planes
// first, whose steps then truncate a small accumulator.
//
// Work units are runs of tiles: the cross entropy carries its row statistics
// over a run of column tiles, everything else has runs of one.  The reducing
// products of a backward pass (dx and dW) are two jobs of one launch, so that
// the units of one fill the last round of the other.  K may consist of two
// segments with their own operands (dx = dg Wg + du Wu is one product), and may
// be split between units, each writing its own fp32 slab, which a second kernel
// adds in a fixed order.
//
// Warp roles: warp 0 loads, warp 1 issues the MMAs (the even CTA's, for the
// pair), eight warps run the epilogue, two per 32 TMEM lanes, each half the
// tile's columns.  Two accumulators of 256 columns fill tensor memory, so a
// tile's epilogue overlaps the next tile's main loop.  Epilogues that hold
// their 128 columns in registers run in three warpgroups, of which the first
// (load, issue, two idle warps) hands registers to the other two.
#pragma once
#include "train.h"

namespace jepa {
namespace tg {

constexpr int kBM = 128;        // rows per CTA, 256 per pair
constexpr int kBN = 256;        // columns per pair tile
constexpr int kBK = 64;
constexpr int kEpiWarps = 8;
constexpr int kRegsControl = 72, kRegsEpi = 216;   // 128 x 72 + 256 x 216 = 384 x 168, the launch allocation
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
  REDUCE = 0,    // C per job: see Out
  CE_FWD = 1,    // row statistics of z = acc + bias
  CE_BWD = 2,    // dz (T, or planes) from z = acc + bias
  GATE_FWD = 3,  // h (T, or fp32); columns 0-127 of the tile are gates, 128-255 the same columns' ups
  GATE_BWD = 4   // dg, du (T, or planes)
};
enum Out : int {
  STORE = 0,     // C (T) = acc * scale
  F32 = 1,       // slab, or C in fp32 = acc
  F32_ADD = 2    // slab, or C in fp32 += acc
};

struct EpiArgs {
  const float* bias;       // CE: [N], GATE: gate's [N]
  const float* bias2;      // GATE: up's [N]
  // cross entropy (columns are v0 .. v0 + N of V)
  const int64_t* labels;
  long ignore_index;
  const float* lse;
  const float* dloss;
  const float* dz_scale;   // CE_BWD, 16-bit: [0] what dloss is divided by, [1] the factor of every dz
  float smoothing;
  int v0, V;
  float2* part_ms;         // CE_FWD: [parts][M] (max, sum) in base 2
  float* part_sum;         // CE_FWD: [parts][M] sum of z, or null
  float* zy;               // CE_FWD: [M] the label's logit
  float* col_part;         // CE_BWD, GATE_BWD: [ceil(M/32)][ld_col] column sums of 32 rows, or null
  float* col_part2;
  int ld_col;
  const void* dh;          // GATE_BWD: [M, N] in the operator's type
  int dh_vec;              // its rows start on 16 bytes
  int act;
};

// One product, or nz products that share B.
struct Job {
  CUtensorMap a[2], b[2], c[2];   // a[segment + z], b[segment] (gates: gate, up), c[z]
  int M, N;              // extents of the output
  int num_m, num_n;      // pair tiles
  int kb_seg, nseg;      // K blocks per segment, segments
  int nz;
  int splits, kb_split;  // K splits, blocks per split
  int a_plane, b_plane;  // SPLIT: rows from one plane to the next
  int a_mn;              // REDUCE: A is MN-major (B always is); else both are K-major
  int out;               // REDUCE
  int slab_rows;         // REDUCE: rows of a slab
  const float* scale;    // REDUCE, STORE: factor on the device, or null
};

struct Params {
  Job j[2];
  int units[2];          // of each job
  int extra;             // units of job 1 that a pair takes while others do their last of job 0
  int run;               // column tiles per unit
  int kb_chunk;          // blocks accumulated in tensor memory before the epilogue takes them
  int c_plane;           // SPLIT: rows from one plane of C to the next
  void* plain;           // C where TMA cannot store it (rows not multiples of 16 bytes), else null
  long plain_ld;
  EpiArgs ep;
  int* status;
};

// The units of one CTA pair.  Job 0 has the longer units and goes first, round
// robin; in its last, partial round the pairs without a unit of it take `extra`
// units of job 1 each; what is left of job 1 goes round robin, beginning with
// those pairs.
struct Walk {
  int cid, nc, full, part;   // pair, pairs, whole rounds of job 0, pairs in its last one
  __device__ __forceinline__ Walk(const Params& p, int cid_, int nc_) : cid(cid_), nc(nc_) {
    full = p.units[0] / nc;
    part = p.units[0] - full * nc;
  }
  // The i-th unit, counted over both jobs, or -1.
  __device__ __forceinline__ int at(const Params& p, int i) const {
    if (i < full || (i == full && cid < part)) return i * nc + cid;
    if (p.units[1] == 0) return -1;
    i -= full + (cid < part ? 1 : 0);
    int base = 0;
    if (part != 0) {
      base = min(p.units[1], (nc - part) * p.extra);
      if (cid >= part) {
        if (i < p.extra) {
          const int k = cid - part + i * (nc - part);
          return k < p.units[1] ? p.units[0] + k : -1;
        }
        i -= p.extra;
      }
    }
    const int k = base + i * nc + (cid >= part ? cid - part : cid - part + nc);
    return k < p.units[1] ? p.units[0] + k : -1;
  }
};

// One unit: row tile m, columns tiles n0 .. n0 + nr, product z, K blocks kb0 .. kb1.
struct Unit {
  int job, m, n0, nr, run_index, z, split, kb0, kb1;
};
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  Unit t;
  t.job = u >= p.units[0] ? 1 : 0;
  if (t.job) u -= p.units[0];
  const Job& j = p.j[t.job];
  const int runs = (j.num_n + p.run - 1) / p.run;
  const int tiles = j.num_m * runs;
  const int q = u / tiles;
  const int r = u - q * tiles;
  t.split = q / j.nz;
  t.z = q - t.split * j.nz;
  const int group = kGroupM * runs;
  const int gi = r / group, w = r - gi * group;
  const int gm = min(j.num_m - gi * kGroupM, kGroupM);
  t.run_index = w / gm;
  t.m = gi * kGroupM + (w - t.run_index * gm);
  t.n0 = t.run_index * p.run;
  t.nr = min(p.run, j.num_n - t.n0);
  t.kb0 = t.split * j.kb_split;
  t.kb1 = min(t.kb0 + j.kb_split, j.kb_seg * j.nseg);
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

// Arrival on a barrier of the pair that hands back tensor memory: the loads
// before it have completed (tcgen05.wait::ld and the fence), and no memory is
// passed on, so it need not wait for the thread's stores as a release does.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Packed arithmetic on two neighbouring values: (a, b) = (a, b) m + (c, c), and
// products with one factor.  The epilogues are bound by instruction issue.
__device__ __forceinline__ void fma2(float& a, float& b, float m, float c) {
  uint64_t v, k, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(k) : "f"(m));
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(c));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(k), "l"(d));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ void mul2(float& a, float& b, float m) {
  uint64_t v, k;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(k) : "f"(m));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(k));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
  uint64_t v, k;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(k) : "f"(x), "f"(y));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(k));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// v += the 32 biases from column col on; columns at or past n get `past`.
// Every lane reads the same addresses.
__device__ __forceinline__ void add_bias(const float* bias, int col, int n, float past, float* v) {
  const float* b = bias + col;
  if (col + 32 <= n && (reinterpret_cast<uintptr_t>(b) & 15) == 0) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(b + j));
      add2f(v[j], v[j + 1], q.x, q.y);
      add2f(v[j + 2], v[j + 3], q.z, q.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += col + j < n ? __ldg(b + j) : past;
  }
}

// Column sums over the warp's 32 rows of 32 columns, written to part[0 .. n):
// the block goes through the staging buffer (its last store has to have been
// read), a lane sums 16 rows of two columns, and the two row groups are joined.
__device__ __forceinline__ void col_sum32(const float* v, uint8_t* buf, int lane, float* part, int n) {
  uint8_t* row = buf + lane * 128;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    *reinterpret_cast<float4*>(row + ((k ^ (lane & 7)) << 4)) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  __syncwarp();
  // lane (g, k) sums rows 16 g .. 16 g + 15 of columns 2 k, 2 k + 1
  const int k = lane & 15, g = lane >> 4;
  float s0 = 0.f, s1 = 0.f, t0 = 0.f, t1 = 0.f;
#pragma unroll
  for (int r = 0; r < 16; r += 2) {
    const float2 q = *reinterpret_cast<const float2*>(buf + (g * 16 + r) * 128 + (((k >> 1) ^ (r & 7)) << 4) + (k & 1) * 8);
    const float2 p = *reinterpret_cast<const float2*>(buf + (g * 16 + r + 1) * 128 + (((k >> 1) ^ ((r + 1) & 7)) << 4) + (k & 1) * 8);
    add2f(s0, s1, q.x, q.y);
    add2f(t0, t1, p.x, p.y);
  }
  s0 += t0;
  s1 += t1;
  s0 += __shfl_xor_sync(0xffffffffu, s0, 16);
  s1 += __shfl_xor_sync(0xffffffffu, s1, 16);
  __syncwarp();   // the buffer has been read
  const int c = 2 * k + g;
  if (c < n) part[c] = g == 0 ? s0 : s1;
}

// This warp's 32 x 128-byte block of C at column x, row y, from each lane's row
// of eight 16-byte words: through the staging buffer (swizzled, so neither side
// has bank conflicts) and out with one TMA store, which clips it to C.
template <typename Put>
__device__ __forceinline__ void emit(const CUtensorMap* c, uint8_t* buf, int lane, int x, int y, bool add, Put&& put) {
  if (lane == 0) bulk_wait_read_all();   // the previous store has read the buffer
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
// The same with plain stores, a row at a time, for a C that TMA cannot address.
template <typename E, typename Put>
__device__ __forceinline__ void emit_plain(E* c, long ld, int rows, int cols, uint8_t* buf, int lane, int x, int y,
                                           Put&& put) {
  __syncwarp();
  uint8_t* row = buf + lane * 128;
#pragma unroll
  for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(row + ((k ^ (lane & 7)) << 4)) = put(k);
  __syncwarp();
  constexpr int kPer = 4 / sizeof(E);
  for (int r = 0; r < 32 && y + r < rows; ++r) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
    E e[kPer];
    memcpy(e, &w, 4);
    E* dst = c + (long)(y + r) * ld + x + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (x + lane * kPer + i < cols) dst[i] = e[i];
  }
  __syncwarp();
}

__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 64 columns v[at ..] of an intermediate operand (dz, dg, du): the type's
// rounding, or three bf16 planes, each the rounding of what the ones before
// leave (v is used up).
template <typename T, bool SPLIT>
__device__ __forceinline__ void emit_operand(const Params& p, const CUtensorMap* c, float (&v)[128], int at,
                                             uint8_t* buf, int lane, int x, int y) {
#pragma unroll
  for (int pl = 0; pl < (SPLIT ? 3 : 1); ++pl) {
    emit(c, buf, lane, x, y + pl * p.c_plane, false, [&](int k) {
      const float* q = v + at + 8 * k;
      return make_uint4(pack2<T>(q[0], q[1]), pack2<T>(q[2], q[3]), pack2<T>(q[4], q[5]), pack2<T>(q[6], q[7]));
    });
    if (SPLIT && pl < 2) {
#pragma unroll
      for (int j = 0; j < 64; ++j) v[at + j] -= DT<T>::to(DT<T>::from(v[at + j]));
    }
  }
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
__device__ __forceinline__ void ce_fwd_tile(const Params& p, float (&v)[128], int row, int col0, int lane, int label,
                                            RowStats& st) {
  const EpiArgs& ep = p.ep;
  const int ly = label - col0;
  if (ly >= 0 && ly < 128) {
    float zy = 0.f;
#pragma unroll
    for (int j = 0; j < 128; ++j) zy = j == ly ? v[j] : zy;
    ep.zy[row] = zy + (ep.bias != nullptr ? __ldg(ep.bias + label) : 0.f);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int col = col0 + c * 32;
    if (col >= p.j[0].N) continue;
    float* w = v + c * 32;
    if (ep.bias != nullptr) {
      add_bias(ep.bias, col, p.j[0].N, -INFINITY, w);
    } else if (col + 32 > p.j[0].N) {
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = col + j < p.j[0].N ? w[j] : -INFINITY;
    }
    if constexpr (SUM) {
      float s = 0.f;
      if (col + 32 <= p.j[0].N) {
#pragma unroll
        for (int j = 0; j < 32; ++j) s += w[j];
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) s += col + j < p.j[0].N ? w[j] : 0.f;
      }
      st.sum += s;
    }
    float m0 = max3(w[0], w[1], w[2]), m1 = max3(w[3], w[4], w[5]);
#pragma unroll
    for (int j = 6; j < 30; j += 4) {
      m0 = max3(m0, w[j], w[j + 1]);
      m1 = max3(m1, w[j + 2], w[j + 3]);
    }
    const float m = fmaxf(st.m, max3(m0, m1, fmaxf(w[30], w[31])) * kLog2e);
    const float ref = m == -INFINITY ? 0.f : m;   // nothing but -inf so far: every power is 0
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      fma2(w[j], w[j + 1], kLog2e, -ref);
      fma2(w[j + 2], w[j + 3], kLog2e, -ref);
      add2f(s0, s1, ex2(w[j]), ex2(w[j + 1]));
      add2f(s2, s3, ex2(w[j + 2]), ex2(w[j + 3]));
    }
    st.s = fmaf(st.s, ex2(st.m - ref), (s0 + s1) + (s2 + s3));
    st.m = m;
  }
}

// What the cross entropy's gradient needs of a thread's row.  A row that takes
// no part (past M, ignored, bad label) gets zeros.
struct RowGrad {
  bool part;
  int label;      // the label's column of this piece, if it lies in it
  float l2, g;    // lse in base 2, the row's factor
};
template <bool SPLIT>
__device__ __forceinline__ RowGrad ce_bwd_row(const Params& p, int row, bool report) {
  const EpiArgs& ep = p.ep;
  RowGrad r{false, -1, 0.f, 0.f};
  if (row < p.j[0].M) {
    const long y = __ldg(reinterpret_cast<const long long*>(ep.labels) + row);
    const float lse = __ldg(ep.lse + row), dl = __ldg(ep.dloss + row);
    r.part = y != ep.ignore_index && y >= 0 && y < ep.V;
    if (r.part) {
      r.label = (int)y - ep.v0;
      r.l2 = lse * kLog2e;
      r.g = dl;
      if constexpr (!SPLIT) r.g = dl / __ldg(ep.dz_scale) * __ldg(ep.dz_scale + 1);
    } else if (y != ep.ignore_index && report) {
      atomicOr(p.status, DEV_BAD_INDEX);
    }
  }
  return r;
}

template <typename T, bool SPLIT>
__device__ __forceinline__ void ce_bwd_tile(const Params& p, float (&v)[128], const RowGrad& rg, int row, int col0,
                                            uint8_t* buf, int lane) {
  const EpiArgs& ep = p.ep;
  const bool part = rg.part;
  const int label = rg.label;
  const float l2 = rg.l2, g = rg.g;
  // 16-bit dz is held as g ((p - e / V) / (1 - e) - [v = y]) with g = dloss / max |dloss| (times 2^14 in fp16): with one
  // dloss for all rows, as a mean's, the label's entry is then near -1, which 16 bits hold exactly.  (As dloss (p - (1 - e)
  // [v = y] - e / V) those entries, which make up most of dx and dW, were all off by the same rounding of dloss: dx and
  // dW 3.0e-3 from the exact gradients in norm instead of 1.7e-3 at 1999 x 768 x 50021 in bf16.)
  const float uni = ep.smoothing / (float)ep.V;
  const float cs = SPLIT ? 1.0f : 1.0f / (1.0f - ep.smoothing), hit = SPLIT ? 1.0f - ep.smoothing : 1.0f;
  const int y = row - lane;
  if (ep.col_part != nullptr) {
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int cc = col0 + c * 32;
    float* w = v + c * 32;
    if (cc >= p.j[0].N) continue;
    // columns past N keep finite values: nothing reads them
    if (ep.bias != nullptr) add_bias(ep.bias, cc, p.j[0].N, 0.f, w);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      fma2(w[j], w[j + 1], kLog2e, -l2);
      w[j] = ex2(w[j]);
      w[j + 1] = ex2(w[j + 1]);
    }
    if (ep.smoothing > 0.f) {
#pragma unroll
      for (int j = 0; j < 32; j += 2) fma2(w[j], w[j + 1], cs, -uni * cs);
    }
    const int ly = label - cc;
    if (part && ly >= 0 && ly < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = j == ly ? w[j] - hit : w[j];
    }
#pragma unroll
    for (int j = 0; j < 32; j += 2) mul2(w[j], w[j + 1], g);
    if (!part) {
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = 0.f;
    }
    // its column sums, while the next 32 columns are computed
    if (ep.col_part != nullptr)
      col_sum32(w, buf, lane, ep.col_part + (size_t)(y >> 5) * ep.ld_col + cc, y < p.j[0].M ? p.j[0].N - cc : 0);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (col0 + c * 64 < p.j[0].N) emit_operand<T, SPLIT>(p, &p.j[0].c[0], v, c * 64, buf, lane, col0 + c * 64, y);
}

// Copies this warp's 32 x 64 block of dh into the staging buffer (swizzled as
// emit's), whose last store has to have been read; rows are multiples of 16
// bytes.
template <typename T>
__device__ __forceinline__ void fetch_dh(const Params& p, uint8_t* buf, int lane, int col, int row0) {
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
  const int k = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    const bool in = row0 + r < p.j[0].M && col + 8 * k < p.j[0].N;
    const T* src = static_cast<const T*>(p.ep.dh) + (in ? (size_t)(row0 + r) * p.j[0].N + col + 8 * k : 0);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(buf + r * 128 + ((k ^ (r & 7)) << 4))),
                 "l"(src), "r"(in ? 16 : 0)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// 64 output columns col .. col + 63 from the gates v[0..63] and the ups v[64..127].
template <typename T, bool SPLIT, int ACT, bool BWD>
__device__ __forceinline__ void gate_tile(const Params& p, float (&v)[128], int row, int col, uint8_t* buf, int lane) {
  using TD = typename std::conditional<SPLIT, float, T>::type;   // the operator's type
  const EpiArgs& ep = p.ep;
  if constexpr (BWD && !SPLIT) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  if (col >= p.j[0].N) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int cc = col + h * 32;
    float* g = v + h * 32;
    float* u = v + 64 + h * 32;
    if (ep.bias != nullptr) add_bias(ep.bias, cc, p.j[0].N, 0.f, g);
    if (ep.bias2 != nullptr) add_bias(ep.bias2, cc, p.j[0].N, 0.f, u);
    if constexpr (!BWD) {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float a, da;
        gate<ACT, false>(g[j], a, da);
        g[j] = a * u[j];
      }
    } else {
      constexpr int kPer = 16 / sizeof(TD);   // values of dh in 16 bytes
      const TD* dh = static_cast<const TD*>(ep.dh) + (size_t)row * p.j[0].N + cc;
#pragma unroll
      for (int j = 0; j < 32; j += kPer) {
        TD d[kPer];
        if (ep.dh_vec) {
          uint4 q;
          if constexpr (!SPLIT)   // fetch_dh has put it into the staging buffer
            q = *reinterpret_cast<const uint4*>(buf + lane * 128 + (((h * 4 + j / 8) ^ (lane & 7)) << 4));
          else   // rows are multiples of 16 bytes: a piece is inside or outside as a whole
            q = row < p.j[0].M && cc + j < p.j[0].N ? __ldg(reinterpret_cast<const uint4*>(dh + j)) : make_uint4(0, 0, 0, 0);
          memcpy(d, &q, 16);
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i) d[i] = row < p.j[0].M && cc + j + i < p.j[0].N ? dh[j + i] : DT<TD>::from(0.f);
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          float a, da;
          gate<ACT, true>(g[j + i], a, da);
          const float dd = DT<TD>::to(d[i]);
          g[j + i] = dd * u[j + i] * da;
          u[j + i] = dd * a;
        }
      }
    }
  }
  if constexpr (BWD) {
    const int y = row - lane;
    __syncwarp();   // dh has been read from the staging buffer
    if (ep.col_part != nullptr || ep.col_part2 != nullptr) {
      if (lane == 0) bulk_wait_read_all();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float* part = k == 0 ? ep.col_part : ep.col_part2;
        if (part == nullptr) continue;
        float* to = part + (size_t)(y >> 5) * ep.ld_col + col;
        const int n = y < p.j[0].M ? p.j[0].N - col : 0;
        col_sum32(v + k * 64, buf, lane, to, n);
        col_sum32(v + k * 64 + 32, buf, lane, to + 32, n - 32);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) emit_operand<T, SPLIT>(p, &p.j[0].c[k], v, k * 64, buf, lane, col, y);
  } else if constexpr (!SPLIT) {
    auto put = [&](int k) {
      const float* q = v + 8 * k;
      return make_uint4(pack2<T>(q[0], q[1]), pack2<T>(q[2], q[3]), pack2<T>(q[4], q[5]), pack2<T>(q[6], q[7]));
    };
    if (p.plain == nullptr) emit(&p.j[0].c[0], buf, lane, col, row - lane, false, put);
    else emit_plain(static_cast<T*>(p.plain), p.plain_ld, p.j[0].M, p.j[0].N, buf, lane, col, row - lane, put);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      auto put = [&](int k) {
        const float* q = v + h * 32 + 4 * k;
        return make_uint4(__float_as_uint(q[0]), __float_as_uint(q[1]), __float_as_uint(q[2]), __float_as_uint(q[3]));
      };
      const int cc = col + h * 32;
      if (cc >= p.j[0].N) break;
      if (p.plain == nullptr) emit(&p.j[0].c[0], buf, lane, cc, row - lane, false, put);
      else emit_plain(static_cast<float*>(p.plain), p.plain_ld, p.j[0].M, p.j[0].N, buf, lane, cc, row - lane, put);
    }
  }
}

// 128 columns of a 16-bit C straight from tensor memory.
template <typename T>
__device__ __forceinline__ void store_tile(const Job& p, const CUtensorMap* c, uint32_t taddr, int row0, int col0,
                                           uint8_t* buf, int lane) {
  const float sc = p.scale != nullptr ? __ldg(p.scale) : 1.0f;
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
    emit(c, buf, lane, col0 + c0, row0, false,
         [&](int k) { return make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]); });
  }
}
// 128 columns of an fp32 C: straight from tensor memory, or the register sums.
__device__ __forceinline__ void slab_tile(const Job& p, const CUtensorMap* c, uint32_t taddr, int row0, int col0,
                                          uint8_t* buf, int lane, bool add) {
#pragma unroll 1
  for (int c0 = 0; c0 < kBN / 2; c0 += 32) {
    if (col0 + c0 >= p.N) break;
    uint32_t w[32];
    tmem_ld32(taddr + c0, w);
    tmem_wait_ld();
    emit(c, buf, lane, col0 + c0, row0, add,
         [&](int k) { return make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]); });
  }
}
__device__ __forceinline__ void slab_regs(const Job& p, const CUtensorMap* c, const float (&v)[128], int row0,
                                          int col0, uint8_t* buf, int lane, bool add) {
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += 32) {
    if (col0 + c0 >= p.N) continue;
    emit(c, buf, lane, col0 + c0, row0, add, [&](int k) {
      const float* q = v + c0 + 4 * k;
      return make_uint4(__float_as_uint(q[0]), __float_as_uint(q[1]), __float_as_uint(q[2]), __float_as_uint(q[3]));
    });
  }
}

// Whether an epilogue adds a tile's chunks in registers, and the block's shape.
template <bool SPLIT, int EPI>
struct Shape {
  static constexpr bool kRegs = SPLIT || EPI >= CE_FWD;
  static constexpr int kFirstEpi = kRegs ? 4 : 2;
  static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
};

template <typename T, bool SPLIT, int EPI>
__global__ void __launch_bounds__(Shape<SPLIT, EPI>::kThreads, 1) train_gemm_kernel(const __grid_constant__ Params p) {
  constexpr bool kGate = EPI == GATE_FWD || EPI == GATE_BWD;
  constexpr int kPlanes = SPLIT ? 3 : 1;
  static_assert(kStages % kPlanes == 0, "the planes of a block take consecutive stages");
  constexpr bool BMN = EPI == REDUCE;
  constexpr bool kRegs = Shape<SPLIT, EPI>::kRegs;
  constexpr int kFirstEpi = Shape<SPLIT, EPI>::kFirstEpi;
  constexpr bool kStageDh = EPI == GATE_BWD && !SPLIT;   // 64 columns of 16 bits are a row of the staging buffer
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
  const Walk walk(p, (int)cluster_id_x(), (int)cluster_count_x());

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
    tma_prefetch_desc(&p.j[0].a[0]);
    tma_prefetch_desc(&p.j[0].b[0]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers and tensor memory exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < kFirstEpi) {
    if constexpr (kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer (both CTAs)
      if (lane == 0) {
        const uint32_t full0 = mapa_shared(smem_u32(full), 0);
        int stage = 0;
        uint32_t phase = 0;
        long issued = 0;
        bool stop = false;
        for (int i = 0, u; !stop && (u = walk.at(p, i)) >= 0; ++i) {
          const Unit t = unit_of(p, u);
          const Job& job = p.j[t.job];
          const bool amn = BMN && job.a_mn != 0;
          const int ra = (t.m * 2 + rank) * kBM;
          for (int r = 0; r < t.nr && !stop; ++r) {
            const int rb = kGate ? (t.n0 + r) * (kBN / 2) : (t.n0 + r) * kBN + rank * (kBN / 2);
            for (int q = t.kb0 * kPlanes; q < t.kb1 * kPlanes; ++q) {
              if (*abort_flag || !mbar_wait(&empty[stage], phase ^ 1)) {
                atomicOr(p.status, DEV_TIMEOUT);
                *abort_flag = 1;
                stop = true;
                break;
              }
              const int kb = SPLIT ? q / 3 : q, plane = SPLIT ? q - 3 * kb : 0;
              const int seg = kb >= job.kb_seg ? 1 : 0;
              const int k = (kb - seg * job.kb_seg) * kBK;
              const CUtensorMap* ma = &job.a[seg + t.z];
              const CUtensorMap* mb = &job.b[kGate ? rank : seg];
              if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
              const uint32_t bar = full0 + 8 * stage;
              uint8_t* da = sA + stage * kABytes;
              uint8_t* db = sB + stage * kBBytes;
              // the planes lie one after another along the stored matrix's rows
              const int pa = plane * job.a_plane, pb = plane * job.b_plane;
              if (amn) {
                tma_load_2d_pair(da, ma, bar, ra, k + pa);
                tma_load_2d_pair(da + 8192, ma, bar, ra + 64, k + pa);
              } else {
                tma_load_2d_pair(da, ma, bar, k, ra + pa);
              }
              if constexpr (BMN) {
                tma_load_2d_pair(db, mb, bar, rb, k + pb);
                tma_load_2d_pair(db + 8192, mb, bar, rb + 64, k + pb);
              } else {
                tma_load_2d_pair(db, mb, bar, k, rb + pb);
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
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        bool ok = true;
        for (int i = 0, u; ok && (u = walk.at(p, i)) >= 0; ++i) {
          const Unit t = unit_of(p, u);
          const bool amn = BMN && p.j[t.job].a_mn != 0;
          const uint32_t idesc = idesc_f16<T, 2 * kBM, kBN>() | (amn ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u);
          const uint32_t step = amn ? 128 : 2;   // 16 k on in A's descriptor
          for (int r = 0; r < t.nr && ok; ++r) {
            for (int c0 = t.kb0; c0 < t.kb1 && ok; c0 += p.kb_chunk, ++acc) {
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
              const int c1 = min(c0 + p.kb_chunk, t.kb1);
              for (int kb = c0; kb < c1 && ok; ++kb) {
#pragma unroll
                for (int pl = 0; pl < kPlanes; ++pl)
                  ok = ok && __all_sync(0xffffffffu, mbar_wait(&full[stage + pl], phase));
                if (!ok) break;
                tc_fence_after();
                uint64_t da[kPlanes], db[kPlanes];
#pragma unroll
                for (int pl = 0; pl < kPlanes; ++pl) {
                  const uint32_t aa = smem_u32(sA + (stage + pl) * kABytes), bb = smem_u32(sB + (stage + pl) * kBBytes);
                  da[pl] = amn ? smem_desc_mnmajor(aa) : smem_desc_kmajor<128>(aa);
                  db[pl] = BMN ? smem_desc_mnmajor(bb) : smem_desc_kmajor<128>(bb);
                }
                // planes (i, j) with i + j = 2, then 1, then 0: the small products first
#pragma unroll
                for (int order = kPlanes - 1; order >= 0; --order)
#pragma unroll
                  for (int pa = 0; pa <= order; ++pa)
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                      umma_f16_ss_pair_warp(d, da[pa] + k * step, db[order - pa] + k * (BMN ? 128 : 2), idesc,
                                            kb != c0 || order != kPlanes - 1 || pa != 0 || k != 0);
#pragma unroll
                for (int pl = 0; pl < kPlanes; ++pl) umma_commit_pair_warp(&empty[stage + pl], (uint16_t)0x3);
                stage += kPlanes;
                if (stage == kStages) {
                  stage = 0;
                  phase ^= 1;
                }
              }
              if (ok) umma_commit_pair_warp(&tfull[buf], (uint16_t)0x3);
            }
          }
        }
        if (!ok && lane == 0) {
          atomicOr(p.status, DEV_TIMEOUT);
          *abort_flag = 1;
        }
        umma_commit_pair_warp(mma_done, (uint16_t)0x1);   // no MMA may still run when tensor memory is released
        mbar_wait(mma_done, 0);
      }
    }
  } else {
    if constexpr (kRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3, half = (warp - kFirstEpi) >> 2;
    const uint32_t tempty0 = mapa_shared(smem_u32(tempty), 0);
    uint8_t* buf_s = sEpi + (warp - kFirstEpi) * kEpiStage;
    int acc = 0;
    bool stop = false;
    for (int i = 0, u; !stop && (u = walk.at(p, i)) >= 0; ++i) {
      const Unit t = unit_of(p, u);
      const Job& job = p.j[t.job];
      const int row = (t.m * 2 + rank) * kBM + quarter * 32 + lane;
      RowStats st{-INFINITY, 0.f, 0.f};
      RowGrad rg{};
      if constexpr (EPI == CE_BWD) rg = ce_bwd_row<SPLIT>(p, row, t.n0 == 0 && half == 0);
      int label = -1;
      if constexpr (EPI == CE_FWD) {
        if (row < job.M) {
          const long y = p.ep.labels[row];
          label = y >= 0 && y < p.ep.V ? (int)y : -1;
        }
      }
      for (int r = 0; r < t.nr && !stop; ++r) {
        const int col = (t.n0 + r) * kBN + half * (kBN / 2);
        const uint32_t tl = tmem_base + ((uint32_t)(quarter * 32) << 16);
        float v[kRegs ? 128 : 1];
        // waits for the accumulator of the next chunk; false: the kernel is winding down
        auto chunk_ready = [&](int buf) {
          const bool ok = mbar_wait(&tfull[buf], (acc >> 1) & 1);
          // tcgen05.ld is warp-collective: the stop decision is warp-uniform
          if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
            if (lane == 0) atomicOr(p.status, DEV_TIMEOUT);
            *abort_flag = 1;
            return false;
          }
          tc_fence_after();
          return true;
        };
        auto chunk_taken = [&](int buf) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + 8 * buf);
          ++acc;
        };
        // of this thread's 128 columns, where the c-th 32 start (gates: this half's 64 gate columns, then its 64 up columns)
        auto column = [&](int c) {
          return (uint32_t)(kGate ? half * 64 + (c & 1) * 32 + (c >> 1) * (kBN / 2) : half * (kBN / 2) + c * 32);
        };
        // what the epilogue reads from memory, on its way while the products run
        float warm = 0.f;
        if constexpr (EPI >= CE_FWD) {
          const int c = kGate ? (t.n0 + r) * (kBN / 2) + half * 64 + lane * 2 : col + lane * 4;
          const int at = min(c, job.N - 1);
          if (p.ep.bias != nullptr) warm = __ldg(p.ep.bias + at);
          if (kGate && p.ep.bias2 != nullptr) warm += __ldg(p.ep.bias2 + at);
        }
        if constexpr (kStageDh) {
          if (p.ep.dh_vec) fetch_dh<T>(p, buf_s, lane, (t.n0 + r) * (kBN / 2) + half * 64, row - lane);
        }
        if (!chunk_ready(acc & 1)) {
          stop = true;
          break;
        }
        asm volatile("" ::"f"(warm));
        if constexpr (kRegs) {
          {
            const uint32_t tb = tl + (acc & 1) * kBN;
            uint32_t w[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tb + column(c), w[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 32; ++j) v[c * 32 + j] = __uint_as_float(w[c][j]);
            chunk_taken(acc & 1);
          }
#pragma unroll 1
          for (int c0 = t.kb0 + p.kb_chunk; c0 < t.kb1; c0 += p.kb_chunk) {
            if (!chunk_ready(acc & 1)) {
              stop = true;
              break;
            }
            const uint32_t tb = tl + (acc & 1) * kBN;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[32];
              tmem_ld32(tb + column(c), w);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; j += 2)
                add2f(v[c * 32 + j], v[c * 32 + j + 1], __uint_as_float(w[j]), __uint_as_float(w[j + 1]));
            }
            chunk_taken(acc & 1);
          }
        } else {
          const int buf = acc & 1;
          const uint32_t tb = tl + buf * kBN;
          if (job.out == STORE)
            store_tile<T>(job, &job.c[t.z], tb + half * (kBN / 2), row - lane, col, buf_s, lane);
          else
            slab_tile(job, &job.c[t.z], tb + half * (kBN / 2), row - lane + t.split * job.slab_rows, col, buf_s, lane,
                      job.out == F32_ADD);
          chunk_taken(buf);
        }
        if constexpr (kRegs) {
          if (stop) break;
          if constexpr (EPI == CE_FWD) {
            if (p.ep.part_sum != nullptr) ce_fwd_tile<true>(p, v, row, col, lane, label, st);
            else ce_fwd_tile<false>(p, v, row, col, lane, label, st);
          } else if constexpr (EPI == CE_BWD) {
            ce_bwd_tile<T, SPLIT>(p, v, rg, row, col, buf_s, lane);
          } else if constexpr (kGate) {
            const int oc = (t.n0 + r) * (kBN / 2) + half * 64;
            if (p.ep.act == ACT_SILU) gate_tile<T, SPLIT, ACT_SILU, EPI == GATE_BWD>(p, v, row, oc, buf_s, lane);
            else gate_tile<T, SPLIT, ACT_GELU, EPI == GATE_BWD>(p, v, row, oc, buf_s, lane);
          } else {
            slab_regs(job, &job.c[t.z], v, row - lane + t.split * job.slab_rows, col, buf_s, lane, job.out == F32_ADD);
          }
        }
      }
      if constexpr (EPI == CE_FWD) {
        if (!stop && row < job.M) {
          const size_t i = (size_t)(t.run_index * 2 + half) * job.M + row;
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
template <typename T, bool SPLIT, int EPI>
cudaError_t launch(const Params& p, int num_sms, cudaStream_t s) {
  auto kern = train_gemm_kernel<T, SPLIT, EPI>;
  using S = Shape<SPLIT, EPI>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
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
    if constexpr (S::kRegs) {
      // setmaxnreg.inc waits for registers of the block's launch allocation: refuse to launch when that is short
      cudaFuncAttributes fa;
      r = cudaFuncGetAttributes(&fa, kern);
      if (r != cudaSuccess) return r;
      if (fa.numRegs * S::kThreads < 128 * kRegsControl + 256 * kRegsEpi) return cudaErrorInvalidConfiguration;
    }
    int resident = num_sms / 2, n = 0;
    cudaLaunchConfig_t probe = cfg;
    probe.gridDim = dim3(2 * (num_sms / 2));
    if (cudaOccupancyMaxActiveClusters(&n, kern, &probe) == cudaSuccess && n >= 1) resident = n;
    resident_on[d] = resident;
    return cudaSuccess;
  }, &dev);
  if (e != cudaSuccess) return e;
  const long units = (long)p.units[0] + p.units[1];
  if (p.units[0] < 1 || p.units[1] < 0 || units > 0x7fffffffl - 4096) return cudaErrorInvalidValue;
  const int clusters = units < resident_on[dev] ? (int)units : resident_on[dev];
  cfg.gridDim = dim3(2 * clusters);
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace tg
}  // namespace jepa

// The instantiations for one operand type; each has its own translation unit.
#define JEPA_TRAIN_GEMM_INSTANCES(T, SPLIT, NAME)                              \
  namespace jepa {                                                             \
  namespace tg {                                                               \
  cudaError_t NAME(int epi, const Params& p, int num_sms, cudaStream_t s) {    \
    switch (epi) {                                                             \
      case REDUCE: return launch<T, SPLIT, REDUCE>(p, num_sms, s);             \
      case CE_FWD: return launch<T, SPLIT, CE_FWD>(p, num_sms, s);             \
      case CE_BWD: return launch<T, SPLIT, CE_BWD>(p, num_sms, s);             \
      case GATE_FWD: return launch<T, SPLIT, GATE_FWD>(p, num_sms, s);         \
      case GATE_BWD: return launch<T, SPLIT, GATE_BWD>(p, num_sms, s);         \
    }                                                                          \
    return cudaErrorInvalidValue;                                              \
  }                                                                            \
  }                                                                            \
  }
