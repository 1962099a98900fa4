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
// The tensor core truncates at every step of 16 k, so that a sum of products of
// one sign ends too small: by up to 2^-23 of itself a step (measured, all
// products positive: fp16 2.7 2^-23 after 4 steps, 27 after 32, 0.85 a step from
// 256 steps on; bf16, whose products are shorter, up to 9.6 after 32, 0.86 a step
// from 1000 on; logits of products of both signs over 1024 k, bf16: 12.6 after
// 64).  Epilogues whose results are fp32 therefore take the accumulator out every few
// blocks (kb_chunk) and add the pieces in registers, with rounding; SPLIT does so
// every block, with the products of the small planes first, whose steps then
// truncate a small accumulator.  16-bit results keep sums in it as long as the
// loss is below half a rounding of theirs: 2048 steps in fp16, 16384 in bf16
// (long_blocks); REDUCE adds the pieces of longer ones in memory.  The logits
// of the distillation are also given back what a piece loses on average
// (logit_loss).
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
//
// What bounds it, on large bf16 products: the tensor pipe in the forward passes
// (gates 16384 x 1024 x 2736 twice: 100 us, pipe busy 92% of the time; cross
// entropy 8192 x 2048 x 131072: 2.55 ms, 1.72 PFLOP/s, at the power cap, 2.30 ms
// below it); the epilogue's latency in the backward ones (CE_BWD of 1999 x 768 x
// 50021: 116 us, pipe 62%; GATE_BWD of 16384 x 1024 x 2736: 124 us, 72%); operand
// delivery in REDUCE (64 k take 640 to 710 clocks against the forward passes' 526;
// pipe 74 to 77%).
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
  GATE_BWD = 4,  // dg, du (T, or planes)
  DISTILL_FWD = 5,   // CE_FWD of z / temperature, without a label
  DISTILL_BWD = 6    // CE_BWD of z / temperature, without a label: the teacher's entries are put in afterwards
};
__host__ __device__ constexpr bool ce_fwd(int epi) { return epi == CE_FWD || epi == DISTILL_FWD; }
__host__ __device__ constexpr bool ce_bwd(int epi) { return epi == CE_BWD || epi == DISTILL_BWD; }
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
  float* dz_scale;         // CE_BWD, 16-bit: [0] what dloss is divided by, [1] what brings products of dz back
  float dz_factor;         // CE_BWD, 16-bit: the factor of every dz
  int dz_inline;           // dz_scale is computed here, and written for the kernels that follow
  float smoothing;
  float z_scale;           // DISTILL: log2 e / temperature
  float z_loss;            // DISTILL, 16-bit: the part of acc that the accumulator's truncation takes off it
  const uint32_t* hits;    // DISTILL_FWD: [M][top] a row's wanted columns (Hits)
  const uint16_t* starts;  // DISTILL_FWD: [M][2][runs + 1] where those of a half and a run begin
  float* hit_z;            // DISTILL_FWD: [M][top] where their z go
  int top, runs;
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
  int kb_chunk;          // blocks accumulated in tensor memory before the epilogue takes them (STORE: all of a unit's)
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
  template <int EPI>
  __device__ __forceinline__ int at(const Params& p, int i) const {
    if constexpr (ce_bwd(EPI) || EPI == GATE_BWD) {   // one job (so have the forward passes, but they then spill 1 KB)
      const int k = i * nc + cid;
      return k < p.units[0] ? k : -1;
    }
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
template <int EPI>
__device__ __forceinline__ Unit unit_of(const Params& p, int u) {
  // dividing is what takes time here: only CE_FWD has longer runs, only REDUCE has two jobs and splits, and most groups
  // of row tiles are full
  Unit t{};
  if constexpr (EPI == REDUCE) {
    t.job = u >= p.units[0] ? 1 : 0;
    if (t.job) u -= p.units[0];
  }
  const Job& j = p.j[t.job];
  const int runs = ce_fwd(EPI) ? (j.num_n + p.run - 1) / p.run : j.num_n;
  t.kb1 = j.kb_seg * j.nseg;
  if constexpr (EPI == REDUCE) {
    const int tiles = j.num_m * runs;
    const int q = u / tiles;
    u -= q * tiles;
    t.split = q / j.nz;
    t.z = q - t.split * j.nz;
    t.kb0 = t.split * j.kb_split;
    t.kb1 = min(t.kb0 + j.kb_split, t.kb1);
  }
  const int group = kGroupM * runs;
  const int gi = (int)((unsigned)u / (unsigned)group), w = u - gi * group;
  const int gm = min(j.num_m - gi * kGroupM, kGroupM);
  t.run_index = gm == kGroupM ? w / kGroupM : w / gm;
  t.m = gi * kGroupM + (w - t.run_index * gm);
  t.n0 = ce_fwd(EPI) ? t.run_index * p.run : t.run_index;
  t.nr = ce_fwd(EPI) ? min(p.run, j.num_n - t.n0) : 1;
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

// Tensor memory is handed back to the issuing warp in the order that the PTX ISA
// gives for it: tcgen05.wait::ld, tcgen05.fence::before_thread_sync, an arrival;
// then a wait, tcgen05.fence::after_thread_sync, tcgen05.mma.  It is the fences
// that order the accesses to tensor memory, so the arrival and the wait are
// relaxed, both at cluster scope, for half of the arrivals come from the other
// CTA.  No other memory is passed on, and a release would wait for the warp's
// stores (cross entropy backward, 4096 x 1024 x 32768 in fp16 537 us instead of
// 512, 1999 x 768 x 50021 in bf16 329 instead of 314).
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// mbar_wait for such arrivals.
__device__ __forceinline__ bool mbar_wait_cluster_relaxed(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  auto arrived = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (arrived()) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (arrived()) return true;
    if ((unsigned long long)(clock64() - t0) > 2ull * kWaitLimitNs) return false;
  }
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
// (a, b) = (a, b) m + (x, y)
__device__ __forceinline__ void fma2(float& a, float& b, float m, float x, float y) {
  uint64_t p, q, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(q) : "f"(m));
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(p) : "l"(q), "l"(r));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
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

// The backward epilogues (CE_BWD, GATE_BWD) hold their 32 rows x 2 x 64 columns
// in 8 x 8 blocks, as stmatrix and ldmatrix do: v[32 c + 4 g + e] with c = 2 h +
// q is row 16 h + 8 (e / 2) + lane / 4, column 8 g + 2 (lane % 4) + e % 2 of the
// q-th 64 columns.  Four rows of a column are in one thread and eight threads
// share it, so that column sums cost 28 shuffles instead of a pass of fp32
// values through shared memory, whose bandwidth the main loop needs (a row a
// thread: dg and du of 16384 x 1024 x 2736 with their sums 170 us instead of
// 131).
__device__ __forceinline__ void tmem_ld_blocks(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Where the pair of columns of block g and the rows lane / 4 + 8 i lies in v.
__device__ __forceinline__ constexpr int block_at(int q, int g, int i) { return (2 * (i >> 1) + q) * 32 + g * 4 + (i & 1) * 2; }

__device__ __forceinline__ void stmatrix4(uint8_t* row, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(row)), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4(const uint8_t* row, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(row))
               : "memory");
}

// The biases of 64 columns at this thread's (0 past the last), loaded at once.
struct Biases {
  float2 b[8];   // [g]
};
__device__ __forceinline__ void load_biases(Biases& t, const float* bias, int col, int n, int lane) {
  const int c = col + 2 * (lane & 3);
  if (bias != nullptr && col + 64 <= n && (reinterpret_cast<uintptr_t>(bias) & 7) == 0) {
#pragma unroll
    for (int g = 0; g < 8; ++g) t.b[g] = __ldg(reinterpret_cast<const float2*>(bias + c + 8 * g));
  } else {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int k = c + 8 * g;
      t.b[g].x = bias != nullptr && k < n ? __ldg(bias + k) : 0.f;
      t.b[g].y = bias != nullptr && k + 1 < n ? __ldg(bias + k + 1) : 0.f;
    }
  }
}

// This thread's part of the column sums of block column (q, g): its four rows.
__device__ __forceinline__ void sum_rows(const float (&v)[128], int q, int g, float& s0, float& s1) {
  const int a = block_at(q, g, 0), b = block_at(q, g, 1), c = block_at(q, g, 2), d = block_at(q, g, 3);
  s0 = v[a];
  s1 = v[a + 1];
  add2f(s0, s1, v[b], v[b + 1]);
  float t0 = v[c], t1 = v[c + 1];
  add2f(t0, t1, v[d], v[d + 1]);
  add2f(s0, s1, t0, t1);
}
// The sums s[2 g + e % 2] of 64 columns over the eight threads of each: a step
// hands over half of what is left.  fold_sums leaves the four of blocks g / 2 =
// (lane & 12) / 4, over half the threads; join_sums joins those of q = 0 (to
// part0, columns below n0) and of q = 1 (to part1, columns below n1).
__device__ __forceinline__ void fold_sums(float (&s)[16], int lane) {
#pragma unroll
  for (int half = 8; half >= 4; half >>= 1) {
    const bool up = (lane & half) != 0;
#pragma unroll
    for (int j = 0; j < half; ++j) {
      const float keep = up ? s[half + j] : s[j], give = up ? s[j] : s[half + j];
      s[j] = keep + __shfl_xor_sync(0xffffffffu, give, half);
    }
  }
}
__device__ __forceinline__ void join_sums(const float (&s0)[16], const float (&s1)[16], int lane, float* part0, int n0,
                                          float* part1, int n1) {
  const bool up = (lane & 16) != 0;
  float s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] = (up ? s1[j] : s0[j]) + __shfl_xor_sync(0xffffffffu, up ? s0[j] : s1[j], 16);
  float* part = up ? part1 : part0;
  const int n = up ? n1 : n0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = ((lane & 12) << 2) + 8 * j + 2 * (lane & 3);
    if (c + 1 < n) *reinterpret_cast<float2*>(part + c) = make_float2(s[2 * j], s[2 * j + 1]);
    else if (c < n) part[c] = s[2 * j];
  }
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

// The q-th 64 columns of an intermediate operand (dz, dg, du): the type's
// rounding, or three bf16 planes, each the rounding of what the ones before
// leave (v is used up).
template <typename T, bool SPLIT>
__device__ __forceinline__ void emit_operand(const Params& p, const CUtensorMap* c, float (&v)[128], int q,
                                             uint8_t* buf, int lane, int x, int y) {
#pragma unroll
  for (int pl = 0; pl < (SPLIT ? 3 : 1); ++pl) {
    if (lane == 0) bulk_wait_read_all();   // the previous store has read the buffer
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = block_at(q, g, i);
        w[i] = pack2<T>(v[at], v[at + 1]);
        if (SPLIT && pl < 2) {
          v[at] -= DT<T>::to(DT<T>::from(v[at]));
          v[at + 1] -= DT<T>::to(DT<T>::from(v[at + 1]));
        }
      }
      stmatrix4(buf + lane * 128 + ((g ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(c, buf, x, y + pl * p.c_plane);
      bulk_commit_group();
    }
  }
}

// Gate and its slope.  silu: a = g s, a' = s (1 + g (1 - s)) with s = 1 / (1 +
// 2^(-g log2 e)); gelu: a = g Phi(g), a' = Phi(g) + g phi(g).
//
// Phi(-x), x >= 0, is e^(-x^2 / 2) t P(t) with t = 1 / (1 + 11/32 x): t P(t) =
// e^(x^2 / 2) Phi(-x) is smooth, and a minimax fit of degree 8 over 0 <= x <= 14
// has a relative error of 2.2e-8.  So gates far on the negative side keep their
// relative accuracy (1/2 + erf(g / sqrt 2) / 2 cancels there: 4 % off at g = -5, 0
// from -6 on), and the exponential serves phi too.  16384 x 1024 x 2736 in bf16:
// 120-128 us, backward 400; through erff 119-125 and 414, through erfcf 151 and
// 503.
template <int ACT, bool GRAD>
__device__ __forceinline__ void gate(float g, float& a, float& da) {
  if constexpr (ACT == ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + ex2(-g * kLog2e));
    a = g * s;
    if constexpr (GRAD) da = s * fmaf(g, 1.0f - s, 1.0f);
  } else {
    const float e = ex2(g * g * (-0.5f * kLog2e));
    const float t = __fdividef(1.0f, fmaf(0.34375f, fabsf(g), 1.0f));
    float q = fmaf(-0x1.c7a0b8p-6f, t, 0x1.269a58p-3f);
    q = fmaf(q, t, -0x1.163c2ap-2f);
    q = fmaf(q, t, 0x1.870184p-3f);
    q = fmaf(q, t, -0x1.4201p-5f);
    q = fmaf(q, t, 0x1.cd7274p-4f);
    q = fmaf(q, t, 0x1.de2b3ep-4f);
    q = fmaf(q, t, 0x1.19afc4p-3f);
    q = fmaf(q, t, 0x1.18d232p-3f);
    const float tail = e * t * q, cdf = g < 0.f ? tail : 1.0f - tail;
    a = g * cdf;
    if constexpr (GRAD) da = fmaf(g * 0.3989422804014327f, e, cdf);
  }
}

// Statistics a thread carries over a run of the cross entropy: its row's max
// and sum of powers in base 2 (z log2 e), and the sum of z.
struct RowStats {
  float m, s, sum;
};

// The columns of a row whose z are wanted are sorted by hit_key: those of the left
// halves of the tiles, then those of the right ones, each in the order in which the
// threads of a half meet them.  A word of them has the column in its run (at most
// 16 tiles), and where the z goes.  starts has, for a row and a half, where the
// columns of each run begin.  A thread's first kHeld of a run are copied into its
// warp's staging buffer while the products run: a load that a lane waits for would
// hold up all of them.
constexpr int kHeld = 32;
__host__ __device__ constexpr uint32_t hit_key(uint32_t col) { return (col >> 7 & 1) << 31 | col; }   // col < 2^24 + 2^12
__host__ __device__ constexpr uint32_t hit_word(uint32_t col, uint32_t place) { return col << 10 | place; }
struct Hits {
  const uint32_t *at, *held;   // the row's, and its first ones in the buffer
  int i, n;
  uint32_t next;
  __device__ __forceinline__ void load() {
    next = ~0u;
    if (i < n) next = i < kHeld ? held[i * 32] : __ldg(at + i);
  }
};
__device__ __forceinline__ void find_hits(Hits& h, const EpiArgs& ep, int row, bool in, int half, int run_index, uint8_t* buf,
                                          int lane) {
  const uint16_t* first = ep.starts + ((size_t)row * 2 + half) * (ep.runs + 1) + run_index;
  const int lo = in ? first[0] : 0;
  h.i = 0;
  h.n = in ? first[1] - lo : 0;
  h.at = ep.hits + (size_t)row * ep.top + lo;
  uint32_t* held = reinterpret_cast<uint32_t*>(buf) + lane;
  h.held = held;
  __syncwarp();
#pragma unroll 1
  for (int k = 0; k < kHeld && __any_sync(0xffffffffu, k < h.n); ++k)
    if (k < h.n) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(held + k * 32)), "l"(h.at + k) : "memory");
}
// Before the first of them is looked at.
__device__ __forceinline__ void wait_hits(Hits& h) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  h.load();
}
// v[i] of a thread's own i.
__device__ __forceinline__ float pick(const float* v, int i) {
  float t[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) t[j] = i & 1 ? v[2 * j + 1] : v[2 * j];
#pragma unroll
  for (int b = 1; b < 5; ++b)
#pragma unroll
    for (int j = 0; j < 16 >> b; ++j) t[j] = i >> b & 1 ? t[2 * j + 1] : t[2 * j];
  return t[0];
}

template <bool SUM, bool DISTILL = false, bool SPLIT = false>
__device__ __forceinline__ void ce_fwd_tile(const Params& p, float (&v)[128], int row, int col0, int lane, int label,
                                            RowStats& st, Hits& hits, int run_col) {
  const EpiArgs& ep = p.ep;
  const float scale = DISTILL ? ep.z_scale : kLog2e;
  const int ly = label - col0;
  if (!DISTILL && ly >= 0 && ly < 128) {
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
    if constexpr (DISTILL && !SPLIT) {   // planes lose nothing that is given back; 0 times an infinite sum would be NaN
#pragma unroll
      for (int j = 0; j < 32; j += 2) fma2(w[j], w[j + 1], ep.z_loss, w[j], w[j + 1]);
    }
    if (ep.bias != nullptr) {
      add_bias(ep.bias, col, p.j[0].N, -INFINITY, w);
    } else if (col + 32 > p.j[0].N) {
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = col + j < p.j[0].N ? w[j] : -INFINITY;
    }
    if constexpr (DISTILL) {   // the lanes' wanted columns among these 32, one of each lane at a time
      const uint32_t end = hit_word(run_col + c * 32 + 32, 0);
      while (true) {
        const bool mine = hits.next < end;
        if (!__any_sync(0xffffffffu, mine)) break;
        const float z = pick(w, (int)(hits.next >> 10) & 31);
        if (mine) {
          ep.hit_z[(size_t)row * ep.top + hits.next % 1024] = z;
          ++hits.i;
          hits.load();
        }
      }
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
    const float m = fmaxf(st.m, max3(m0, m1, fmaxf(w[30], w[31])) * scale);
    const float ref = m == -INFINITY ? 0.f : m;   // nothing but -inf so far: every power is 0
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      fma2(w[j], w[j + 1], scale, -ref);
      fma2(w[j + 2], w[j + 3], scale, -ref);
      add2f(s0, s1, ex2(w[j]), ex2(w[j + 1]));
      add2f(s2, s3, ex2(w[j + 2]), ex2(w[j + 3]));
    }
    st.s = fmaf(st.s, ex2(st.m - ref), (s0 + s1) + (s2 + s3));
    st.m = m;
  }
}

// What the cross entropy's gradient needs of a thread's four rows, row0 + lane / 4
// + 8 i.  A row that takes no part (past M, ignored, bad label) gets zeros.
struct RowGrads {
  float l2[4], g[4];   // lse in base 2, the row's factor
  int label[4];        // the label's column of this piece, if it lies in it
  int part;            // bit i: the row takes part
};
struct RowLoads {
  long y[4];
  float lse[4], dl[4];
};
__device__ __forceinline__ void load_rows(RowLoads& r, const Params& p, int row0, int lane) {
  const EpiArgs& ep = p.ep;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = min(row0 + (lane >> 2) + 8 * i, p.j[0].M - 1);
    r.y[i] = __ldg(reinterpret_cast<const long long*>(ep.labels) + row);
    r.lse[i] = __ldg(ep.lse + row);
    r.dl[i] = __ldg(ep.dloss + row);
  }
}
template <bool SPLIT>
__device__ __forceinline__ RowGrads ce_bwd_rows(const RowLoads& l, const Params& p, float unit, int row0, int lane, bool report) {
  RowGrads r;
  r.part = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool in = row0 + (lane >> 2) + 8 * i < p.j[0].M && l.y[i] != p.ep.ignore_index;
    const bool part = in && l.y[i] >= 0 && l.y[i] < p.ep.V;
    r.part |= part ? 1 << i : 0;
    r.label[i] = part ? (int)l.y[i] - p.ep.v0 : -1;
    r.l2[i] = part ? l.lse[i] * kLog2e : 0.f;
    r.g[i] = part ? (SPLIT ? l.dl[i] : l.dl[i] / unit * p.ep.dz_factor) : 0.f;
    if (in && !part && report) atomicOr(p.status, DEV_BAD_INDEX);
  }
  return r;
}

// max |dloss| over the rows that have a gradient, of this thread's of `threads`.
// A dloss that is not finite makes its own row's dz so, and leaves the unit to
// the others.
__device__ __forceinline__ float dz_max(const float* dloss, const int64_t* labels, long ignore_index, int M, int V,
                                        int thread, int threads) {
  float m = 0.f;
  for (int i0 = thread; i0 < M; i0 += 8 * threads) {
    long label[8];
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {   // past M: again the last row
      const int i = min(i0 + j * threads, M - 1);
      label[j] = __ldg(reinterpret_cast<const long long*>(labels) + i);
      d[j] = __ldg(dloss + i);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (label[j] != ignore_index && label[j] >= 0 && label[j] < V && fabsf(d[j]) < INFINITY) m = fmaxf(m, fabsf(d[j]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// What dz is held in units of, from the maximum over all rows: that, or 1 if it
// is 0.
__device__ __forceinline__ float dz_unit(float m, float factor, float smoothing, float* scale) {
  if (!(m > 0.f)) m = 1.f;
  if (scale != nullptr) {
    scale[0] = m;
    scale[1] = m * (1.0f - smoothing) / factor;
  }
  return m;
}
// The same by the eight epilogue warps of every CTA, through their staging
// buffers, while the first products run.
__device__ __forceinline__ float dz_unit_inline(const Params& p, uint8_t* stage, int warp, int lane) {
  const EpiArgs& ep = p.ep;
  float m = dz_max(ep.dloss, ep.labels, ep.ignore_index, p.j[0].M, ep.V, warp * 32 + lane, 32 * kEpiWarps);
  if (lane == 0) *reinterpret_cast<float*>(stage + warp * kEpiStage) = m;
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
  for (int k = 0; k < kEpiWarps; ++k) m = fmaxf(m, *reinterpret_cast<const float*>(stage + k * kEpiStage));
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");   // read before a buffer is used
  return dz_unit(m, ep.dz_factor, ep.smoothing, blockIdx.x == 0 && warp == 0 && lane == 0 ? ep.dz_scale : nullptr);
}

// Asks for what the epilogue of a pair's next tile reads: the lines of 32 rows'
// labels, lse and dloss, of dh, and of the biases.
__device__ __forceinline__ void prefetch_l1(const void* q) { asm volatile("prefetch.global.L1 [%0];" ::"l"(q)); }
__device__ __forceinline__ void prefetch_l2(const void* q) { asm volatile("prefetch.global.L2 [%0];" ::"l"(q)); }
template <typename T, bool SPLIT, int EPI>
__device__ __forceinline__ void prefetch_tile(const Params& p, int row0, int col, int lane) {
  const EpiArgs& ep = p.ep;
  const int row = min(row0 + lane, p.j[0].M - 1), N = p.j[0].N;
  if constexpr (ce_bwd(EPI)) {
    if ((lane & 15) == 0) prefetch_l1(ep.labels + row);
    if (lane == 0) prefetch_l1(ep.lse + row);
    if (lane == 0) prefetch_l1(ep.dloss + row);
    if (ep.bias != nullptr && lane < 4) prefetch_l1(ep.bias + min(col + 32 * lane, N - 1));
  } else {
    if (ep.bias != nullptr && lane < 2) prefetch_l1(ep.bias + min(col + 32 * lane, N - 1));
    if (ep.bias2 != nullptr && lane < 2) prefetch_l1(ep.bias2 + min(col + 32 * lane, N - 1));
    using TD = typename std::conditional<SPLIT, float, T>::type;
    const TD* dh = static_cast<const TD*>(ep.dh) + (size_t)row * N;
    prefetch_l2(dh + min(col, N - 1));
    prefetch_l2(dh + min(col + 63, N - 1));
  }
}

template <typename T, bool SPLIT, bool DISTILL = false>
__device__ __forceinline__ void ce_bwd_tile(const Params& p, float (&v)[128], const RowGrads& rg, Biases& bias,
                                            int row0, int col0, uint8_t* buf, int lane) {
  const EpiArgs& ep = p.ep;
  const int N = p.j[0].N;
  // 16-bit dz is held as g ((p - e / V) / (1 - e) - [v = y]) with g = dloss / max |dloss| (times a power of 2 in fp16): with one
  // dloss for all rows, as a mean's, the label's entry is then near -1, which 16 bits hold exactly.  (As dloss (p - (1 - e)
  // [v = y] - e / V) those entries, which make up most of dx and dW, were all off by the same rounding of dloss: dx and
  // dW 3.0e-3 from the exact gradients in norm instead of 1.7e-3 at 1999 x 768 x 50021 in bf16.)
  const float uni = ep.smoothing / (float)ep.V;
  const float cs = SPLIT ? 1.0f : 1.0f / (1.0f - ep.smoothing), hit = SPLIT ? 1.0f - ep.smoothing : 1.0f;
  const float scale = DISTILL ? ep.z_scale : kLog2e;
  const int lc = 2 * (lane & 3);
  const bool whole = __all_sync(0xffffffffu, rg.part == 15);
  float s[2][16] = {};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int cc = col0 + q * 64;
    if (cc >= N) continue;
    // columns past N keep finite values: nothing reads them
#pragma unroll
    for (int g = 0; g < 8; ++g) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& z0 = v[block_at(q, g, i)];
        float& z1 = v[block_at(q, g, i) + 1];
        if constexpr (DISTILL && !SPLIT) {   // as in ce_fwd_tile
          float t0 = z0, t1 = z1;
          add2f(t0, t1, bias.b[g].x, bias.b[g].y);
          fma2(z0, z1, ep.z_loss, t0, t1);
        } else {
          add2f(z0, z1, bias.b[g].x, bias.b[g].y);
        }
        fma2(z0, z1, scale, -rg.l2[i]);
        z0 = ex2(z0);
        z1 = ex2(z1);
        if (!DISTILL && ep.smoothing > 0.f) fma2(z0, z1, cs, -uni * cs);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ly = rg.label[i] - cc;
      if (!DISTILL && __any_sync(0xffffffffu, ly >= 0 && ly < 64)) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const int at = block_at(q, g, i);
          v[at] -= ly == 8 * g + lc ? hit : 0.f;
          v[at + 1] -= ly == 8 * g + lc + 1 ? hit : 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < 8; ++g) mul2(v[block_at(q, g, i)], v[block_at(q, g, i) + 1], rg.g[i]);
    if (!whole) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool part = (rg.part >> i & 1) != 0;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          float& z0 = v[block_at(q, g, i)];
          float& z1 = v[block_at(q, g, i) + 1];
          z0 = part ? z0 : 0.f;
          z1 = part ? z1 : 0.f;
        }
      }
    }
    if (q == 0) load_biases(bias, ep.bias, cc + 64, N, lane);
    if (ep.col_part != nullptr) {
#pragma unroll
      for (int g = 0; g < 8; ++g) sum_rows(v, q, g, s[q][2 * g], s[q][2 * g + 1]);
      fold_sums(s[q], lane);
    }
    emit_operand<T, SPLIT>(p, &p.j[0].c[0], v, q, buf, lane, cc, row0);
  }
  if (ep.col_part != nullptr) {
    float* part = ep.col_part + (size_t)(row0 >> 5) * ep.ld_col + col0;
    const int n = row0 < p.j[0].M ? N - col0 : 0;
    join_sums(s[0], s[1], lane, part, n, part + 64, n - 64);
  }
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

// 64 columns of h from the gates v[0 .. 63] and the ups v[64 .. 127] of a row.
template <typename T, bool SPLIT, int ACT>
__device__ __forceinline__ void gate_fwd_tile(const Params& p, float (&v)[128], int row, int col, uint8_t* buf, int lane) {
  const EpiArgs& ep = p.ep;
  if (col >= p.j[0].N) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int cc = col + h * 32;
    float* g = v + h * 32;
    float* u = v + 64 + h * 32;
    if (ep.bias != nullptr) add_bias(ep.bias, cc, p.j[0].N, 0.f, g);
    if (ep.bias2 != nullptr) add_bias(ep.bias2, cc, p.j[0].N, 0.f, u);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float a, da;
      gate<ACT, false>(g[j], a, da);
      g[j] = a * u[j];
    }
  }
  if constexpr (!SPLIT) {
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

// dg and du of 64 columns: gates are the blocks of q = 0, ups those of q = 1.
template <typename T, bool SPLIT, int ACT>
__device__ __forceinline__ void gate_bwd_tile(const Params& p, float (&v)[128], const Biases (&bias)[2], int row0, int col, uint8_t* buf,
                                              int lane) {
  using TD = typename std::conditional<SPLIT, float, T>::type;   // the operator's type
  const EpiArgs& ep = p.ep;
  const int M = p.j[0].M, N = p.j[0].N;
  if constexpr (!SPLIT) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");   // fetch_dh's
    __syncwarp();
  }
  if (col >= N) return;
  const int lc = 2 * (lane & 3), row = row0 + (lane >> 2);
  const TD* dh = static_cast<const TD*>(ep.dh) + (size_t)row * N + col + lc;
  float s[2][16] = {};
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const int left = N - (col + 8 * g + lc);   // columns from this thread's first on
    float2 d[4];
    if (!SPLIT && ep.dh_vec) {
      uint32_t w[4];
      ldmatrix4(buf + lane * 128 + ((g ^ (lane & 7)) << 4), w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        TD t[2];
        memcpy(t, &w[i], 4);   // of a 16-bit type
        d[i] = make_float2(DT<TD>::to(t[0]), DT<TD>::to(t[1]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const TD* q = dh + (size_t)(8 * i) * N + 8 * g;
        const bool in = row + 8 * i < M;
        if (SPLIT && ep.dh_vec)   // rows are multiples of 16 bytes: a pair is inside or outside as a whole
          d[i] = in && left > 0 ? __ldg(reinterpret_cast<const float2*>(q)) : make_float2(0.f, 0.f);
        else
          d[i] = make_float2(in && left > 0 ? DT<TD>::to(q[0]) : 0.f, in && left > 1 ? DT<TD>::to(q[1]) : 0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* vg = v + block_at(0, g, i);
      float* vu = v + block_at(1, g, i);
      add2f(vg[0], vg[1], bias[0].b[g].x, bias[0].b[g].y);
      add2f(vu[0], vu[1], bias[1].b[g].x, bias[1].b[g].y);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a, da;
        gate<ACT, true>(vg[e], a, da);
        const float dd = e == 0 ? d[i].x : d[i].y;
        vg[e] = dd * vu[e] * da;
        vu[e] = dd * a;
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) sum_rows(v, q, g, s[q][2 * g], s[q][2 * g + 1]);
  }
  __syncwarp();   // dh has been read from the staging buffer
#pragma unroll
  for (int q = 0; q < 2; ++q) emit_operand<T, SPLIT>(p, &p.j[0].c[q], v, q, buf, lane, col, row0);
  if (ep.col_part != nullptr || ep.col_part2 != nullptr) {
    const size_t at = (size_t)(row0 >> 5) * ep.ld_col + col;
    const int n = row0 < M ? N - col : 0;
    for (int q = 0; q < 2; ++q) fold_sums(s[q], lane);
    join_sums(s[0], s[1], lane, ep.col_part + at, ep.col_part != nullptr ? n : 0, ep.col_part2 + at,
              ep.col_part2 != nullptr ? n : 0);
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
        for (int i = 0, u; !stop && (u = walk.at<EPI>(p, i)) >= 0; ++i) {
          const Unit t = unit_of<EPI>(p, u);
          const Job& job = p.j[EPI == REDUCE ? t.job : 0];
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
        for (int i = 0, u; ok && (u = walk.at<EPI>(p, i)) >= 0; ++i) {
          const Unit t = unit_of<EPI>(p, u);
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
              if (!__all_sync(0xffffffffu, mbar_wait_cluster_relaxed(&tempty[buf], ((acc >> 1) & 1) ^ 1))) {
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
    [[maybe_unused]] float unit = 1.f;
    if constexpr (ce_bwd(EPI) && !SPLIT)
      unit = p.ep.dz_inline ? dz_unit_inline(p, sEpi, warp - kFirstEpi, lane) : __ldg(p.ep.dz_scale);
    int acc = 0;
    bool stop = false;
    int u = walk.at<EPI>(p, 0);
    for (int i = 1; !stop && u >= 0; ++i) {
      const Unit t = unit_of<EPI>(p, u);
      u = walk.at<EPI>(p, i);   // the next one
      const Job& job = p.j[EPI == REDUCE ? t.job : 0];
      const int row = (t.m * 2 + rank) * kBM + quarter * 32 + lane;
      RowStats st{-INFINITY, 0.f, 0.f};
      int label = -1;
      Hits hits{};
      if constexpr (EPI == DISTILL_FWD) find_hits(hits, p.ep, row, row < job.M, half, t.run_index, buf_s, lane);
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
          if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + 8 * buf);   // the even CTA's barrier
          ++acc;
        };
        // the c-th 32 values of this thread: of its row's 128 columns (gates: 64 gate columns, then the 64 up columns),
        // or blocks (block_at)
        auto load = [&](uint32_t tb, int c, uint32_t (&w)[32]) {
          if constexpr (ce_bwd(EPI) || EPI == GATE_BWD)
            tmem_ld_blocks(tb + ((uint32_t)(c >> 1) << 20) +
                               (EPI == GATE_BWD ? half * 64 + (c & 1) * (kBN / 2) : half * (kBN / 2) + (c & 1) * 64), w);
          else
            tmem_ld32(tb + (kGate ? half * 64 + (c & 1) * 32 + (c >> 1) * (kBN / 2) : half * (kBN / 2) + c * 32), w);
        };
        // what the epilogue reads from memory, on its way while the products run
        float warm = 0.f;
        [[maybe_unused]] RowLoads rows;
        [[maybe_unused]] Biases biases[EPI == GATE_BWD ? 2 : 1];
        if constexpr (ce_bwd(EPI)) {
          load_rows(rows, p, row - lane, lane);
          load_biases(biases[0], p.ep.bias, col, job.N, lane);
        } else if constexpr (EPI == GATE_BWD) {
          for (int q = 0; q < 2; ++q)
            load_biases(biases[q], q == 0 ? p.ep.bias : p.ep.bias2, (t.n0 + r) * (kBN / 2) + half * 64, job.N, lane);
        } else if constexpr (EPI >= CE_FWD) {
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
        [[maybe_unused]] RowGrads rg;
        if constexpr (ce_bwd(EPI)) rg = ce_bwd_rows<SPLIT>(rows, p, unit, row - lane, lane, t.n0 == 0 && half == 0);
        if constexpr (kRegs) {
          {
            const uint32_t tb = tl + (acc & 1) * kBN;
            uint32_t w[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) load(tb, c, w[c]);
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
              load(tb, c, w);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; j += 2)
                add2f(v[c * 32 + j], v[c * 32 + j + 1], __uint_as_float(w[j]), __uint_as_float(w[j + 1]));
            }
            chunk_taken(acc & 1);
          }
        } else {
          // a sum of several pieces (its C is fp32) adds those after the first to what this warp has stored
          bool add = job.out == F32_ADD;
#pragma unroll 1
          for (int c0 = t.kb0;;) {
            const int buf = acc & 1;
            const uint32_t tb = tl + buf * kBN;
            if (job.out == STORE)
              store_tile<T>(job, &job.c[t.z], tb + half * (kBN / 2), row - lane, col, buf_s, lane);
            else
              slab_tile(job, &job.c[t.z], tb + half * (kBN / 2), row - lane + t.split * job.slab_rows, col, buf_s, lane,
                        add);
            chunk_taken(buf);
            c0 += p.kb_chunk;
            if (c0 >= t.kb1) break;
            if (lane == 0) bulk_wait_all();   // the piece before is in memory
            if (!chunk_ready(acc & 1)) {
              stop = true;
              break;
            }
            add = true;
          }
        }
        if constexpr (kRegs) {
          if (stop) break;
          if constexpr (ce_bwd(EPI) || EPI == GATE_BWD) {
            if (u >= 0) {
              const Unit next = unit_of<EPI>(p, u);
              prefetch_tile<T, SPLIT, EPI>(p, (next.m * 2 + rank) * kBM + quarter * 32,
                                           ce_bwd(EPI) ? next.n0 * kBN + half * (kBN / 2) : next.n0 * (kBN / 2) + half * 64,
                                           lane);
            }
          }
          if constexpr (ce_fwd(EPI)) {
            if constexpr (EPI == DISTILL_FWD)
              if (r == 0) wait_hits(hits);
            if constexpr (EPI == DISTILL_FWD) ce_fwd_tile<false, true, SPLIT>(p, v, row, col, lane, label, st, hits, r * kBN + half * (kBN / 2));
            else if (p.ep.part_sum != nullptr) ce_fwd_tile<true>(p, v, row, col, lane, label, st, hits, r * kBN + half * (kBN / 2));
            else ce_fwd_tile<false>(p, v, row, col, lane, label, st, hits, r * kBN + half * (kBN / 2));
          } else if constexpr (ce_bwd(EPI)) {
            ce_bwd_tile<T, SPLIT, EPI == DISTILL_BWD>(p, v, rg, biases[0], row - lane, col, buf_s, lane);
          } else if constexpr (kGate) {
            const int oc = (t.n0 + r) * (kBN / 2) + half * 64;
            if constexpr (EPI == GATE_FWD) {
              if (p.ep.act == ACT_SILU) gate_fwd_tile<T, SPLIT, ACT_SILU>(p, v, row, oc, buf_s, lane);
              else gate_fwd_tile<T, SPLIT, ACT_GELU>(p, v, row, oc, buf_s, lane);
            } else {
              if (p.ep.act == ACT_SILU) gate_bwd_tile<T, SPLIT, ACT_SILU>(p, v, biases, row - lane, oc, buf_s, lane);
              else gate_bwd_tile<T, SPLIT, ACT_GELU>(p, v, biases, row - lane, oc, buf_s, lane);
            }
          } else {
            slab_regs(job, &job.c[t.z], v, row - lane + t.split * job.slab_rows, col, buf_s, lane, job.out == F32_ADD);
          }
        }
      }
      if constexpr (ce_fwd(EPI)) {
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
  if (p.units[0] < 1 || p.units[1] < 0 || units > 0x7fffffffl - 4096 || p.kb_chunk < 1) return cudaErrorInvalidValue;
  for (const Job& j : p.j)   // a STORE takes its whole sum from tensor memory
    if (EPI == REDUCE && !SPLIT && j.out == STORE && j.kb_split > p.kb_chunk) return cudaErrorInvalidValue;
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
      case DISTILL_FWD: return launch<T, SPLIT, DISTILL_FWD>(p, num_sms, s);   \
      case DISTILL_BWD: return launch<T, SPLIT, DISTILL_BWD>(p, num_sms, s);   \
    }                                                                          \
    return cudaErrorInvalidValue;                                              \
  }                                                                            \
  }                                                                            \
  }
