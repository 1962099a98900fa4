// The training operators: which products they launch, in which pieces, and the
// small kernels between them.
//
// fp32 matrices are split into three bf16 planes first; 16-bit ones whose rows
// are not multiples of 16 bytes are copied to rows that are (TMA addresses
// nothing else).  Everything else reads the caller's matrices in place.
#include <algorithm>
#include <cmath>

#include "gemm_train.cuh"
#include "row_stats.cuh"

namespace jepa {

namespace tg {
cudaError_t gemm_bf16(int epi, const Params& p, int num_sms, cudaStream_t s);
cudaError_t gemm_f16(int epi, const Params& p, int num_sms, cudaStream_t s);
cudaError_t gemm_f32(int epi, const Params& p, int num_sms, cudaStream_t s);
}  // namespace tg

namespace {

using tg::Job;
using tg::Params;

constexpr int kBlock = 256;
constexpr int kPairs = 76;      // CTA pairs of 152 SMs: the plans (and workspaces) assume it, the launch asks the device

#define JEPA_TRY_CUDA(expr)                 \
  do {                                      \
    const cudaError_t e_ = (expr);          \
    if (e_ != cudaSuccess) return e_;       \
  } while (0)

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }
int ceil_div(long a, long b) { return (int)((a + b - 1) / b); }
long round_up(long a, long b) { return (a + b - 1) / b * b; }
unsigned blocks_for(long n, int block) { return (unsigned)((n + block - 1) / block); }
size_t elem(int dtype) { return dtype == DTYPE_F32 ? 4 : 2; }
bool split(int dtype) { return dtype == DTYPE_F32; }

// A workspace cut into 256-byte aligned buffers; over a null base, its size.
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

// ----------------------------------------------------------------------------- operands
// A 16-bit matrix that TMA can address: rows x cols, row stride ld, and for
// fp32 three planes of it, plane_rows apart (0: one plane).
struct Mat {
  const uint8_t* p = nullptr;
  long rows = 0, cols = 0, ld = 0, plane_rows = 0;
  bool own = false;   // a copy in the workspace
};
// Where the operator's matrix is or will be: in place, or in the workspace.
Mat operand(int dtype, const void* src, long rows, long cols, Carver& cv) {
  Mat m;
  m.rows = rows;
  m.cols = cols;
  m.ld = round_up(cols, 8);
  m.own = split(dtype) || cols % 8 != 0;
  if (split(dtype)) m.plane_rows = round_up(rows, 64);
  m.p = m.own ? cv.take<uint8_t>(2 * (size_t)m.ld * (split(dtype) ? 3 * m.plane_rows : rows))
              : static_cast<const uint8_t*>(src);
  return m;
}
// Rows from r0 on.
Mat rows_from(const Mat& m, long r0, long rows) {
  Mat t = m;
  t.p += 2 * (size_t)r0 * m.ld;
  t.rows = rows;
  return t;
}

// The extent of the map's row dimension: a single plane ends at its rows (TMA
// reads zeros past them); planes run on, and a row past a plane's end is the
// zero padding or the next plane's, whose products are dropped or meet zeros.
long map_rows(const Mat& m, long r0) { return m.plane_rows != 0 ? 3 * m.plane_rows - r0 : m.rows; }
// m is [rows, k]: boxes of 64 k x 128 rows.  r0: how far m starts into its plane.
cudaError_t map_k(CUtensorMap* t, const Mat& m, long r0 = 0) {
  return make_tmap_2d(t, m.p, 2, m.cols, map_rows(m, r0), m.ld * 2, tg::kBK, tg::kBM);
}
// m is [k, rows]: boxes of 64 rows x 64 k.
cudaError_t map_mn(CUtensorMap* t, const Mat& m, long r0 = 0) {
  return make_tmap_2d(t, m.p, 2, m.cols, map_rows(m, r0), m.ld * 2, 64, tg::kBK);
}
// Outputs: 16-bit in blocks of 64 columns x 32 rows, fp32 of 32 x 32.
cudaError_t map_out16(CUtensorMap* t, void* p, long rows, long cols, long ld) {
  return make_tmap_2d(t, p, 2, cols, rows, ld * 2, 64, 32);
}
cudaError_t map_out32(CUtensorMap* t, void* p, long rows, long cols, long ld) {
  return make_tmap_2d(t, p, 4, cols, rows, ld * 4, 32, 32);
}

// Up to three matrices to be laid out at once (grid.y).
struct Fills {
  const void* src[3];
  uint16_t* dst[3];
  long rows[3], plane_rows[3];
  int cols[3], ld8[3];   // row length in the workspace, in 8 values
  int count;
};
// Rows to rows of 16 bytes.  8 columns a thread.
__global__ void __launch_bounds__(kBlock) pad_kernel(const __grid_constant__ Fills f) {
  const int y = blockIdx.y;
  const int cols = f.cols[y], ld8 = f.ld8[y];
  const uint16_t* src = static_cast<const uint16_t*>(f.src[y]);
  const long i = (long)blockIdx.x * kBlock + threadIdx.x;
  const long r = i / ld8;
  if (r >= f.rows[y]) return;
  const int c = (int)(i - r * ld8) * 8;
  uint16_t h[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) h[j] = c + j < cols ? __ldg(src + r * cols + c + j) : (uint16_t)0;
  uint4 q;
  memcpy(&q, h, 16);
  reinterpret_cast<uint4*>(f.dst[y])[i] = q;
}
// fp32 rows to three bf16 planes x = x0 + x1 + x2, each the rounding of what
// the ones before leave.  A finite value that rounds to infinity is truncated
// instead; one that is not finite has no further planes.  Padding is zero.
// 8 columns a thread.
__global__ void __launch_bounds__(kBlock) split_kernel(const __grid_constant__ Fills f) {
  const int y = blockIdx.y;
  const int cols = f.cols[y], ld8 = f.ld8[y];
  const long rows = f.rows[y], plane_rows = f.plane_rows[y];
  const long i = (long)blockIdx.x * kBlock + threadIdx.x;
  const long r = i / ld8;
  if (r >= plane_rows) return;
  const int c = (int)(i - r * ld8) * 8;
  float x[8];
  const float* p = static_cast<const float*>(f.src[y]) + r * cols + c;
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    if (cols % 4 == 0) {   // rows start on 16 bytes
      const float4 q = r < rows && c + j < cols ? __ldg(reinterpret_cast<const float4*>(p + j)) : make_float4(0, 0, 0, 0);
      x[j] = q.x; x[j + 1] = q.y; x[j + 2] = q.z; x[j + 3] = q.w;
    } else {
#pragma unroll
      for (int k = j; k < j + 4; ++k) x[k] = r < rows && c + k < cols ? __ldg(p + k) : 0.f;
    }
  }
  __nv_bfloat16 h[3][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h[0][j] = __float2bfloat16_rn(x[j]);
    if (fabsf(x[j]) > 3.3895e38f) h[0][j] = __float2bfloat16_rz(x[j]);
    float rem = x[j] - __bfloat162float(h[0][j]);
    if (!(fabsf(x[j]) < INFINITY)) rem = 0.f;
    h[1][j] = __float2bfloat16_rn(rem);
    h[2][j] = __float2bfloat16_rn(rem - __bfloat162float(h[1][j]));
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint4 q;
    memcpy(&q, h[k], 16);
    reinterpret_cast<uint4*>(f.dst[y])[k * plane_rows * ld8 + i] = q;
  }
}
// An operand that lives in the workspace is to be filled.
void add_fill(Fills& f, const void* src, const Mat& m) {
  if (!m.own) return;
  const int k = f.count++;
  f.src[k] = src;
  f.dst[k] = reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(m.p));
  f.rows[k] = m.rows;
  f.plane_rows[k] = m.plane_rows;
  f.cols[k] = (int)m.cols;
  f.ld8[k] = (int)(m.ld / 8);
}
cudaError_t fill(int dtype, const Fills& f, cudaStream_t s) {
  if (f.count == 0) return cudaSuccess;
  long most = 0;
  for (int k = 0; k < f.count; ++k) {
    const long n = (split(dtype) ? f.plane_rows[k] : f.rows[k]) * f.ld8[k];
    most = n > most ? n : most;
  }
  const dim3 g(blocks_for(most, kBlock), f.count);
  if (split(dtype)) split_kernel<<<g, kBlock, 0, s>>>(f);
  else pad_kernel<<<g, kBlock, 0, s>>>(f);
  return cudaGetLastError();
}

// ----------------------------------------------------------------------------- products
Job base_job(long M, long N, int cols_per_tile) {
  Job j{};
  j.M = (int)M;
  j.N = (int)N;
  j.num_m = ceil_div(M, 2 * tg::kBM);
  j.num_n = ceil_div(N, cols_per_tile);
  j.nseg = j.nz = j.splits = 1;
  return j;
}
void set_k(Job& j, long k_per_seg, int nseg, int splits) {
  j.kb_seg = ceil_div(k_per_seg, tg::kBK);
  j.nseg = nseg;
  const int total = j.kb_seg * nseg;
  j.kb_split = ceil_div(total, splits);
  j.splits = ceil_div(total, j.kb_split);
}
// A launch of one K-major product (the cross entropy's and the gates').
Params forward_params(const Job& j, int run, int* status) {
  Params p{};
  p.j[0] = j;
  p.run = run;
  const long units = (long)j.num_m * ceil_div(j.num_n, run);
  p.units[0] = units > 0x7fffffffl ? -1 : (int)units;   // launch refuses what it cannot count
  p.status = status;
  return p;
}

// The reducing products of a backward pass: outputs M x N of the operator's
// type, `nz` of them, each a sum over kb blocks of K (dx, and dW).
struct Product {
  long M, N;
  int nz, kb;
};
// How they are scheduled: the splits of K of each, which goes first, and the
// units of the second that fill the first one's last round.
struct PairPlan {
  int splits[2], first, extra;
};

// Time of one unit over `per` blocks in us: 0.34 us a block (256 x 256 x 64 on a
// CTA pair; 1.6 for planes), but at least an epilogue's, and a little to change
// over.
double unit_us(bool sp, int per) {
  const double t = per * (sp ? 1.6 : 0.34), epilogue = sp ? 2.5 : 2.0;
  return (t > epilogue ? t : epilogue) + 0.3;
}
// Rounds of the 76 pairs for n[0] units of c[0] us, then n[1] of c[1] (Walk's order).
double rounds_us(const long (&n)[2], const double (&c)[2], int* extra) {
  const long full = n[0] / kPairs, part = n[0] % kPairs, idle = kPairs - part;
  double best = 1e300;
  const int most = part == 0 ? 0 : (int)(c[0] / c[1]) + 1;
  for (int e = 0; e <= most; ++e) {
    const long taken = part == 0 ? 0 : (idle * e < n[1] ? idle * e : n[1]);
    const long rest = n[1] - taken;
    double t = full * c[0] + (taken + idle - 1) / idle * c[1] + (rest + kPairs - 1) / kPairs * c[1];
    if (part != 0) {
      const long busy = rest > idle ? (rest - idle + kPairs - 1) / kPairs : 0;
      const double u = (full + 1) * c[0] + busy * c[1];
      if (u > t) t = u;
    }
    if (t < best) {
      best = t;
      *extra = e;
    }
  }
  return best;
}
PairPlan search_plan(bool sp, const Product (&pr)[2]) {
  static const int kTry[] = {1, 2, 3, 4, 6, 8, 12, 16};
  const int least = sp ? 1 : 4;   // blocks of a split
  long tiles[2];
  for (int k = 0; k < 2; ++k) tiles[k] = (long)ceil_div(pr[k].M, 256) * ceil_div(pr[k].N, 256) * pr[k].nz;
  PairPlan best{};
  double best_t = 1e300;
  for (int s0 : kTry) {
    if (s0 > 1 && (pr[0].kb / s0 < least || tiles[0] > 4 * kPairs)) break;
    for (int s1 : kTry) {
      if (s1 > 1 && (pr[1].kb / s1 < least || tiles[1] > 4 * kPairs)) break;
      const int want[2] = {s0, s1};
      int real[2];
      long n[2];
      double c[2], slabs = 0.0;
      for (int k = 0; k < 2; ++k) {
        const int per = ceil_div(pr[k].kb, want[k]);
        real[k] = ceil_div(pr[k].kb, per);
        n[k] = tiles[k] * real[k];
        c[k] = unit_us(sp, per);
        // fp32 slabs written and added at 5 TB/s
        if (real[k] > 1) slabs += 2.0 * real[k] * pr[k].nz * (double)pr[k].M * pr[k].N * 4.0 / 5e6;
      }
      if (slabs > 0.0) slabs += 2.0;
      const int first = c[1] > c[0] ? 1 : 0;
      const long no[2] = {n[first], n[1 - first]};
      const double co[2] = {c[first], c[1 - first]};
      int extra = 0;
      const double t = rounds_us(no, co, &extra) + slabs;
      if (t < best_t) {
        best_t = t;
        best = PairPlan{{real[0], real[1]}, first, extra};
      }
    }
  }
  return best;
}
// The search takes a few us, so a thread keeps the plans of the shapes it has seen.
PairPlan plan_pair(int dtype, const Product& a, const Product& b) {
  struct Entry {
    Product pr[2];
    bool sp, used;
    PairPlan plan;
  };
  static thread_local Entry cache[64];
  const bool sp = split(dtype);
  size_t h = sp;
  for (const Product* p : {&a, &b})
    for (long v : {p->M, p->N, (long)p->nz, (long)p->kb}) h = h * 1000003u + (size_t)v;
  Entry& e = cache[h % 64];
  auto same = [](const Product& x, const Product& y) {
    return x.M == y.M && x.N == y.N && x.nz == y.nz && x.kb == y.kb;
  };
  if (!e.used || e.sp != sp || !same(e.pr[0], a) || !same(e.pr[1], b)) {
    const Product pr[2] = {a, b};
    e = Entry{{a, b}, sp, true, search_plan(sp, pr)};
  }
  return e.plan;
}

// K blocks of a sum with a 16-bit result that stay in the accumulator: it then
// loses at most half as much as the result's rounding.
int long_blocks(int dtype) { return dtype == DTYPE_F16 ? 512 : 4096; }

// How a product's C of the operator's type comes about: written by the
// product, or through fp32 slabs, one per split (and z).
struct Reduce {
  int splits = 1;
  bool direct = false;
  long np = 0, mp = 0;    // a slab's columns and rows
  float* slab[2] = {nullptr, nullptr};
};
Reduce plan_reduce(int dtype, const Product& pr, int splits, bool add, Carver& cv) {
  Reduce r;
  r.splits = splits;
  // fp32 adds pieces in place; 16-bit pieces add up in fp32
  r.direct = splits == 1 && (split(dtype) ? pr.N % 4 == 0 : pr.N % 8 == 0 && !add && pr.kb <= long_blocks(dtype));
  r.np = round_up(pr.N, 8);
  r.mp = round_up(pr.M, 256);
  if (!r.direct)
    for (int z = 0; z < pr.nz; ++z) r.slab[z] = cv.take<float>((size_t)splits * r.mp * r.np * 4);
  return r;
}
// Sets j's output z; with slabs, finish is still to come.
cudaError_t reduce_output(int dtype, const Reduce& rd, Job& j, int z, void* out, float* slab, bool add) {
  const long rows = j.M, N = j.N;
  j.out = add ? tg::F32_ADD : tg::F32;
  if (rd.direct) {
    if (split(dtype)) return map_out32(&j.c[z], out, rows, N, N);
    j.out = tg::STORE;
    return map_out16(&j.c[z], out, rows, N, N);
  }
  j.slab_rows = (int)round_up(rows, 256);
  return map_out32(&j.c[z], slab, (long)j.slab_rows * j.splits, rd.np, rd.np);
}

// K blocks between the register sums of a 16-bit product with column sums
// (bias gradients).  Many tiles take up to 12 blocks, evenly: a sum less is 5% of
// a whole backward pass (1999 x 768 x 50021 344 us with 8 + 4, 326 in one go),
// and dbias is 6e-7 off in norm; in one go over 16 blocks it would be 1.9e-6
// (4096 x 1024 x 32768).  Other widths with limits of 8, 12 and 16, 4096 rows,
// 32768 classes: 640 442, 412, 412 us; 896 519, 519, 501; 1280 657, 615, 615; 1536
// 830, 768, 768; 2048 1063, 1044, 1015.  Of few tiles more sums are affordable.
//
// A call that wants no column sums takes the same blocks, so that its dx and dW
// are those of one that does (4096 x 1024 x 32768 without dbias 545 us, in one go
// 516, with it 535; 1024 x 1024 x 1000 29.4, 26.6, 31.8; gates of 16384 x 1024 x
// 2736 360, 346, 366).
int column_blocks(const Job& j) {
  const long tiles = (long)j.num_m * j.num_n;
  if (tiles > 4 * kPairs) return ceil_div(j.kb_seg, ceil_div(j.kb_seg, 12));
  return tiles > kPairs ? 4 : 2;
}
// The same of the cross entropy's logits.  The forward pass hides the sums behind
// its products: 8 (512 k), logits then lose about 2^-20 of themselves (27 2^-23 at
// most, where all products have one sign).  Where a class has many rows, the
// entries p - [v = label] of its dbias cancel, but an error of z of one sign adds
// up over the rows: it counts sqrt(M / V) times as much, so that the blocks go
// down with M / V, in both passes, for what they share in lse and z cancels too.
// dbias of 100000 x 768 x 12 is then 1.2e-7 off in norm (bf16, lse of the forward
// pass; with 8 and 12 blocks 3.0e-6, and 6.4e-6 with an exact lse, now 9e-7), for
// 66 and 176 us (50 and 153); 73728 x 1024 x 1000 4.5e-7 (and 1.7e-6 with an
// exact lse, from 3.6e-6), 138 and 397 us (106 and 361); 16384 x 1024 x 174 1.2e-7
// (2.6e-6), 17.7 and 49.7 us (15.4 and 50).
int logit_blocks(const Job& j, int M, int V, bool backward) {
  const long per_class = M / V;
  if (per_class < 8) return backward ? column_blocks(j) : 8;
  const int most = per_class >= 128 ? 2 : (per_class >= 32 ? 4 : 8);
  return std::min(column_blocks(j), most);
}

// The part of a logit that the accumulator's truncation takes off on average: a
// sum that is truncated at every step of 16 k ends too near to 0 in proportion to
// itself and to the steps.  Measured over 2^19 logits of 64 to 2048 products of
// both signs, in pieces of n steps, in 2^-23 of the piece: bf16 0.103 n + 0.07, fp16
// 0.138 n + 0.27, each within a tenth (within a fifth where the products have a mean
// of 0.01 of their variance; where all are positive bf16 0.10 to 0.17 n, fp16 0.23
// to 0.44 n).  A distillation's dbias is the sum of the student's probabilities less
// that of the teacher's, which are nearly equal where the student has learnt: without
// it given back dbias was 1.7e-6 off in norm at 1999 x 768 x 50021, now 2.6e-7, and 3.6e-6 at 8000 x
// 1024 x 300, now 1.1e-6.  It is a mean: a logit whose sum is exact (a one-hot row, small
// whole numbers) loses nothing, and comes out that much too large, 3.4 (bf16) or 4.7
// (fp16) steps of 2^-23 of itself in pieces of 512 products, 5.0 and 6.9 in the backward
// pass' longest, of 768.
float logit_loss(int dtype, int D, int kb_chunk) {
  if (split(dtype)) return 0.0f;
  const int piece = tg::kBK * std::min(kb_chunk, ceil_div(D, tg::kBK)), rest = D % piece;
  auto loss = [&](int k) { return (dtype == DTYPE_F16 ? 0.138 * ceil_div(k, 16) + 0.27 : 0.103 * ceil_div(k, 16) + 0.07) * k; };
  return (float)ldexp((D / piece * loss(piece) + (rest > 0 ? loss(rest) : 0.0)) / D, -23);
}

cudaError_t gemm(int dtype, int epi, const Params& p, int num_sms, cudaStream_t s) {
  if (dtype == DTYPE_F32) return tg::gemm_f32(epi, p, num_sms, s);
  return dtype == DTYPE_BF16 ? tg::gemm_bf16(epi, p, num_sms, s) : tg::gemm_f16(epi, p, num_sms, s);
}
// The wanted ones of two reducing jobs in one launch, planned as `plan`.
cudaError_t gemm_reduce(int dtype, const Job* a, const Job* b, const PairPlan& plan, int* status, int num_sms,
                        cudaStream_t s) {
  const Job* jobs[2] = {a, b};
  if (plan.first == 1) {
    jobs[0] = b;
    jobs[1] = a;
  }
  if (jobs[0] == nullptr) {
    jobs[0] = jobs[1];
    jobs[1] = nullptr;
  }
  if (jobs[0] == nullptr) return cudaSuccess;
  Params p{};
  p.run = 1;
  p.kb_chunk = split(dtype) ? 1 : long_blocks(dtype);
  p.extra = plan.extra;
  p.status = status;
  for (int k = 0; k < 2; ++k)
    if (jobs[k] != nullptr) {
      p.j[k] = *jobs[k];
      const long units = (long)p.j[k].num_m * p.j[k].num_n * p.j[k].nz * p.j[k].splits;
      p.units[k] = units > 0x7fffffffl ? -1 : (int)units;
    }
  return gemm(dtype, tg::REDUCE, p, num_sms, s);
}

// What is left after the products, in one launch (each launch less is 2 us of a
// small call): outputs that went through fp32 slabs, out[r, c] = scale * sum
// over the slabs, in slab order; and column sums from their parts, out[c] =
// scale * sum over r of part[r, c], 32 columns a block, G threads a column,
// each over every G-th row, joined in a fixed order.
struct Finish {
  // slabs
  const float* slab[3];
  long stride[3];      // from slab to slab
  int slabs[3];
  void* out[3];
  long rows[3];
  int N, np;           // columns of the outputs and of the slabs
  int count;
  unsigned end[3];     // of each output's blocks
  // column sums
  const float* part[2];
  float* sum[2];
  long ld;
  int part_rows, n, sums;
  unsigned sum_blocks; // of each
  // what the first one's are lessened by, in units of *less_unit 2^-less_shift, and of *less_unit 2^-2 less_shift; or null
  const long long *less, *less_low;
  const float* less_unit;
  int less_shift;
};
template <int G>
__device__ __forceinline__ void part_sum(const Finish& f, int k, int block, const float* scale, float (*sm)[33]) {
  const float* a = f.part[k];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = block * 32 + lane;
  float s = 0.f;
  if (c < f.n) {
#pragma unroll 8
    for (int r = g; r < f.part_rows; r += G) s += __ldg(a + (long)r * f.ld + c);
  }
  sm[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < f.n) {
    for (int j = 1; j < G; ++j) s += sm[j][lane];
    float sum = scale != nullptr ? s * __ldg(scale) : s;
    if (k == 0 && f.less != nullptr)
      sum -= (ldexpf((float)f.less[c], -f.less_shift) + ldexpf((float)f.less_low[c], -2 * f.less_shift)) * __ldg(f.less_unit);
    f.sum[k][c] = sum;
  }
}
// Column sums of many parts.
__global__ void __launch_bounds__(1024) part_sum_kernel(const __grid_constant__ Finish f, const float* scale) {
  __shared__ float sm[32][33];
  part_sum<32>(f, blockIdx.y, blockIdx.x, scale, sm);
}
// The column sums' blocks come first, then those of each slab output.  VEC: N is
// the slabs' row length, 8 values a thread; else one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kBlock) finish_kernel(const __grid_constant__ Finish q, const float* __restrict__ scale) {
  __shared__ float sm[kBlock / 32][33];
  unsigned block = blockIdx.x;
  const unsigned sums = q.sums * q.sum_blocks;
  if (block < sums) {
    const int k = block < q.sum_blocks ? 0 : 1;
    part_sum<kBlock / 32>(q, k, (int)(block - k * q.sum_blocks), scale, sm);
    return;
  }
  block -= sums;
  const int y = block < q.end[0] ? 0 : (block < q.end[1] ? 1 : 2);
  if (y > 0) block -= q.end[y - 1];
  const long i = (long)block * kBlock + threadIdx.x;
  const float sc = scale != nullptr ? __ldg(scale) : 1.f;
  T* out = static_cast<T*>(q.out[y]);
  const int n_slabs = q.slabs[y];
  const long stride = q.stride[y];
  if constexpr (VEC) {
    if (i * 8 >= q.rows[y] * q.N) return;
    float v[8] = {};
    const float4* a = reinterpret_cast<const float4*>(q.slab[y]) + 2 * i;
#pragma unroll 4
    for (int k = 0; k < n_slabs; ++k, a += stride / 4) {
      const float4 x = __ldg(a), w = __ldg(a + 1);
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w; v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= sc;
    if constexpr (sizeof(T) == 2) {
      reinterpret_cast<uint4*>(out)[i] =
          make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    } else {
      reinterpret_cast<float4*>(out)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(out)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
    const long r = i / q.N;
    if (r >= q.rows[y]) return;
    const float* a = q.slab[y] + r * q.np + (i - r * q.N);
    float v = 0.f;
#pragma unroll 4
    for (int k = 0; k < n_slabs; ++k, a += stride) v += __ldg(a);
    out[i] = DT<T>::from(v * sc);
  }
}
// Adds an output of j that went through slabs.
void add_slab_sum(Finish& q, const Reduce& rd, int z, int slabs, long slab_rows, void* out, long rows, long N) {
  if (rd.direct || out == nullptr) return;
  const int k = q.count++;
  q.slab[k] = rd.slab[z];
  q.stride[k] = slab_rows * rd.np;
  q.slabs[k] = slabs;
  q.out[k] = out;
  q.rows[k] = rows;
  q.N = (int)N;
  q.np = (int)rd.np;
}
// Adds sums of n columns from `rows` rows of parts, ld apart.
void add_part_sum(Finish& q, const float* part, float* sum, long ld, int rows, int n) {
  if (sum == nullptr) return;
  const int k = q.sums++;
  q.part[k] = part;
  q.sum[k] = sum;
  q.ld = ld;
  q.part_rows = rows;
  q.n = n;
  q.sum_blocks = blocks_for(n, 32);
}
template <typename T>
cudaError_t finish_t(Finish& q, const float* scale, cudaStream_t s) {
  const bool vec = q.N % 8 == 0;
  unsigned blocks = 0;
  for (int k = 0; k < 3; ++k) {
    if (k < q.count) blocks += blocks_for(vec ? q.rows[k] * q.N / 8 : q.rows[k] * q.N, kBlock);
    q.end[k] = blocks;
  }
  blocks += q.sums * q.sum_blocks;
  if (vec) finish_kernel<T, true><<<blocks, kBlock, 0, s>>>(q, scale);
  else finish_kernel<T, false><<<blocks, kBlock, 0, s>>>(q, scale);
  return cudaGetLastError();
}
cudaError_t finish(int dtype, Finish& q, const float* scale, cudaStream_t s) {
  if (q.sums > 0 && q.part_rows > 512) {   // a launch of its own, 32 threads a column
    part_sum_kernel<<<dim3(q.sum_blocks, q.sums), 1024, 0, s>>>(q, scale);
    JEPA_TRY_CUDA(cudaGetLastError());
    q.sums = 0;
  }
  if (q.count == 0 && q.sums == 0) return cudaSuccess;
  if (dtype == DTYPE_F32) return finish_t<float>(q, scale, s);
  return dtype == DTYPE_F16 ? finish_t<__half>(q, scale, s) : finish_t<__nv_bfloat16>(q, scale, s);
}

// ----------------------------------------------------------------------------- column sums
// Column sums of an [M, N] matrix: block (256 columns, strip of rows), 8
// consecutive columns a thread (VEC: rows of 16 bytes) or 8 columns 32 apart,
// 8 rows at a time.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kBlock) col_strip_kernel(const T* __restrict__ a, int M, int N, int rows_per,
                                                           float* __restrict__ part) {
  __shared__ float sm[8][256 + 8];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 256 + (VEC ? lane * 8 : lane);
  const int r0 = blockIdx.y * rows_per, r1 = min(M, r0 + rows_per);
  float v[8] = {};
#pragma unroll 4
  for (int r = r0 + g; r < r1; r += 8) {
    const T* p = a + (size_t)r * N + c;
    if constexpr (VEC) {
      constexpr int kPer = 16 / sizeof(T);
#pragma unroll
      for (int j = 0; j < 8; j += kPer) {
        if (c + j < N) {
          const uint4 q = __ldg(reinterpret_cast<const uint4*>(p + j));
          T h[kPer];
          memcpy(h, &q, 16);
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[j + i] += DT<T>::to(h[i]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + 32 * j < N) v[j] += DT<T>::to(p[32 * j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sm[g][VEC ? lane * 8 + j : lane + 32 * j] = v[j];
  __syncthreads();
  const int cc = blockIdx.x * 256 + threadIdx.x;
  if (cc < N) {
    float s = 0.f;
    for (int k = 0; k < 8; ++k) s += sm[k][threadIdx.x];
    part[(size_t)blockIdx.y * N + cc] = s;
  }
}
int col_strips(int M, int N) {
  const int want = ceil_div(4 * 152, ceil_div(N, 256)), most = ceil_div(M, 32);
  return want < most ? want : most;
}
// The strips' sums in part, or with one strip in out.
template <typename T>
cudaError_t col_strip_t(const void* a, int M, int N, int strips, float* to, cudaStream_t s) {
  const int per = ceil_div(M, strips);
  const dim3 g(ceil_div(N, 256), strips);
  if ((N * sizeof(T)) % 16 == 0) col_strip_kernel<T, true><<<g, kBlock, 0, s>>>((const T*)a, M, N, per, to);
  else col_strip_kernel<T, false><<<g, kBlock, 0, s>>>((const T*)a, M, N, per, to);
  return cudaGetLastError();
}
cudaError_t col_strip(int dtype, const void* a, int M, int N, int strips, float* to, cudaStream_t s) {
  if (dtype == DTYPE_F32) return col_strip_t<float>(a, M, N, strips, to, s);
  if (dtype == DTYPE_F16) return col_strip_t<__half>(a, M, N, strips, to, s);
  return col_strip_t<__nv_bfloat16>(a, M, N, strips, to, s);
}

cudaError_t zero(void* p, size_t bytes, cudaStream_t s) {
  return p == nullptr || bytes == 0 ? cudaSuccess : cudaMemsetAsync(p, 0, bytes, s);
}

// ----------------------------------------------------------------------------- softmax cross entropy
// Joins the statistics of a row's parts, in a fixed order: a block takes 32 rows,
// its 8 warps every eighth part each, or with ONE a single row, its threads every
// 256th part each (many parts of few rows).
// Of the row that this thread is to finish (true): its lse = ln(2^m s), and the sum.
template <bool ONE>
__device__ __forceinline__ bool join_row(const float2* __restrict__ ms, const float* __restrict__ sums, int parts, int M,
                                         int& row, float& lse, float& sum) {
  __shared__ Ms sm[8][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  row = ONE ? (int)blockIdx.x : (int)blockIdx.x * 32 + lane;
  Ms a{-INFINITY, 0.f, 0.f};
  if (row < M) {
#pragma unroll 4
    for (int k = ONE ? threadIdx.x : g; k < parts; k += ONE ? kBlock : 8) {
      const float2 q = __ldg(ms + (size_t)k * M + row);
      ms_join(a, q.x, q.y, sums != nullptr ? __ldg(sums + (size_t)k * M + row) : 0.f);
    }
  }
  if constexpr (ONE) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, a.m, o), v = __shfl_xor_sync(0xffffffffu, a.s, o);
      ms_join(a, m, v, __shfl_xor_sync(0xffffffffu, a.sum, o));
    }
  }
  sm[g][lane] = a;
  __syncthreads();
  if (g != 0 || row >= M || (ONE && lane != 0)) return false;
  for (int k = 1; k < 8; ++k) ms_join(a, sm[k][lane].m, sm[k][lane].s, sm[k][lane].sum);
  lse = (a.m + log2f(a.s)) * 0.69314718055994531f;
  sum = a.sum;
  return true;
}
template <bool ONE>
__global__ void __launch_bounds__(kBlock) ce_join_kernel(const float2* __restrict__ ms, const float* __restrict__ sums,
                                                         const float* __restrict__ zy, int parts, int M, int V,
                                                         const int64_t* __restrict__ labels, long ignore_index,
                                                         float smoothing, float* __restrict__ loss,
                                                         float* __restrict__ lse_out, int* status) {
  int row;
  float lse, sum;
  if (!join_row<ONE>(ms, sums, parts, M, row, lse, sum)) return;
  const long label = labels[row];
  float l;
  if (label == ignore_index) {
    l = 0.f;
  } else if (label < 0 || label >= V) {
    l = NAN;
    atomicOr(status, DEV_BAD_INDEX);
  } else {
    l = lse - (1.0f - smoothing) * zy[row];
    if (smoothing > 0.f) l -= smoothing * (sum / (float)V);
  }
  if (loss != nullptr) loss[row] = l;
  lse_out[row] = lse;
}
cudaError_t ce_join(const CeArgs& a, const float2* ms, const float* sums, const float* zy, int parts, float* loss,
                    float* lse, cudaStream_t s) {
  if (a.M <= 16)
    ce_join_kernel<true><<<a.M, kBlock, 0, s>>>(ms, sums, zy, parts, a.M, a.V, a.labels, a.ignore_index, a.smoothing,
                                                loss, lse, a.status);
  else
    ce_join_kernel<false><<<blocks_for(a.M, 32), kBlock, 0, s>>>(ms, sums, zy, parts, a.M, a.V, a.labels,
                                                                 a.ignore_index, a.smoothing, loss, lse, a.status);
  return cudaGetLastError();
}

// 16-bit dz is held in units of the largest finite |dloss| of the rows that have
// a gradient, times a factor: 1 in bf16; in fp16 a power of 2, so that |dz|, at
// most factor / (1 - smoothing), stays below fp16's largest value and small
// probabilities stay normal numbers.
float dz_factor(int dtype, float smoothing) {
  return dtype == DTYPE_F16 ? ldexpf(1.0f, 14 + (int)floorf(log2f(1.0f - smoothing))) : 1.0f;
}
// Up to 16384 rows CE_BWD finds the unit itself (4096 x 256 x 2048: 37 us, with
// a kernel for it 39, and 3 us less on the host); where there are more rows a
// kernel does (65536 x 256 x 512: 103 us, in CE_BWD 110).
constexpr int kInlineRows = 16384;
__global__ void __launch_bounds__(1024) dz_unit_kernel(const float* __restrict__ dloss,
                                                       const int64_t* __restrict__ labels, long ignore_index, int M,
                                                       int V, float factor, float smoothing, float* scale) {
  __shared__ float sm[32];
  const float m = tg::dz_max(dloss, labels, ignore_index, M, V, threadIdx.x, 1024);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    float all = m;
    for (int k = 1; k < 32; ++k) all = fmaxf(all, sm[k]);
    tg::dz_unit(all, factor, smoothing, scale);
  }
}

// Column tiles per unit of the forward pass: at least 8 units a pair, at most 16 tiles.
int ce_run(long M, long V) {
  const long tiles = (long)ceil_div(M, 256) * ceil_div(V, 256);
  const long r = tiles / (kPairs * 8);
  return (int)(r < 1 ? 1 : (r > 16 ? 16 : r));
}

struct CeFwd {
  Mat x, w;
  int run, parts;
  float2* ms;
  float *sums, *zy;
  size_t bytes;
};
CeFwd ce_fwd_layout(const CeArgs& a, void* ws) {
  Carver cv{static_cast<uint8_t*>(ws)};
  CeFwd l;
  if (few_rows_ok(a.dtype, a.M, a.D)) {
    l.parts = few_rows_ce_parts(a.V);
  } else {
    l.x = operand(a.dtype, a.x, a.M, a.D, cv);
    l.w = operand(a.dtype, a.w, a.V, a.D, cv);
    l.run = ce_run(a.M, a.V);
    l.parts = 2 * ceil_div(ceil_div(a.V, 256), l.run);
  }
  const size_t n = (size_t)l.parts * a.M;
  l.ms = cv.take<float2>(n * 8);
  l.sums = a.smoothing > 0.f ? cv.take<float>(n * 4) : nullptr;
  l.zy = cv.take<float>((size_t)a.M * 4);
  l.bytes = cv.used;
  return l;
}

// The backward pass goes over the vocabulary in pieces whose dz takes at most
// 256 MB, but that have 4096 columns at least (more than 32768 rows in 16 bits,
// 10922 in fp32: 8 GB at 2^20 rows), all of the same width up to rounding to 256.
struct CeBwd {
  Mat x, w;
  int piece, dz_plane;
  uint8_t* dz;
  float *scale, *colp;
  PairPlan plan;
  Reduce dx, dw;
  size_t bytes;
};
CeBwd ce_bwd_layout(const CeArgs& a, void* ws) {
  Carver cv{static_cast<uint8_t*>(ws)};
  CeBwd l;
  l.x = operand(a.dtype, a.x, a.M, a.D, cv);
  l.w = operand(a.dtype, a.w, a.V, a.D, cv);
  const long rows = split(a.dtype) ? 3 * round_up(a.M, 256) : a.M;
  long most = ((long)256 << 20) / (2 * rows) / 256 * 256;
  if (most < 4096) most = 4096;
  int pieces = ceil_div(a.V, most);
  l.piece = (int)round_up(ceil_div(a.V, pieces), 256);
  pieces = ceil_div(a.V, l.piece);
  l.dz_plane = split(a.dtype) ? (int)round_up(a.M, 256) : 0;
  l.dz = cv.take<uint8_t>((size_t)rows * l.piece * 2);
  l.scale = cv.take<float>(2 * sizeof(float));
  l.colp = cv.take<float>((size_t)ceil_div(a.M, 32) * l.piece * 4);
  const int n = a.V < l.piece ? a.V : l.piece;
  const Product dx{a.M, a.D, 1, ceil_div(n, tg::kBK)}, dw{n, a.D, 1, ceil_div(a.M, tg::kBK)};
  l.plan = plan_pair(a.dtype, dx, dw);
  l.dx = plan_reduce(a.dtype, dx, l.plan.splits[0], pieces > 1, cv);
  l.dw = plan_reduce(a.dtype, dw, l.plan.splits[1], false, cv);
  l.bytes = cv.used;
  return l;
}

}  // namespace

size_t linear_ce_workspace(int M, int D, int V, int dtype, bool backward) {
  if (M == 0) return 0;
  CeArgs a{};
  a.M = M;
  a.D = D;
  a.V = V;
  a.dtype = dtype;
  a.smoothing = 0.5f;   // the larger layout
  return backward ? ce_bwd_layout(a, nullptr).bytes : ce_fwd_layout(a, nullptr).bytes;
}

namespace {

// The statistics of every row of z, or with DISTILL_FWD of z / temperature, in
// parts; ep: what the epilogue needs beside the cross entropy's; e: the entries of
// a few rows.
cudaError_t ce_statistics(const CeArgs& a, const CeFwd& l, int epi, const tg::EpiArgs& ep, const FewEntries& e, cudaStream_t s) {
  if (few_rows_ok(a.dtype, a.M, a.D)) return few_rows_ce(a, e, l.ms, l.sums, l.zy, ep.z_scale, s);
  Fills f{};
  add_fill(f, a.x, l.x);
  add_fill(f, a.w, l.w);
  JEPA_TRY_CUDA(fill(a.dtype, f, s));
  Job j = base_job(a.M, a.V, tg::kBN);
  set_k(j, a.D, 1, 1);
  JEPA_TRY_CUDA(map_k(&j.a[0], l.x));
  JEPA_TRY_CUDA(map_k(&j.b[0], l.w));
  j.a_plane = (int)l.x.plane_rows;
  j.b_plane = (int)l.w.plane_rows;
  Params p = forward_params(j, l.run, a.status);
  p.kb_chunk = split(a.dtype) ? 1 : logit_blocks(j, a.M, a.V, false);
  p.ep = ep;
  p.ep.bias = a.bias;
  p.ep.labels = a.labels;
  p.ep.V = a.V;
  p.ep.part_ms = l.ms;
  p.ep.part_sum = l.sums;
  p.ep.zy = l.zy;
  p.ep.z_loss = logit_loss(a.dtype, a.D, p.kb_chunk);
  return gemm(a.dtype, epi, p, a.num_sms, s);
}

// What the sums of a distillation's dz do not have in them: (acc[v] + acc[V + v] 2^-shift) 2^-shift unit.
struct Less {
  const long long* acc;
  int shift;
};
// The gradients, piece by piece of the vocabulary.  after(dz, v0, n) is called
// once a piece's dz is on its way, before the products of it.
template <typename After>
cudaError_t ce_gradients(const CeArgs& a, const CeBwd& l, int epi, float z_scale, const float* lse, const float* dloss,
                         void* dx, void* dw, float* dbias, const Less& less, cudaStream_t s, After&& after) {
  const bool sp = split(a.dtype);
  Fills f{};
  add_fill(f, a.x, l.x);
  add_fill(f, a.w, l.w);
  JEPA_TRY_CUDA(fill(a.dtype, f, s));
  const float* unscale = nullptr;
  if (!sp) unscale = l.scale + 1;
  int dx_slabs = 1;
  for (int v0 = 0; v0 < a.V; v0 += l.piece) {
    const int n = a.V - v0 < l.piece ? a.V - v0 : l.piece;
    const Mat w = rows_from(l.w, v0, n);
    Mat dz;
    dz.p = l.dz;
    dz.rows = a.M;
    dz.cols = n;
    dz.ld = l.piece;
    dz.plane_rows = l.dz_plane;
    {
      Job j = base_job(a.M, n, tg::kBN);
      set_k(j, a.D, 1, 1);
      JEPA_TRY_CUDA(map_k(&j.a[0], l.x));
      JEPA_TRY_CUDA(map_k(&j.b[0], w, v0));
      JEPA_TRY_CUDA(map_out16(&j.c[0], l.dz, sp ? 3 * (long)l.dz_plane : a.M, l.piece, l.piece));
      j.a_plane = (int)l.x.plane_rows;
      j.b_plane = (int)l.w.plane_rows;
      Params p = forward_params(j, 1, a.status);
      p.kb_chunk = sp ? 1 : logit_blocks(j, a.M, a.V, true);
      // where a class has many rows, a distillation's dbias is a small difference of sums over them: half the blocks
      // (4164 x 168 x 41 in fp16 0.8e-6 off in norm instead of 1.2e-6)
      if (epi == tg::DISTILL_BWD && a.M / a.V >= 8) p.kb_chunk = std::max(1, p.kb_chunk / 2);
      p.c_plane = l.dz_plane;
      p.ep.bias = a.bias != nullptr ? a.bias + v0 : nullptr;
      p.ep.labels = a.labels;
      p.ep.ignore_index = a.ignore_index;
      p.ep.lse = lse;
      p.ep.dloss = dloss;
      p.ep.dz_scale = l.scale;
      p.ep.dz_factor = dz_factor(a.dtype, a.smoothing);
      p.ep.dz_inline = a.M <= kInlineRows;
      p.ep.smoothing = a.smoothing;
      p.ep.v0 = v0;
      p.ep.V = a.V;
      p.ep.col_part = dbias != nullptr ? l.colp : nullptr;
      p.ep.ld_col = l.piece;
      p.ep.z_scale = z_scale;
      p.ep.z_loss = logit_loss(a.dtype, a.D, p.kb_chunk);
      JEPA_TRY_CUDA(gemm(a.dtype, epi, p, a.num_sms, s));
      JEPA_TRY_CUDA(after(dz, v0, n));
    }
    Job jx = base_job(a.M, a.D, tg::kBN), jw = base_job(n, a.D, tg::kBN);
    uint8_t* dw_out = dw != nullptr ? static_cast<uint8_t*>(dw) + elem(a.dtype) * (size_t)v0 * a.D : nullptr;
    if (dx != nullptr) {
      set_k(jx, n, 1, l.dx.splits);
      JEPA_TRY_CUDA(map_k(&jx.a[0], dz));
      JEPA_TRY_CUDA(map_mn(&jx.b[0], w, v0));
      jx.a_plane = l.dz_plane;
      jx.b_plane = (int)l.w.plane_rows;
      jx.scale = unscale;
      // the first piece has the most splits: a narrower last piece adds into the first slabs
      if (v0 == 0) dx_slabs = jx.splits;
      JEPA_TRY_CUDA(reduce_output(a.dtype, l.dx, jx, 0, dx, l.dx.slab[0], v0 != 0));
    }
    if (dw != nullptr) {
      set_k(jw, a.M, 1, l.dw.splits);
      JEPA_TRY_CUDA(map_mn(&jw.a[0], dz));
      JEPA_TRY_CUDA(map_mn(&jw.b[0], l.x));
      jw.a_mn = 1;
      jw.a_plane = l.dz_plane;
      jw.b_plane = (int)l.x.plane_rows;
      jw.scale = unscale;
      JEPA_TRY_CUDA(reduce_output(a.dtype, l.dw, jw, 0, dw_out, l.dw.slab[0], false));
    }
    JEPA_TRY_CUDA(gemm_reduce(a.dtype, dx != nullptr ? &jx : nullptr, dw != nullptr ? &jw : nullptr, l.plan, a.status,
                              a.num_sms, s));
    Finish q{};
    if (dbias != nullptr) add_part_sum(q, l.colp, dbias + v0, l.piece, ceil_div(a.M, 32), n);
    if (less.acc != nullptr) {
      q.less = less.acc + v0;
      q.less_low = q.less + a.V;
      q.less_unit = l.scale;
      q.less_shift = less.shift;
    }
    add_slab_sum(q, l.dw, 0, jw.splits, jw.slab_rows, dw_out, n, a.D);
    if (v0 + n == a.V) add_slab_sum(q, l.dx, 0, dx_slabs, l.dx.mp, dx, a.M, a.D);
    JEPA_TRY_CUDA(finish(a.dtype, q, unscale, s));
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t linear_ce_fwd(const CeArgs& a, float* loss, float* lse, void* ws, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  const CeFwd l = ce_fwd_layout(a, ws);
  tg::EpiArgs ep{};
  ep.z_scale = tg::kLog2e;
  JEPA_TRY_CUDA(ce_statistics(a, l, tg::CE_FWD, ep, FewEntries{}, s));
  return ce_join(a, l.ms, l.sums, l.zy, l.parts, loss, lse, s);
}

cudaError_t linear_ce_bwd(const CeArgs& a, const float* lse, const float* dloss, void* dx, void* dw, float* dbias,
                          void* ws, cudaStream_t s) {
  if (a.M == 0) {
    JEPA_TRY_CUDA(zero(dw, elem(a.dtype) * (size_t)a.V * a.D, s));
    return zero(dbias, sizeof(float) * (size_t)a.V, s);
  }
  const CeBwd l = ce_bwd_layout(a, ws);
  if (!split(a.dtype) && a.M > kInlineRows) {
    dz_unit_kernel<<<1, 1024, 0, s>>>(dloss, a.labels, a.ignore_index, a.M, a.V, dz_factor(a.dtype, a.smoothing),
                                      a.smoothing, l.scale);
    JEPA_TRY_CUDA(cudaGetLastError());
  }
  return ce_gradients(a, l, tg::CE_BWD, tg::kLog2e, lse, dloss, dx, dw, dbias, Less{}, s,
                      [](const Mat&, int, int) { return cudaSuccess; });
}

// ----------------------------------------------------------------------------- distillation
namespace {

struct DistillBwd {
  CeBwd ce;
  int64_t* label;
  float *dl, *prob;
  int* cls;
  long long* acc;
  size_t bytes;
};
DistillBwd distill_bwd_layout(const DistillArgs& a, void* ws) {
  DistillBwd l;
  l.ce = ce_bwd_layout(a.ce, ws);
  Carver cv{static_cast<uint8_t*>(ws), l.ce.bytes};
  const size_t n = (size_t)a.ce.M * a.K;
  l.label = cv.take<int64_t>((size_t)a.ce.M * 8);
  l.dl = cv.take<float>((size_t)a.ce.M * 4);
  l.prob = cv.take<float>(n * 4);
  l.cls = cv.take<int>(n * 4);
  l.acc = cv.take<long long>((size_t)a.ce.V * 16);
  l.bytes = cv.used;
  return l;
}

}  // namespace

size_t linear_distill_workspace(int M, int D, int V, int K, int dtype, bool backward) {
  if (M == 0) return 0;
  DistillArgs a{};
  a.ce.M = M;
  a.ce.D = D;
  a.ce.V = V;
  a.ce.dtype = dtype;
  a.K = K;
  if (backward) return distill_bwd_layout(a, nullptr).bytes;
  const CeFwd l = ce_fwd_layout(a.ce, nullptr);
  if (few_rows_ok(dtype, M, D)) return l.bytes;
  return l.bytes + align256((size_t)M * K * 4) + align256((size_t)M * (l.parts + 2) * 2);
}

cudaError_t linear_distill_fwd(const DistillArgs& a, float* loss, float* lse, float* z, void* ws, cudaStream_t s) {
  const CeArgs& c = a.ce;
  if (c.M == 0) return cudaSuccess;
  const CeFwd l = ce_fwd_layout(c, ws);
  tg::EpiArgs ep{};
  ep.z_scale = tg::kLog2e / a.tau;
  FewEntries e{};
  if (few_rows_ok(c.dtype, c.M, c.D)) {
    e = {a.ids, a.K, a.ignore_index, z, 0};
  } else {
    Carver cv{static_cast<uint8_t*>(ws), l.bytes};
    uint32_t* hits = cv.take<uint32_t>((size_t)c.M * a.K * 4);
    uint16_t* starts = cv.take<uint16_t>((size_t)c.M * (l.parts + 2) * 2);
    ep.hits = hits;
    ep.starts = starts;
    ep.hit_z = z;
    ep.top = a.K;
    ep.runs = l.parts / 2;
    JEPA_TRY_CUDA(distill_hits(a, l.run, ep.runs, hits, starts, z, s));
  }
  JEPA_TRY_CUDA(ce_statistics(c, l, tg::DISTILL_FWD, ep, e, s));
  return distill_join(a, l.ms, l.parts, z, loss, lse, s);
}

cudaError_t linear_distill_bwd(const DistillArgs& a, const float* lse, const float* z, const float* dloss, void* dx,
                               void* dw, float* dbias, void* ws, cudaStream_t s) {
  CeArgs c = a.ce;
  if (c.M == 0) {
    JEPA_TRY_CUDA(zero(dw, elem(c.dtype) * (size_t)c.V * c.D, s));
    return zero(dbias, sizeof(float) * (size_t)c.V, s);
  }
  const DistillBwd l = distill_bwd_layout(a, ws);
  const bool sp = split(c.dtype);
  JEPA_TRY_CUDA(distill_teacher(a, dloss, l.label, l.dl, l.cls, l.prob, dbias != nullptr ? l.acc : nullptr, s));
  c.labels = l.label;
  c.ignore_index = -1;
  c.smoothing = 0.f;
  if (c.M > kInlineRows || (sp && dbias != nullptr)) {
    dz_unit_kernel<<<1, 1024, 0, s>>>(l.dl, l.label, -1, c.M, c.V, dz_factor(c.dtype, 0.f), 0.f, l.ce.scale);
    JEPA_TRY_CUDA(cudaGetLastError());
  }
  // a class's sum of up to M probabilities of at most 1 (and the rounding of each) stays below 2^62, and so do M halves of
  // what is left
  int shift = 61;
  while (((long)1 << (61 - shift)) < c.M) --shift;
  DistillPut q{l.cls, l.prob, z, lse, l.dl, c.M, a.K, 0, 0, c.V, tg::kLog2e / a.tau, dz_factor(c.dtype, 0.f),
               l.ce.scale, nullptr, 0, 0, dbias != nullptr ? l.acc : nullptr, shift};
  return ce_gradients(c, l.ce, tg::DISTILL_BWD, tg::kLog2e / a.tau, lse, l.dl, dx, dw, dbias, Less{q.acc, shift}, s,
                      [&](const Mat& dz, int v0, int n) {
                        q.v0 = v0;
                        q.n = n;
                        q.dz = reinterpret_cast<uint16_t*>(const_cast<uint8_t*>(dz.p));
                        q.ld = dz.ld;
                        q.plane_rows = dz.plane_rows;
                        return distill_put(c.dtype, q, c.num_sms, s);
                      });
}

// ----------------------------------------------------------------------------- gated feed-forward
namespace {

struct FfnFwd {
  Mat x, wg, wu;
  size_t bytes;
};
FfnFwd ffn_fwd_layout(const FfnArgs& a, Carver& cv) {
  FfnFwd l;
  l.x = operand(a.dtype, a.x, a.M, a.D, cv);
  l.wg = operand(a.dtype, a.wg, a.F, a.D, cv);
  l.wu = operand(a.dtype, a.wu, a.F, a.D, cv);
  l.bytes = cv.used;
  return l;
}
// dg and du are [M, fp], in planes for fp32.
struct FfnBwd {
  FfnFwd in;
  int fp, d_plane;
  uint8_t* d[2];
  float* colp[2];
  PairPlan plan;
  Reduce dx, dw;
  size_t bytes;
};
FfnBwd ffn_bwd_layout(const FfnArgs& a, void* ws) {
  Carver cv{static_cast<uint8_t*>(ws)};
  FfnBwd l;
  l.in = ffn_fwd_layout(a, cv);
  l.fp = (int)round_up(a.F, 64);
  l.d_plane = split(a.dtype) ? (int)round_up(a.M, 256) : 0;
  const long rows = split(a.dtype) ? 3 * (long)l.d_plane : a.M;
  for (int k = 0; k < 2; ++k) l.d[k] = cv.take<uint8_t>((size_t)rows * l.fp * 2);
  for (int k = 0; k < 2; ++k) l.colp[k] = cv.take<float>((size_t)ceil_div(a.M, 32) * l.fp * 4);
  const Product dx{a.M, a.D, 1, 2 * ceil_div(a.F, tg::kBK)}, dw{a.F, a.D, 2, ceil_div(a.M, tg::kBK)};
  l.plan = plan_pair(a.dtype, dx, dw);
  l.dx = plan_reduce(a.dtype, dx, l.plan.splits[0], false, cv);
  l.dw = plan_reduce(a.dtype, dw, l.plan.splits[1], false, cv);
  l.bytes = cv.used;
  return l;
}
cudaError_t ffn_product(const FfnArgs& a, const FfnFwd& l, Job& j, cudaStream_t s) {
  Fills f{};
  add_fill(f, a.x, l.x);
  add_fill(f, a.wg, l.wg);
  add_fill(f, a.wu, l.wu);
  JEPA_TRY_CUDA(fill(a.dtype, f, s));
  j = base_job(a.M, a.F, tg::kBN / 2);
  set_k(j, a.D, 1, 1);
  JEPA_TRY_CUDA(map_k(&j.a[0], l.x));
  JEPA_TRY_CUDA(map_k(&j.b[0], l.wg));
  JEPA_TRY_CUDA(map_k(&j.b[1], l.wu));
  j.a_plane = (int)l.x.plane_rows;
  j.b_plane = (int)l.wg.plane_rows;
  return cudaSuccess;
}
Params ffn_params(const FfnArgs& a, const Job& j) {
  Params p = forward_params(j, 1, a.status);
  p.kb_chunk = split(a.dtype) ? 1 : long_blocks(a.dtype);
  p.ep.bias = a.bg;
  p.ep.bias2 = a.bu;
  p.ep.act = a.act;
  return p;
}

}  // namespace

size_t gated_ffn_workspace(int M, int D, int F, int dtype, bool backward) {
  if (M == 0) return 0;
  FfnArgs a{};
  a.M = M;
  a.D = D;
  a.F = F;
  a.dtype = dtype;
  if (backward) return ffn_bwd_layout(a, nullptr).bytes;
  if (few_rows_ok(dtype, M, D)) return 0;
  Carver cv{nullptr};
  return ffn_fwd_layout(a, cv).bytes;
}

cudaError_t gated_ffn_fwd(const FfnArgs& a, void* h, void* ws, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  if (few_rows_ok(a.dtype, a.M, a.D)) return few_rows_gate(a, h, s);
  Carver cv{static_cast<uint8_t*>(ws)};
  const FfnFwd l = ffn_fwd_layout(a, cv);
  Job j;
  JEPA_TRY_CUDA(ffn_product(a, l, j, s));
  const bool plain = (a.F * elem(a.dtype)) % 16 != 0;
  if (!plain)
    JEPA_TRY_CUDA(split(a.dtype) ? map_out32(&j.c[0], h, a.M, a.F, a.F) : map_out16(&j.c[0], h, a.M, a.F, a.F));
  Params p = ffn_params(a, j);
  if (plain) {
    p.plain = h;
    p.plain_ld = a.F;
  }
  return gemm(a.dtype, tg::GATE_FWD, p, a.num_sms, s);
}

cudaError_t gated_ffn_bwd(const FfnArgs& a, const void* dh, void* dx, void* dwg, void* dwu, float* dbg, float* dbu,
                          void* ws, cudaStream_t s) {
  if (a.M == 0) {
    for (void* dw : {dwg, dwu}) JEPA_TRY_CUDA(zero(dw, elem(a.dtype) * (size_t)a.F * a.D, s));
    for (float* db : {dbg, dbu}) JEPA_TRY_CUDA(zero(db, sizeof(float) * (size_t)a.F, s));
    return cudaSuccess;
  }
  const FfnBwd l = ffn_bwd_layout(a, ws);
  const bool sp = split(a.dtype);
  Mat d[2];
  for (int k = 0; k < 2; ++k) {
    d[k].p = l.d[k];
    d[k].rows = a.M;
    d[k].cols = a.F;
    d[k].ld = l.fp;
    d[k].plane_rows = l.d_plane;
  }
  {
    Job j;
    JEPA_TRY_CUDA(ffn_product(a, l.in, j, s));
    for (int k = 0; k < 2; ++k)
      JEPA_TRY_CUDA(map_out16(&j.c[k], l.d[k], sp ? 3 * (long)l.d_plane : a.M, l.fp, l.fp));
    Params p = ffn_params(a, j);
    if (!sp) p.kb_chunk = column_blocks(j);
    p.c_plane = l.d_plane;
    p.ep.dh = dh;
    p.ep.dh_vec = (a.F * elem(a.dtype)) % 16 == 0;
    p.ep.col_part = dbg != nullptr ? l.colp[0] : nullptr;
    p.ep.col_part2 = dbu != nullptr ? l.colp[1] : nullptr;
    p.ep.ld_col = l.fp;
    JEPA_TRY_CUDA(gemm(a.dtype, tg::GATE_BWD, p, a.num_sms, s));
  }
  Job jx = base_job(a.M, a.D, tg::kBN), jw = base_job(a.F, a.D, tg::kBN);
  if (dx != nullptr) {
    set_k(jx, a.F, 2, l.dx.splits);
    for (int k = 0; k < 2; ++k) {
      JEPA_TRY_CUDA(map_k(&jx.a[k], d[k]));
      JEPA_TRY_CUDA(map_mn(&jx.b[k], k == 0 ? l.in.wg : l.in.wu));
    }
    jx.a_plane = l.d_plane;
    jx.b_plane = (int)l.in.wg.plane_rows;
    JEPA_TRY_CUDA(reduce_output(a.dtype, l.dx, jx, 0, dx, l.dx.slab[0], false));
  }
  // the weight gradients that are wanted are one job
  void* dw[2] = {dwg, dwu};
  jw.nz = 0;
  set_k(jw, a.M, 1, l.dw.splits);
  jw.a_mn = 1;
  for (int k = 0; k < 2; ++k) {
    if (dw[k] == nullptr) continue;
    JEPA_TRY_CUDA(map_mn(&jw.a[jw.nz], d[k]));
    JEPA_TRY_CUDA(reduce_output(a.dtype, l.dw, jw, jw.nz, dw[k], l.dw.slab[k], false));
    ++jw.nz;
  }
  if (jw.nz > 0) {
    JEPA_TRY_CUDA(map_mn(&jw.b[0], l.in.x));
    jw.a_plane = l.d_plane;
    jw.b_plane = (int)l.in.x.plane_rows;
  }
  JEPA_TRY_CUDA(gemm_reduce(a.dtype, dx != nullptr ? &jx : nullptr, jw.nz > 0 ? &jw : nullptr, l.plan, a.status,
                            a.num_sms, s));
  Finish q{};
  add_part_sum(q, l.colp[0], dbg, l.fp, ceil_div(a.M, 32), a.F);
  add_part_sum(q, l.colp[1], dbu, l.fp, ceil_div(a.M, 32), a.F);
  add_slab_sum(q, l.dx, 0, jx.splits, jx.slab_rows, dx, a.M, a.D);
  for (int k = 0; k < 2; ++k) add_slab_sum(q, l.dw, k, jw.splits, jw.slab_rows, dw[k], a.F, a.D);
  return finish(a.dtype, q, nullptr, s);
}

// ----------------------------------------------------------------------------- linear layer backward
namespace {

struct LinBwd {
  Mat d, A, W;
  PairPlan plan;
  Reduce dA, dW;
  float* colp;
  size_t bytes;
};
LinBwd lin_bwd_layout(int dtype, const void* dout, const void* A, const void* W, int M, int N, int K, void* ws) {
  Carver cv{static_cast<uint8_t*>(ws)};
  LinBwd l;
  l.d = operand(dtype, dout, M, N, cv);
  l.A = operand(dtype, A, M, K, cv);
  l.W = operand(dtype, W, N, K, cv);
  const Product da{M, K, 1, ceil_div(N, tg::kBK)}, dw{N, K, 1, ceil_div(M, tg::kBK)};
  l.plan = plan_pair(dtype, da, dw);
  l.dA = plan_reduce(dtype, da, l.plan.splits[0], false, cv);
  l.dW = plan_reduce(dtype, dw, l.plan.splits[1], false, cv);
  l.colp = cv.take<float>((size_t)col_strips(M, N) * N * 4);
  l.bytes = cv.used;
  return l;
}

}  // namespace

size_t linear_bwd_workspace(int M, int N, int K, int dtype) {
  return M == 0 ? 0 : lin_bwd_layout(dtype, nullptr, nullptr, nullptr, M, N, K, nullptr).bytes;
}

cudaError_t linear_bwd(int dtype, const void* dout, const void* A, const void* W, void* dA, void* dW, float* dbias,
                       int M, int N, int K, void* ws, int* status, int num_sms, cudaStream_t s) {
  if (M == 0) {
    JEPA_TRY_CUDA(zero(dW, elem(dtype) * (size_t)N * K, s));
    return zero(dbias, sizeof(float) * (size_t)N, s);
  }
  const LinBwd l = lin_bwd_layout(dtype, dout, A, W, M, N, K, ws);
  Fills f{};
  if (dA != nullptr || dW != nullptr) add_fill(f, dout, l.d);
  if (dA != nullptr) add_fill(f, W, l.W);
  if (dW != nullptr) add_fill(f, A, l.A);
  JEPA_TRY_CUDA(fill(dtype, f, s));
  Job jobs[2];
  for (int k = 0; k < 2; ++k) {
    // dA = dout W, dW = dout^T A
    void* out = k == 0 ? dA : dW;
    if (out == nullptr) continue;
    const Mat& b = k == 0 ? l.W : l.A;
    const Reduce& rd = k == 0 ? l.dA : l.dW;
    const int rows = k == 0 ? M : N;
    Job& j = jobs[k] = base_job(rows, K, tg::kBN);
    set_k(j, k == 0 ? N : M, 1, rd.splits);
    JEPA_TRY_CUDA(k == 0 ? map_k(&j.a[0], l.d) : map_mn(&j.a[0], l.d));
    JEPA_TRY_CUDA(map_mn(&j.b[0], b));
    j.a_mn = k;
    j.a_plane = (int)l.d.plane_rows;
    j.b_plane = (int)b.plane_rows;
    JEPA_TRY_CUDA(reduce_output(dtype, rd, j, 0, out, rd.slab[0], false));
  }
  JEPA_TRY_CUDA(gemm_reduce(dtype, dA != nullptr ? &jobs[0] : nullptr, dW != nullptr ? &jobs[1] : nullptr, l.plan, status,
                            num_sms, s));
  Finish q{};
  if (dA != nullptr) add_slab_sum(q, l.dA, 0, jobs[0].splits, jobs[0].slab_rows, dA, M, K);
  if (dW != nullptr) add_slab_sum(q, l.dW, 0, jobs[1].splits, jobs[1].slab_rows, dW, N, K);
  if (dbias != nullptr) {
    const int strips = col_strips(M, N);
    JEPA_TRY_CUDA(col_strip(dtype, dout, M, N, strips, strips == 1 ? dbias : l.colp, s));
    if (strips > 1) add_part_sum(q, l.colp, dbias, N, strips, N);
  }
  return finish(dtype, q, nullptr, s);
}

}  // namespace jepa
