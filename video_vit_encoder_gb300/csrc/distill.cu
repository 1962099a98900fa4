// Distillation of a linear classifier from a teacher's top logits: the kernels
// beside the products.
//
// Of the classifier's z = x W^T + b only the K entries of a row that the teacher
// names are wanted one by one.  Forward the product's epilogue picks them out of
// its tiles, for which they are sorted by column first (products of their own
// would read M K rows of W: 4096 x 1024 x 32768 with K = 64 100 us beside the
// product's 142); a few rows have products of their own (few_rows.cu).  Backward the tiles leave
// dloss tau exp(z / tau - lse) and the entries are written over it afterwards, from
// z in fp32, so that the difference from the teacher's probability is rounded once.
//
// The products bound both (4096 x 1024 x 32768 with K = 64: forward 163 of 174 us, of which
// picking takes 16; backward 494 of 509); these kernels' 8 to 11 us each are latency and,
// of the sorts, shared memory.
#include "row_stats.cuh"

namespace jepa {

namespace {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// One row of the teacher, by a warp: the maximum and the sum of exp((t - max) /
// tau) of the entries that count.  kind 0: none has mass; -1: an id that is neither a
// class nor ignore_index.  An infinite or NaN logit gives a NaN sum.
struct Teacher {
  float max, sum;
  int kind;
};
template <typename TT>
__device__ __forceinline__ Teacher teacher_row(const TT* top, const int64_t* ids, int K, int V, long ignore, float inv_tau,
                                               int lane) {
  Teacher r;
  float m = -INFINITY, bad = 0.f;
  bool nan = false;
  for (int j = lane; j < K; j += 32) {
    const long id = ids[j];
    if (id == ignore) continue;
    if (id < 0 || id >= V) {
      bad = 1.f;
      continue;
    }
    const float t = DT<TT>::to(top[j]);
    nan |= t != t;
    m = fmaxf(m, t);
  }
  r.max = warp_max(m);
  bad = warp_max(bad);
  if (__any_sync(0xffffffffu, nan)) r.max = NAN;
  float s = 0.f;
  if (r.max != -INFINITY)
    for (int j = lane; j < K; j += 32) {
      const long id = ids[j];
      if (id != ignore && id >= 0 && id < V) s += expf((DT<TT>::to(top[j]) - r.max) * inv_tau);
    }
  r.sum = warp_sum(s);
  r.kind = bad > 0.f ? -1 : (r.max == -INFINITY ? 0 : 1);
  return r;
}

// Sorts a warp's n values in shared memory (n a power of 2 of at least 2).
template <typename K>
__device__ __forceinline__ void warp_sort(K* v, int n, int lane) {
  for (int size = 2; size <= n; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {
      __syncwarp();
      for (int i = lane; i < n / 2; i += 32) {
        const int lo = (i & ~(step - 1)) * 2 | (i & (step - 1)), hi = lo | step;
        const K a = v[lo], b = v[hi];
        if ((a > b) == ((lo & size) == 0)) {
          v[lo] = b;
          v[hi] = a;
        }
      }
    }
  __syncwarp();
}
__host__ __device__ constexpr int power_of_2(int n) {
  int p = 2;
  while (p < n) p *= 2;
  return p;
}

// A warp a row: its entries sorted by tg::hit_key, those that are out last, and
// where those of each half and run of column tiles begin.
constexpr int kRowWarps = 4;
__global__ void __launch_bounds__(32 * kRowWarps) hits_kernel(const int64_t* __restrict__ ids, int M, int V, int K, long ignore,
                                                              int run, int runs, uint32_t* __restrict__ hits,
                                                              uint16_t* __restrict__ starts, float* __restrict__ z) {
  extern __shared__ uint64_t keys[];   // of each warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = power_of_2(K);
  const long row = (long)blockIdx.x * kRowWarps + warp;
  if (row >= M) return;
  uint64_t* mine = keys + warp * n;
  for (int j = lane; j < n; j += 32) {
    const long id = j < K ? ids[row * K + j] : -1;
    const bool in = id != ignore && id >= 0 && id < V;
    mine[j] = (uint64_t)(in ? tg::hit_key((uint32_t)id) : 0xffffffffu) << 32 | (uint32_t)j;
    if (j < K && !in) z[row * K + j] = 0.f;
  }
  warp_sort(mine, n, lane);
  for (int j = lane; j < K; j += 32) {
    const uint32_t col = (uint32_t)(mine[j] >> 32) & 0x7fffffffu;
    hits[row * K + j] = tg::hit_word(col % (uint32_t)(run * tg::kBN), (uint32_t)mine[j]);   // those that are out are not read
  }
  for (int i = lane; i < 2 * (runs + 1); i += 32) {
    const int half = i > runs, r = half ? i - runs - 1 : i;
    // the end of the left halves is where the right ones begin, the end of those where entries are out
    const uint32_t key = r < runs ? tg::hit_key((uint32_t)(r * run * tg::kBN + half * (tg::kBN / 2))) : (half ? 0xffffffffu : 1u << 31);
    int lo = 0, hi = K;   // mine[lo ..] are from key on
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if ((uint32_t)(mine[mid] >> 32) < key) lo = mid + 1;
      else hi = mid;
    }
    starts[row * 2 * (runs + 1) + i] = (uint16_t)lo;
  }
}

// A row's sum p (log p - (z / tau - lse)), by a warp: entry by entry, or what the logits have in common would be
// taken off lse only after the sum, of which it takes digits.
template <typename TT>
__device__ __forceinline__ float row_term(const Teacher& t, const TT* top, const int64_t* ids, const float* z, float lse, int K,
                                          int V, long ignore, float inv_tau, int lane) {
  const float log_sum = logf(t.sum);
  float term = 0.f;
  for (int j = lane; j < K; j += 32) {
    const long id = ids[j];
    if (id == ignore || id < 0 || id >= V) continue;
    const float a = (DT<TT>::to(top[j]) - t.max) * inv_tau;
    const float p = expf(a) / t.sum;
    if (!(p == 0.f)) term += p * ((a - log_sum) - (z[j] * inv_tau - lse));   // a class without mass adds nothing, whatever its z
  }
  return warp_sum(term);
}
// A warp a row: its parts, every 32nd a lane, then its entries.
template <typename TT>
__global__ void __launch_bounds__(kBlock) distill_join_kernel(const float2* __restrict__ ms, int parts, int M,
                                                              const TT* __restrict__ top, const int64_t* __restrict__ ids,
                                                              const float* __restrict__ z, int V, int K, long ignore,
                                                              float tau, float* __restrict__ loss,
                                                              float* __restrict__ lse_out, int* status) {
  const int lane = threadIdx.x & 31;
  const long row = (long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= M) return;
  Ms a{-INFINITY, 0.f, 0.f};
#pragma unroll 4
  for (int k = lane; k < parts; k += 32) {
    const float2 q = __ldg(ms + (size_t)k * M + row);
    ms_join(a, q.x, q.y, 0.f);
  }
  const float inv_tau = 1.0f / tau;
  const Teacher t = teacher_row(top + row * K, ids + row * K, K, V, ignore, inv_tau, lane);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m = __shfl_xor_sync(0xffffffffu, a.m, o), v = __shfl_xor_sync(0xffffffffu, a.s, o);
    ms_join(a, m, v, 0.f);
  }
  const float lse = __shfl_sync(0xffffffffu, (a.m + log2f(a.s)) * 0.69314718055994531f, 0);   // ln(2^m s)
  const float term = row_term(t, top + row * K, ids + row * K, z + row * K, lse, K, V, ignore, inv_tau, lane);
  if (lane != 0) return;
  lse_out[row] = lse;
  if (loss != nullptr) loss[row] = t.kind == 0 ? 0.f : (t.kind < 0 ? NAN : tau * tau * term);
  if (t.kind < 0) atomicOr(status, DEV_BAD_INDEX);
}

// A warp a row.  Entries of one class are joined into the first of them.
template <typename TT>
__global__ void __launch_bounds__(32 * kRowWarps) teacher_kernel(const TT* __restrict__ top,
                                                                 const int64_t* __restrict__ ids,
                                                                 const float* __restrict__ dloss, int M, int V, int K,
                                                                 long ignore, float tau, int64_t* __restrict__ label,
                                                                 float* __restrict__ dl, int* __restrict__ cls,
                                                                 float* __restrict__ prob, long long* __restrict__ acc,
                                                                 int* status) {
  extern __shared__ uint64_t keys[];   // of each warp: (class, place), sorted
  if (acc != nullptr)
    for (int v = blockIdx.x * 32 * kRowWarps + threadIdx.x; v < 2 * V; v += gridDim.x * 32 * kRowWarps) acc[v] = 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = power_of_2(K);
  const long row = (long)blockIdx.x * kRowWarps + warp;
  if (row >= M) return;
  uint64_t* mine = keys + warp * n;
  top += row * K;
  ids += row * K;
  const float inv_tau = 1.0f / tau;
  const Teacher t = teacher_row(top, ids, K, V, ignore, inv_tau, lane);
  auto p_of = [&](int j) { return expf((DT<TT>::to(top[j]) - t.max) * inv_tau) / t.sum; };
  for (int j = lane; j < n; j += 32) {
    const long id = j < K ? ids[j] : ignore;
    const bool in = t.kind == 1 && id != ignore;   // then every other id is a class
    mine[j] = (uint64_t)(in ? (uint32_t)id : 0xffffffffu) << 32 | (uint32_t)j;
  }
  warp_sort(mine, n, lane);
  for (int i = lane; i < n; i += 32) {
    const uint32_t c = (uint32_t)(mine[i] >> 32), j = (uint32_t)mine[i];
    if (j >= K) continue;
    const bool first = c != 0xffffffffu && (i == 0 || (uint32_t)(mine[i - 1] >> 32) != c);
    float p = 0.f;
    if (first)
      for (int k = i; k < n && (uint32_t)(mine[k] >> 32) == c; ++k) p += p_of((uint32_t)mine[k]);
    cls[row * K + j] = first ? (int)c : -1;
    prob[row * K + j] = p;
  }
  if (lane == 0) {
    label[row] = t.kind == 1 ? 0 : -1;
    // a teacher without a finite maximum makes its row's gradient NaN
    dl[row] = t.sum < INFINITY ? dloss[row] * tau : NAN;
    if (t.kind < 0) atomicOr(status, DEV_BAD_INDEX);
  }
}

// The teacher's part of dbias is summed in whole numbers, whose sum has no order: of
// 2^-shift of the unit, and of 2^-2 shift for what that leaves of an entry (nothing,
// unless its dloss times its probability is below 2^(24 - shift) of the unit), so that
// an entry keeps fp32's accuracy next to a row whose dloss is 2^(2 shift - 24) times as
// large.  With HELD a block sums those of a few classes in shared memory first (5555
// rows of 62 entries over 80 classes in global memory 64 us).
constexpr int kHeldClasses = 2048;
template <typename T, bool SPLIT, bool HELD>
__global__ void __launch_bounds__(kBlock) put_kernel(const __grid_constant__ DistillPut q) {
  __shared__ unsigned long long held[HELD ? kHeldClasses : 1];
  if constexpr (HELD) {
    for (int v = threadIdx.x; v < q.V; v += kBlock) held[v] = 0;
    __syncthreads();
  }
  for (long i = (long)blockIdx.x * kBlock + threadIdx.x; i < (long)q.M * q.K; i += (long)gridDim.x * kBlock) {
    const int cls = q.cls[i], c = cls - q.v0;
    if (cls < 0 || c < 0 || c >= q.n) continue;
    const long row = i / q.K;
    const float dl = q.dl[row], p = q.prob[i];
    float ds = exp2f(fmaf(q.z[i], q.z_scale, -q.lse[row] * 1.4426950408889634f)) - p;
    if constexpr (SPLIT) {
      ds *= dl;
      __nv_bfloat16 h[3];
      h[0] = __float2bfloat16_rn(ds);
      float rem = ds - __bfloat162float(h[0]);
      if (!(fabsf(ds) < INFINITY)) rem = 0.f;
      h[1] = __float2bfloat16_rn(rem);
      h[2] = __float2bfloat16_rn(rem - __bfloat162float(h[1]));
#pragma unroll
      for (int k = 0; k < 3; ++k) reinterpret_cast<__nv_bfloat16*>(q.dz)[(k * q.plane_rows + row) * q.ld + c] = h[k];
    } else {
      reinterpret_cast<T*>(q.dz)[row * q.ld + c] = DT<T>::from(ds * (dl / *q.unit * q.factor));
    }
    if (q.acc != nullptr && fabsf(dl) < INFINITY) {
      const float t = ldexpf(p * (dl / *q.unit), q.shift);
      const long long a = __float2ll_rn(t);
      const float left = t - (float)a;   // exact: a is t's own digits, or t < 2^24
      if constexpr (HELD) atomicAdd(held + cls, (unsigned long long)a);
      else atomicAdd(reinterpret_cast<unsigned long long*>(q.acc + cls), (unsigned long long)a);
      if (left != 0.f)
        atomicAdd(reinterpret_cast<unsigned long long*>(q.acc + q.V + cls), (unsigned long long)__float2ll_rn(ldexpf(left, q.shift)));
    }
  }
  if constexpr (HELD) {
    __syncthreads();
    for (int v = threadIdx.x; v < q.V; v += kBlock)
      if (held[v] != 0) atomicAdd(reinterpret_cast<unsigned long long*>(q.acc + v), held[v]);
  }
}
template <typename T, bool SPLIT>
cudaError_t put_t(const DistillPut& q, int num_sms, cudaStream_t s) {
  const long blocks = ((long)q.M * q.K + kBlock - 1) / kBlock;
  if (q.acc != nullptr && q.V <= kHeldClasses) {
    const long most = 4l * num_sms;
    put_kernel<T, SPLIT, true><<<(unsigned)(blocks < most ? blocks : most), kBlock, 0, s>>>(q);
  } else {
    put_kernel<T, SPLIT, false><<<(unsigned)blocks, kBlock, 0, s>>>(q);
  }
  return cudaGetLastError();
}

template <typename TT>
cudaError_t join_t(const DistillArgs& a, const float2* ms, int parts, const float* z, float* loss, float* lse, cudaStream_t s) {
  const CeArgs& c = a.ce;
  distill_join_kernel<TT><<<(c.M + kWarps - 1) / kWarps, kBlock, 0, s>>>(ms, parts, c.M, (const TT*)a.top, a.ids, z, c.V, a.K,
                                                                         a.ignore_index, a.tau, loss, lse, c.status);
  return cudaGetLastError();
}
template <typename TT>
cudaError_t teacher_t(const DistillArgs& a, const float* dloss, int64_t* label, float* dl, int* cls, float* prob,
                      long long* acc, cudaStream_t s) {
  const unsigned blocks = (a.ce.M + kRowWarps - 1) / kRowWarps;
  teacher_kernel<TT><<<blocks, 32 * kRowWarps, kRowWarps * power_of_2(a.K) * 8, s>>>(
      (const TT*)a.top, a.ids, dloss, a.ce.M, a.ce.V, a.K, a.ignore_index, a.tau, label, dl, cls, prob, acc, a.ce.status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t distill_hits(const DistillArgs& a, int run, int runs, uint32_t* hits, uint16_t* starts, float* z, cudaStream_t s) {
  const unsigned blocks = (a.ce.M + kRowWarps - 1) / kRowWarps;
  hits_kernel<<<blocks, 32 * kRowWarps, kRowWarps * power_of_2(a.K) * 8, s>>>(a.ids, a.ce.M, a.ce.V, a.K, a.ignore_index, run,
                                                                               runs, hits, starts, z);
  return cudaGetLastError();
}

cudaError_t distill_join(const DistillArgs& a, const float2* ms, int parts, const float* z, float* loss, float* lse,
                         cudaStream_t s) {
  if (a.top_dtype == DTYPE_F32) return join_t<float>(a, ms, parts, z, loss, lse, s);
  return a.top_dtype == DTYPE_F16 ? join_t<__half>(a, ms, parts, z, loss, lse, s)
                                  : join_t<__nv_bfloat16>(a, ms, parts, z, loss, lse, s);
}

cudaError_t distill_teacher(const DistillArgs& a, const float* dloss, int64_t* label, float* dl, int* cls, float* prob,
                            long long* acc, cudaStream_t s) {
  if (a.top_dtype == DTYPE_F32) return teacher_t<float>(a, dloss, label, dl, cls, prob, acc, s);
  return a.top_dtype == DTYPE_F16 ? teacher_t<__half>(a, dloss, label, dl, cls, prob, acc, s)
                                  : teacher_t<__nv_bfloat16>(a, dloss, label, dl, cls, prob, acc, s);
}

cudaError_t distill_put(int dtype, const DistillPut& q, int num_sms, cudaStream_t s) {
  if (dtype == DTYPE_F32) return put_t<float, true>(q, num_sms, s);
  return dtype == DTYPE_F16 ? put_t<__half, false>(q, num_sms, s) : put_t<__nv_bfloat16, false>(q, num_sms, s);
}

}  // namespace jepa
