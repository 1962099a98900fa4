// Embedding of tokens, out[i] = scale table[token i], and the table's gradient.
//
// The gradient of a row is a sum over the places of its token, which is made in
// an order that the tokens alone decide, whatever the schedule: the tokens are
// sorted, chunks of 16 sorted places are summed on their own, in the places' order,
// and runs of one token that cross a chunk's border are joined from the chunks'
// parts, a short run's in order, a long one's by 32 warps that take every 32nd.
//
// Both are bound by memory where they are large: 65536 x 1024 of 131072 rows of bf16
// from and to fp32 takes 50 us forward (0.91 of the copy bandwidth) and 107 backward
// (0.74: 25 of the sort, with zeros written beside it, 65 of the sums and the other
// zeros, and rows that are written twice).  The gradient of 8190 x 768 over 50021 (26 us,
// 0.50) is three latencies, the sort's 14 us the longest.
#include <algorithm>

#include "decoder.h"

namespace jepa {

namespace {

constexpr int kBlock = 256;

unsigned blocks_for(long n, int block) { return (unsigned)((n + block - 1) / block); }
size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// N consecutive values as floats, from and to memory that is aligned to them.
template <typename T, int N> struct alignas(sizeof(T) * N) Pack { T v[N]; };
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  const Pack<T, N> q = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = DT<T>::to(q.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
  Pack<T, N> q;
#pragma unroll
  for (int i = 0; i < N; ++i) q.v[i] = DT<T>::from(v[i]);
  *reinterpret_cast<Pack<T, N>*>(p) = q;
}

// ----------------------------------------------------------------------------- forward
// 2^lg neighbouring threads take R rows, a thread K times V columns of each.
template <typename TT, typename TO, int V, int R, int K>
__global__ void __launch_bounds__(kBlock) embed_kernel(const __grid_constant__ EmbedArgs a, int lg,
                                                       const TT* __restrict__ table, TO* __restrict__ out) {
  const long row = (((long)blockIdx.x * kBlock + threadIdx.x) >> lg) * R;
  const int step = V << lg, c = (int)blockIdx.y * K * step + (threadIdx.x & ((1 << lg) - 1)) * V;
  if (c >= a.dim) return;
  long t[R];
#pragma unroll
  for (int r = 0; r < R; ++r) t[r] = row + r < a.n ? a.tokens[row + r] : a.ignore_index;
  float v[R][K][V];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool in = t[r] >= 0 && t[r] < a.vocab && t[r] != a.ignore_index, bad = !in && t[r] != a.ignore_index;
    const TT* src = table + t[r] * a.dim + c;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (in && c + k * step < a.dim) {
        load_n<TT, V>(src + k * step, v[r][k]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[r][k][j] = bad ? NAN : 0.f;
      }
    }
    if (bad && c == 0) atomicOr(a.status, DEV_BAD_INDEX);
  }
  out += row * a.dim + c;
#pragma unroll
  for (int r = 0; r < R; ++r, out += a.dim) {
    if (row + r >= a.n) break;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[r][k][j] *= a.scale;
      if (c + k * step < a.dim) store_n<TO, V>(out + k * step, v[r][k]);
    }
  }
}

// ----------------------------------------------------------------------------- sort
// Stable sort of the places by token, from the lowest digit up, by the blocks of
// one cluster, each with a consecutive part of the places: a block counts its
// digits, the counts are exchanged through distributed shared memory, and each
// place goes to where its digit's run of its block begins plus its rank among
// those of the same digit, which keeps equal tokens in order.  Digits of 9 bits:
// two passes for up to 2^18 - 1 rows of the table.  Places without a row (ignored,
// or outside the table) get the key `vocab` and end up last.
//
// The other clusters of the launch write zeros into the first rows of the
// gradient meanwhile, about as many as the sort takes time for; rows that have
// tokens are written again afterwards.  The rest is left to the next kernel's
// blocks, to which the sort tells which rows have none (a bit a row).
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kMaxRanks = 16;
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits, kItems = 8, kTile = kSortThreads * kItems;
struct SortArgs {
  const int64_t* tokens;
  int n, vocab;
  long ignore_index;
  uint32_t *keys[2], *places[2];   // pass p writes [p & 1]
  int passes, bits;                // bits of a digit
  int ranks;                       // blocks that sort
  int* joins;                      // two counts that are set to 0
  uint32_t* some;                  // a bit of each row of the table: whether it has places; null: not wanted
  int* status;
  uint8_t* zeros;                  // what is filled
  size_t zero_bytes;
};
// Zeros of n bytes (whole elements) by `threads` threads: 16 bytes at a time
// between the first and the last address that allows it.
__device__ __forceinline__ void write_zeros(uint8_t* p, size_t n, size_t me, size_t threads) {
  const size_t head = min((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16, n), vecs = (n - head) / 16;
  uint4* v = reinterpret_cast<uint4*>(p + head);
  for (size_t i = me; i < vecs; i += threads) v[i] = make_uint4(0, 0, 0, 0);
  if (me < 8) {   // two bytes each
    if (2 * me < head) *reinterpret_cast<uint16_t*>(p + 2 * me) = 0;
    const size_t tail = head + vecs * 16 + 2 * me;
    if (tail < n) *reinterpret_cast<uint16_t*>(p + tail) = 0;
  }
}
// Kernels that are launched before the one they follow has ended begin with this.
__device__ __forceinline__ void follow() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void lead() { asm volatile("griddepcontrol.launch_dependents;"); }
struct SortShared {
  uint2 held[kTile];                     // key and place of the block's part, between passes
  uint16_t warps[kSortWarps][kDigits];   // of each warp of the tile, then before it
  int count[kDigits];                    // of the block: the others read it
  int next[kDigits];                     // where the block's next place of a digit goes
  int sums[kSortWarps];
};
__device__ __forceinline__ uint32_t key_of(const SortArgs& a, long i, int* bad) {
  const long t = a.tokens[i];
  if (t == a.ignore_index) return a.vocab;
  if (t < 0 || t >= a.vocab) {
    *bad = 1;
    return a.vocab;
  }
  return (uint32_t)t;
}
// The lanes whose digit is this one's.
__device__ __forceinline__ uint32_t same_digit(uint32_t d, bool in) {
  uint32_t peers = __ballot_sync(0xffffffffu, in);
#pragma unroll
  for (int b = 0; b < kDigitBits; ++b) {
    const bool one = d >> b & 1;
    const uint32_t set = __ballot_sync(0xffffffffu, one);
    peers &= one ? set : ~set;
  }
  return peers;
}
// Where the block's places of each digit begin, from all blocks' sm.count, which
// stay as they are until the next cluster_sync().
__device__ __forceinline__ void exchange_counts(const SortArgs& a, SortShared& sm, int rank) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cluster_sync();
  // exclusive sums over the digits, then over the blocks before this one
  int all = 0, before = 0;
  if (tid < kDigits) {
    const uint32_t mine = smem_u32(&sm.count[tid]);
#pragma unroll 8
    for (int r = 0; r < a.ranks; ++r) {
      int c;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c) : "r"(mapa_shared(mine, r)) : "memory");
      before += r < rank ? c : 0;
      all += c;
    }
  }
  int x = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm.sums[warp] = x;
  __syncthreads();
  if (tid < kDigits) {
    for (int w = 0; w < warp; ++w) x += sm.sums[w];
    sm.next[tid] = x - all + before;
  }
  __syncthreads();
}
__device__ void sort_places(const SortArgs& a, SortShared& sm) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank(), digits = 1 << a.bits;
  // this block's places; parts are multiples of a warp's 32
  const int part = ((a.n + a.ranks - 1) / a.ranks + 31) / 32 * 32;
  const int begin = min(rank * part, a.n), end = min(begin + part, a.n);
  // at most a tile a block: its counts are the block's, and places stay in shared memory between passes
  const bool one = part <= kTile;
  const int items = one ? (part + kSortThreads - 1) / kSortThreads : kItems;   // places of a thread in a tile
  const int tile_size = items * kSortThreads;
  int bad = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    const uint32_t* keys = a.keys[(pass & 1) ^ 1];
    const uint32_t* places = a.places[(pass & 1) ^ 1];
    auto key_at = [&](int i) { return pass == 0 ? key_of(a, i, &bad) : __ldcg(keys + i); };
    if (!one) {
      if (tid < kDigits) sm.count[tid] = 0;
      __syncthreads();
      for (int i = begin + tid; i < end; i += kTile) {
        uint32_t k[kItems];
#pragma unroll
        for (int j = 0; j < kItems; ++j) k[j] = i + j * kSortThreads < end ? key_at(i + j * kSortThreads) : 0u;
#pragma unroll
        for (int j = 0; j < kItems; ++j)
          if (i + j * kSortThreads < end) atomicAdd(&sm.count[(k[j] >> shift) & (digits - 1)], 1);
      }
      __syncwarp();
      exchange_counts(a, sm, rank);
    }
    for (int base = begin; base < end || (one && base == begin); base += tile_size) {
      for (int d = lane; d < digits; d += 32) sm.warps[warp][d] = 0;
      __syncwarp();
      uint32_t key[kItems], place[kItems];
      int at[kItems];
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        const int i = base + (warp * items + j) * 32 + lane;
        key[j] = place[j] = 0u;
        if (j >= items || i >= end) continue;
        if (pass == 0) {
          key[j] = key_of(a, i, &bad);
          place[j] = (uint32_t)i;
        } else if (one) {
          const uint2 q = sm.held[i - begin];
          key[j] = q.x;
          place[j] = q.y;
        } else {
          key[j] = __ldcg(keys + i);
          place[j] = __ldcg(places + i);
        }
      }
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        if (j >= items) break;
        const bool in = base + (warp * items + j) * 32 + lane < end;
        const uint32_t d = (key[j] >> shift) & (digits - 1);
        const uint32_t same = same_digit(d, in);
        const int count = in ? sm.warps[warp][d] : 0;
        __syncwarp();
        at[j] = count + __popc(same & ((1u << lane) - 1));
        if (in && lane == __ffs(same) - 1) sm.warps[warp][d] = (uint16_t)(count + __popc(same));
        __syncwarp();
      }
      __syncthreads();
      int tile = 0;
      if (tid < digits) {
        uint16_t c[kSortWarps];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) c[w] = sm.warps[w][tid];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
          sm.warps[w][tid] = (uint16_t)tile;
          tile += c[w];
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kItems; ++j)
        if (j < items && base + (warp * items + j) * 32 + lane < end) at[j] += sm.warps[warp][(key[j] >> shift) & (digits - 1)];
      if (one) {
        if (tid < kDigits) sm.count[tid] = tile;
        __syncwarp();
        exchange_counts(a, sm, rank);
      }
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        if (j >= items || base + (warp * items + j) * 32 + lane >= end) continue;
        const int to = sm.next[(key[j] >> shift) & (digits - 1)] + at[j];
        if (one && pass + 1 < a.passes) {   // everybody has read what was held: the counts came after it
          const int owner = to / part;
          const uint32_t dst = mapa_shared(smem_u32(&sm.held[to - owner * part]), owner);
          asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(key[j]), "r"(place[j]) : "memory");
        } else {
          a.keys[pass & 1][to] = key[j];
          a.places[pass & 1][to] = place[j];
        }
      }
      __syncthreads();
      if (!one && tid < digits) sm.next[tid] += tile;
      __syncthreads();
    }
    __syncwarp();
    cluster_sync();   // the pass's places are there, and nobody reads this pass's counts any more
  }
  const uint32_t* sorted = a.keys[(a.passes - 1) & 1];
  if (a.some != nullptr)
    for (int i = begin + tid; i < end; i += kSortThreads) {
      const uint32_t k = __ldcg(sorted + i);
      if (k < a.vocab && (i == 0 || __ldcg(sorted + i - 1) != k)) atomicOr(a.some + k / 32, 1u << k % 32);
    }
  if (bad) atomicOr(a.status, DEV_BAD_INDEX);
}
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ SortArgs a) {
  lead();
  extern __shared__ __align__(16) uint8_t shared[];
  SortShared& sm = *reinterpret_cast<SortShared*>(shared);
  if (blockIdx.x < a.ranks) {
    if (blockIdx.x == 0 && threadIdx.x < 2) a.joins[threadIdx.x] = 0;
    if (a.some != nullptr)
      for (int i = blockIdx.x * kSortThreads + threadIdx.x; i < (a.vocab + 31) / 32; i += a.ranks * kSortThreads) a.some[i] = 0;
    cluster_sync();   // every block's shared memory is there
    sort_places(a, sm);
    return;
  }
  const long blocks = gridDim.x - a.ranks, me = (blockIdx.x - a.ranks) * (long)kSortThreads + threadIdx.x;
  write_zeros(a.zeros, a.zero_bytes, me, blocks * kSortThreads);
}

// ----------------------------------------------------------------------------- sums
constexpr int kChunk = 16;       // sorted places that are summed on their own
constexpr int kJoin = 1024;      // threads of a block that joins
struct SumArgs {
  const uint32_t *keys, *places;
  int n, dim, vocab;
  float scale;
  float* part;    // [chunks][2][dim]: what the chunk has of a run that began before it, and of one that goes on after it
  int *joins, *starts[2];   // how many runs go on into other chunks, and the chunks in which they begin: short ones, long ones
  const uint32_t* some;     // the rows that have places
  int zero_row, zero_rows;  // from which row on zeros are still to be written, and how many a block looks at
  size_t row_bytes;
  unsigned chunk_blocks;    // the blocks that sum come first, chunk_cols of them side by side
  unsigned chunk_cols;
  int long_chunks;          // as many after its first make a run a long one
};
// A thread sums V columns of a chunk's places, 2^lg neighbouring threads a chunk.
// A run that lies within the chunk is a row of the gradient.
template <typename TO, typename TT, int V>
__global__ void __launch_bounds__(kBlock, 4) chunk_kernel(const __grid_constant__ SumArgs a, int lg,
                                                          const TO* __restrict__ dout, TT* __restrict__ dtable) {
  constexpr int kAt = V * sizeof(TO) <= 4 ? 16 : 8;   // rows on their way at a time
  follow();
  lead();
  if (blockIdx.x >= a.chunk_blocks) {   // rows without places, a warp a row
    const int first = a.zero_row + (int)(blockIdx.x - a.chunk_blocks) * a.zero_rows, end = min(first + a.zero_rows, a.vocab);
    for (int r = first + (threadIdx.x >> 5); r < end; r += kBlock / 32)
      if (!(a.some[r / 32] >> r % 32 & 1))   // written by the kernel before, which may still run when this one begins: no __ldg
        write_zeros(reinterpret_cast<uint8_t*>(dtable) + (size_t)r * a.row_bytes, a.row_bytes, threadIdx.x & 31, 32);
    return;
  }
  const long chunk = ((long)(blockIdx.x / a.chunk_cols) * kBlock + threadIdx.x) >> lg;
  const int c = ((int)(blockIdx.x % a.chunk_cols << lg) + (threadIdx.x & ((1 << lg) - 1))) * V;
  const int e0 = (int)min(chunk * kChunk, (long)a.n), e1 = min(e0 + kChunk, a.n);
  if (e0 >= e1 || c >= a.dim) return;
  dout += c;
  uint32_t past = e0 > 0 ? a.keys[e0 - 1] : 0xffffffffu;   // the key of a run that began before this chunk, if it goes on here
  float s[V] = {};
#pragma unroll 1
  for (int e = e0; e < e1; e += kAt) {
    uint32_t k[kAt + 1], at[kAt];   // the arrays go on to the end of the last chunk
#pragma unroll
    for (int j = 0; j < kAt; j += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(a.keys + e + j), y = *reinterpret_cast<const uint4*>(a.places + e + j);
      k[j] = x.x; k[j + 1] = x.y; k[j + 2] = x.z; k[j + 3] = x.w;
      at[j] = y.x; at[j + 1] = y.y; at[j + 2] = y.z; at[j + 3] = y.w;
    }
    k[kAt] = e + kAt < a.n ? a.keys[e + kAt] : 0xffffffffu;   // what comes after
    Pack<TO, V> v[kAt];
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      if (e + j >= e1) k[j] = 0xffffffffu;
      // without a condition, or the compiler puts each load where its value is used
      v[j] = *reinterpret_cast<const Pack<TO, V>*>(dout + (size_t)(k[j] < a.vocab ? at[j] : 0u) * a.dim);
    }
#pragma unroll
    for (int j = 0; j < kAt; ++j) {
      if (k[j] >= a.vocab) return;
#pragma unroll
      for (int q = 0; q < V; ++q) s[q] += DT<TO>::to(v[j].v[q]);
      const bool same = k[j + 1] == k[j], goes_on = same && j == kAt - 1 && e + kAt >= e1, began = past == k[j];
      if (same && !goes_on) continue;
      if (!began && !goes_on) {
#pragma unroll
        for (int q = 0; q < V; ++q) s[q] *= a.scale;
        store_n<TT, V>(dtable + (size_t)k[j] * a.dim + c, s);
      } else {
        store_n<float, V>(a.part + ((size_t)chunk * 2 + (began ? 0 : 1)) * a.dim + c, s);
        if (!began && c == 0) {   // the lists may have any order: each entry is a run of its own
          const long far = (long)e0 + (a.long_chunks + 1) * kChunk;
          const int is_long = far < a.n && a.keys[far] == k[j];
          a.starts[is_long][atomicAdd(a.joins + is_long, 1)] = (int)chunk;
        }
      }
      past = 0xffffffffu;
#pragma unroll
      for (int q = 0; q < V; ++q) s[q] = 0.f;
    }
  }
}
// Runs that cross chunks, 32 vectors of V columns at a time: short ones by a warp,
// long ones by a block, each of whose warps takes every 32nd part; all in a fixed
// order.
template <typename TT, int V>
__global__ void __launch_bounds__(kJoin) join_kernel(const __grid_constant__ SumArgs a, TT* __restrict__ dtable) {
  __shared__ float sm[kJoin / 32][32][V + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (a.dim / V + 31) / 32;
  follow();
  // how many of the 32 chunks from `first` on begin with key
  auto chunks_of = [&](long first, uint32_t key) {
    const long e = (first + lane) * kChunk;
    const uint32_t same = __ballot_sync(0xffffffffu, e < a.n && a.keys[e] == key);
    return same == 0xffffffffu ? 32 : __ffs(~same) - 1;
  };
  auto add_part = [&](float (&s)[V], long chunk, int slot, int c) {
    float v[V];
    load_n<float, V>(a.part + ((size_t)chunk * 2 + slot) * a.dim + c, v);
#pragma unroll
    for (int q = 0; q < V; ++q) s[q] += v[q];
  };
  auto store = [&](float (&s)[V], uint32_t key, int c) {
#pragma unroll
    for (int q = 0; q < V; ++q) s[q] *= a.scale;
    store_n<TT, V>(dtable + (size_t)key * a.dim + c, s);
  };
  const long longs = (long)a.joins[1] * groups, shorts = (long)a.joins[0] * groups;
  for (long item = blockIdx.x; item < longs; item += gridDim.x) {
    const int chunk = a.starts[1][item / groups], c = ((int)(item % groups) * 32 + lane) * V;
    const uint32_t key = a.keys[(chunk + 1) * kChunk];
    int end = chunk;   // the chunk in which the run ends: they begin with its key up to there
    for (int more = kJoin; more == kJoin; end += more) {
      const long e = (end + 1l + threadIdx.x) * kChunk;
      more = __syncthreads_count(e < a.n && a.keys[e] == key);
    }
    float s[V] = {};
    if (c < a.dim) {
      if (warp == 0) add_part(s, chunk, 1, c);
#pragma unroll 4
      for (int k = chunk + 1 + warp; k <= end; k += kJoin / 32) add_part(s, k, 0, c);
    }
#pragma unroll
    for (int q = 0; q < V; ++q) sm[warp][lane][q] = s[q];
    __syncthreads();
    if (warp == 0 && c < a.dim) {
      for (int w = 1; w < kJoin / 32; ++w)
#pragma unroll
        for (int q = 0; q < V; ++q) s[q] += sm[w][lane][q];
      store(s, key, c);
    }
    __syncthreads();
  }
  for (long item = (long)(gridDim.x - 1 - blockIdx.x) * (kJoin / 32) + warp; item < shorts; item += (long)gridDim.x * (kJoin / 32)) {
    const int chunk = a.starts[0][item / groups], c = ((int)(item % groups) * 32 + lane) * V;
    const uint32_t key = a.keys[(chunk + 1) * kChunk];
    const int more = chunks_of(chunk + 1, key);
    if (c >= a.dim) continue;
    float s[V] = {};
    add_part(s, chunk, 1, c);
#pragma unroll 4
    for (int k = 1; k <= more; ++k) add_part(s, chunk + k, 0, c);
    store(s, key, c);
  }
}

struct Layout {
  uint32_t *keys[2], *places[2];
  float* part;
  int *joins, *starts[2];
  uint32_t* some;
  size_t bytes;
};
Layout layout(int n, int dim, int vocab, void* ws) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t used = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = p + used;
    used += align256(bytes);
    return r;
  };
  Layout l;
  const size_t chunks = blocks_for(n, kChunk);
  for (int k = 0; k < 2; ++k) {
    l.keys[k] = reinterpret_cast<uint32_t*>(take(chunks * kChunk * 4));
    l.places[k] = reinterpret_cast<uint32_t*>(take(chunks * kChunk * 4));
  }
  l.part = reinterpret_cast<float*>(take(chunks * 2 * dim * 4));
  l.joins = reinterpret_cast<int*>(take(8));
  for (int k = 0; k < 2; ++k) l.starts[k] = reinterpret_cast<int*>(take(chunks * 4));
  l.some = reinterpret_cast<uint32_t*>(take(((size_t)vocab + 31) / 32 * 4));
  l.bytes = used;
  return l;
}

// The power of 2 of threads that share a row of `vecs` vectors, at most 2^most.
int group_of(int vecs, int most) {
  int lg = 0;
  while (lg < most && (1 << lg) < vecs) ++lg;
  return lg;
}
template <typename TT, typename TO, int V>
cudaError_t fwd_v(const EmbedArgs& a, const void* table, void* out, cudaStream_t s) {
  // four rows a thread where that still fills the GPU; of short vectors four of each row, too, which share what it takes
  // to find it (30000 x 777 in fp16 34 us; one of each of eight rows 48)
  constexpr int kCols = V * sizeof(TT) <= 4 ? 4 : 1;
  const int vecs = a.dim / V, lg = group_of((vecs + kCols - 1) / kCols, 8);
  const unsigned y = blocks_for(vecs, kCols << lg);
  const bool four = (long)a.n * vecs >= 4l * kCols * 1024 * a.num_sms;
  const dim3 g(blocks_for((long)blocks_for(a.n, four ? 4 : 1) << lg, kBlock), y);
  if (four) embed_kernel<TT, TO, V, 4, kCols><<<g, kBlock, 0, s>>>(a, lg, (const TT*)table, (TO*)out);
  else embed_kernel<TT, TO, V, 1, kCols><<<g, kBlock, 0, s>>>(a, lg, (const TT*)table, (TO*)out);
  return cudaGetLastError();
}
// A launch that may begin before the one before it has ended (follow()).
template <typename K, typename... A>
cudaError_t launch_next(K kern, unsigned blocks, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename TT, typename TO, int V>
cudaError_t bwd_v(SumArgs q, const void* dout, void* dtable, long num_sms, cudaStream_t s) {
  const long chunks = blocks_for(q.n, kChunk), vecs = q.dim / V;
  const int lg = group_of(vecs, 8);
  q.chunk_cols = blocks_for(vecs, 1 << lg);
  q.chunk_blocks = blocks_for(chunks << lg, kBlock) * q.chunk_cols;
  q.row_bytes = sizeof(TT) * q.dim;
  // A block that joins a long run takes 32 vectors of its columns: quicker than a warp, but where there may be many such
  // items they go in waves, and fewer runs are left to them.  With 8 | 32 chunks 8190 x 768 over 50021 in bf16 (512 chunks
  // of 3 groups) 26.3 | 29.7 us, 8000 x 4096 over 30000 in fp32 (500 of 32) 102 | 107, 30000 x 2048 over 50000 in fp32 (1875 of
  // 16) 119 | 121, 30000 x 777 over 30000 in fp16 (1875 of 25) 61.3 | 57.8.
  const long groups = (vecs + 31) / 32;
  q.long_chunks = chunks * groups <= 40000 ? 8 : 32;
  q.zero_rows = (int)std::max<size_t>(8, 65536 / q.row_bytes);
  const unsigned zero_blocks = blocks_for(q.vocab - q.zero_row, q.zero_rows);
  cudaError_t e = launch_next(chunk_kernel<TO, TT, V>, q.chunk_blocks + zero_blocks, kBlock, s, q, lg, (const TO*)dout, (TT*)dtable);
  if (e != cudaSuccess || chunks < 2) return e;
  // an SM takes one block that joins, so that one wave of them is best (65536 x 1024 over 131072 111 | 109 us with two | one)
  const long items = (chunks - 1) * groups;   // at most
  return launch_next(join_kernel<TT, V>, (unsigned)std::min((items + 31) / 32, num_sms), kJoin, s, q, (TT*)dtable);
}
bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

#define EMBED_TYPES(CALL)                                                                     \
  if (a.table_dtype == DTYPE_F32) return CALL(float, float, 4);                               \
  if (a.table_dtype == DTYPE_F16)                                                             \
    return a.out_dtype == DTYPE_F16 ? CALL(__half, __half, 8) : CALL(__half, float, 4);       \
  return a.out_dtype == DTYPE_BF16 ? CALL(__nv_bfloat16, __nv_bfloat16, 8) : CALL(__nv_bfloat16, float, 4);

cudaError_t embedding_fwd(const EmbedArgs& a, const void* table, void* out, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
#define CALL(TT, TO, V)                                                                    \
  (a.dim % V == 0 && aligned(table, V * sizeof(TT)) && aligned(out, V * sizeof(TO))        \
       ? fwd_v<TT, TO, V>(a, table, out, s)                                                \
       : (a.dim % 2 == 0 && aligned(table, 2 * sizeof(TT)) && aligned(out, 2 * sizeof(TO)) \
              ? fwd_v<TT, TO, 2>(a, table, out, s) : fwd_v<TT, TO, 1>(a, table, out, s)))
  EMBED_TYPES(CALL)
#undef CALL
}

size_t embedding_bwd_workspace(int n, int dim, int vocab) { return n == 0 ? 0 : layout(n, dim, vocab, nullptr).bytes; }

cudaError_t embedding_bwd(const EmbedArgs& a, const void* dout, void* dtable, void* ws, cudaStream_t s) {
  const size_t elem = a.table_dtype == DTYPE_F32 ? 4 : 2, bytes = elem * a.vocab * a.dim;
  if (a.n == 0) return cudaMemsetAsync(dtable, 0, bytes, s);
  const Layout l = layout(a.n, a.dim, a.vocab, ws);
  SortArgs q{a.tokens, a.n, a.vocab, a.ignore_index, {l.keys[0], l.keys[1]}, {l.places[0], l.places[1]}, 0, 0, 0, l.joins,
             l.some, a.status, (uint8_t*)dtable, 0};
  int bits = 1;
  while (((long)1 << bits) < (long)a.vocab + 1) ++bits;
  q.passes = (bits + kDigitBits - 1) / kDigitBits;
  q.bits = (bits + q.passes - 1) / q.passes;
  // the rows that are filled during the sort, about as many MB as it takes time for (64 | 96 | 128 MB with 1000 x 512 over
  // 50000 in fp32 23.6 | 25.1 | 25.0 us, 8190 x 768 over 50021 26.1 | 26.8 | 27.0, 65536 x 1024 over 131072 112 | 108 | 108, 131072 x
  // 512 over 131072 91 | 88 | 78; without any 65536 x 1024 took 14 us longer)
  const size_t row = elem * a.dim;
  const int zero_row = (int)std::min<size_t>(a.vocab, ((size_t)(64 + a.n / 1024) << 20) / row);
  q.zero_bytes = row * zero_row;
  if (zero_row == a.vocab) q.some = nullptr;
  const size_t zero_blocks = q.zero_bytes / 65536 + 1;
  static DeviceOnce once;
  static int most_ranks[kMaxDevices];
  int dev = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = sizeof(SortShared);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kMaxRanks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = once.run([&](int d) {
    cudaError_t r = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SortShared));
    if (r != cudaSuccess) return r;
    int n = 0;
    cfg.gridDim = dim3(kMaxRanks);
    if (cudaOccupancyMaxActiveClusters(&n, sort_kernel, &cfg) != cudaSuccess) cudaGetLastError();
    most_ranks[d] = n > 0 ? kMaxRanks : kMaxRanks / 2;
    return cudaSuccess;
  }, &dev);
  if (e != cudaSuccess) return e;
  // a place a thread, if there are so many blocks: each costs about 1.3 us a pass (8190 tokens by 1 | 2 | 4 | 8 blocks
  // 29 | 21 | 16 | 14 us)
  q.ranks = 1;
  while (q.ranks < most_ranks[dev] && q.ranks * kSortThreads < a.n) q.ranks *= 2;
  const long fill = std::min((long)zero_blocks, 2l * a.num_sms) / q.ranks + 1;
  attr[0].val.clusterDim.x = q.ranks;
  cfg.gridDim = dim3((unsigned)(q.ranks * (1 + fill)));
  e = cudaLaunchKernelEx(&cfg, sort_kernel, q);
  if (e != cudaSuccess) return e;
  const int at = (q.passes - 1) & 1;
  const SumArgs p{l.keys[at], l.places[at], a.n, a.dim, a.vocab, a.scale, l.part, l.joins, {l.starts[0], l.starts[1]},
                  l.some, zero_row};
#define CALL(TT, TO, V)                                                                       \
  (a.dim % V == 0 && aligned(dout, V * sizeof(TO)) && aligned(dtable, V * sizeof(TT))         \
       ? bwd_v<TT, TO, V>(p, dout, dtable, a.num_sms, s)                                      \
       : (a.dim % 2 == 0 && aligned(dout, 2 * sizeof(TO)) && aligned(dtable, 2 * sizeof(TT))  \
              ? bwd_v<TT, TO, 2>(p, dout, dtable, a.num_sms, s) : bwd_v<TT, TO, 1>(p, dout, dtable, a.num_sms, s)))
  EMBED_TYPES(CALL)
#undef CALL
}

}  // namespace jepa
