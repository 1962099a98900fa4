// The gated linear recurrence h_t = f_t h_{t-1} + (1 - f_t) v_t, f = sigmoid(g),
// forward and backward, over [batch, steps, 2 width] of gates and values.
//
// With e = exp(-g), f is 1 / (1 + e), and 1 - f is e f where g is positive and the
// difference from 1 elsewhere, where it loses nothing.  States are fp32.
//
// A run of steps maps a state x to A x + B, A the product of its f; such maps
// compose, so the steps are cut: a block takes pieces of 128 steps of a slab of
// channels, its eight warps 16 steps each.  A warp reads its steps once, into
// registers, and makes their (A, B); one warp of the block composes the warps' maps
// and leaves each warp that of what is before its steps, so that the state before
// the piece is all that is waited for (every warp going over all maps: 1 x 73728 x
// 1024 in bf16 139 us instead of 121; one warp leaving the states, which it can only
// when it has the first: 3 x 4609 x 777 in fp32 34.9 us instead of 32.2).  A warp then
// goes over its steps again in registers.  Where batch and width alone make too few
// blocks, the blocks of a cluster take consecutive pieces and exchange their maps
// through distributed shared memory, so that nothing is read twice and nobody
// waits on memory for a neighbour.
//
// Backward, m_t = f_t l_t = f_t (dh_t + m_{t+1}) is the same kind of map run the
// other way, with the same A; h is computed again inside the piece from its kept
// state by a second warp, at the same barrier (both by one: 16 x 2048 x 1024 60 us
// instead of 58).
//
// Each warp copies its steps of the next piece into shared memory that no other
// warp touches (cp.async), while it works on this one.  A thread has a word of each
// step: two 16-bit channels, whose arithmetic is packed in pairs, or one of fp32;
// rows of 16-bit channels that are not aligned to words are read in place, one
// channel a thread (two from shared memory take more to read than they save: 3 x
// 4609 x 777 in bf16 40 us forward and 56 backward, with SHIFTED rows 44 and 74, when
// this was decided; now 27 and 48, for a floor of 9.5 and 16).
//
// 16-bit types move 6 bytes of memory a channel and step forward and 10 backward.
// 16 x 2048 x 1024 in bf16 takes 35 us forward and 59 backward, 0.84 of the copy
// bandwidth both: issue and the waits for the one warp.  f and u of 16 steps are 64 of
// a thread's 128 registers, which leaves 16 warps an SM; backward f, k and h - v are
// 96 of them, and the 16-bit forms spill, 68 bytes of stores and 52 of loads a thread
// where rows are copied 16 bytes at a time, 264 and 224 where 4 (even widths that are
// no multiple of 8: 3 x 4609 x 778 73 us, 776 53).  One sequence of 73728 x 1024 (118
// us, 0.57) is bound by its chain of rounds, 2.6 us each: read, map, exchange, write.
#include <cmath>

#include "decoder.h"

namespace jepa {

namespace {

constexpr int kFwdSteps = 16, kBwdSteps = 16;   // of a warp
template <int S> constexpr int kWarps = kScanPiece / S;
template <int S> constexpr int kThreads = 32 * kWarps<S>;
constexpr int kMaxCluster = 16;
constexpr int kFewThreads = 128, kFewSteps = 16;

// ----------------------------------------------------------------------------- one or two channels
__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcpf(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// CH values, of which two are computed on at once.
template <int CH> struct Val;
template <> struct Val<1> {
  float x;
  __device__ __forceinline__ Val() {}
  __device__ __forceinline__ explicit Val(float a) : x(a) {}
  __device__ __forceinline__ float get(int) const { return x; }
  __device__ __forceinline__ void set(int, float a) { x = a; }
};
template <> struct alignas(8) Val<2> {
  uint64_t x;
  __device__ __forceinline__ Val() {}
  __device__ __forceinline__ explicit Val(float a) { pack(a, a); }
  __device__ __forceinline__ void pack(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b)); }
  __device__ __forceinline__ float get(int i) const {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
    return i == 0 ? a : b;
  }
  __device__ __forceinline__ void set(int i, float v) { i == 0 ? pack(v, get(1)) : pack(get(0), v); }
};
__device__ __forceinline__ Val<1> mul(Val<1> a, Val<1> b) { return Val<1>(a.x * b.x); }
__device__ __forceinline__ Val<1> add(Val<1> a, Val<1> b) { return Val<1>(a.x + b.x); }
__device__ __forceinline__ Val<1> fma(Val<1> a, Val<1> b, Val<1> c) { return Val<1>(fmaf(a.x, b.x, c.x)); }
__device__ __forceinline__ Val<2> mul(Val<2> a, Val<2> b) {
  Val<2> r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.x) : "l"(a.x), "l"(b.x));
  return r;
}
__device__ __forceinline__ Val<2> add(Val<2> a, Val<2> b) {
  Val<2> r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.x) : "l"(a.x), "l"(b.x));
  return r;
}
__device__ __forceinline__ Val<2> fma(Val<2> a, Val<2> b, Val<2> c) {
  Val<2> r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.x) : "l"(a.x), "l"(b.x), "l"(c.x));
  return r;
}
template <int CH> __device__ __forceinline__ Val<CH> sub(Val<CH> a, Val<CH> b) { return fma(b, Val<CH>(-1.f), a); }

// f and 1 - f
template <int CH>
__device__ __forceinline__ void sigmoid(Val<CH> g, Val<CH>& f, Val<CH>& k) {
  const Val<CH> y = mul(g, Val<CH>(-1.4426950408889634f));
  Val<CH> e;
#pragma unroll
  for (int i = 0; i < CH; ++i) e.set(i, ex2f(y.get(i)));
  const Val<CH> d = add(e, Val<CH>(1.f));
#pragma unroll
  for (int i = 0; i < CH; ++i) f.set(i, rcpf(d.get(i)));
  const Val<CH> ef = mul(e, f), rest = sub(Val<CH>(1.f), f);
#pragma unroll
  for (int i = 0; i < CH; ++i) k.set(i, g.get(i) > 0.f ? ef.get(i) : rest.get(i));
}

// CH neighbouring channels of a step in memory.
template <typename T, int CH> struct alignas(sizeof(T) * CH) Word {
  T v[CH];
  __device__ __forceinline__ Val<CH> get() const {
    Val<CH> x;
#pragma unroll
    for (int c = 0; c < CH; ++c) x.set(c, DT<T>::to(v[c]));
    return x;
  }
  __device__ __forceinline__ void put(Val<CH> x) {
    if constexpr (CH == 2) {
      const uint32_t w = pack2<T>(x.get(0), x.get(1));
      memcpy(v, &w, 4);
    } else {
      v[0] = DT<T>::from(x.get(0));
    }
  }
};

// x -> a x + b, and backward m -> a m + d.
template <int CH, int N> struct Map { Val<CH> v[N]; };

// The steps of a sequence; one outside its range is reported and clamped.
__device__ __forceinline__ int length_of(const ScanArgs& a, int b, bool report) {
  if (a.lengths == nullptr) return a.steps;
  const int n = a.lengths[b];
  if (n >= 0 && n <= a.steps) return n;
  if (report) atomicOr(a.status, DEV_BAD_INDEX);
  return n < 0 ? 0 : a.steps;
}

// ----------------------------------------------------------------------------- staging
// In place; copies of 4 bytes; of 16; of 16 where rows of fp32 start anywhere: from
// the 16 bytes in which the row's first channel lies to those of its last.
enum Stage : int { PLAIN = 0, WORDS = 1, CHUNKS = 2, SHIFTED = 3 };

// Reads `bytes` of SIZE, and writes zeros for the others.
template <int SIZE>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t bytes) {
  if constexpr (SIZE == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kLine = 128;   // a warp's words of a step
template <int STAGE> constexpr int kRowBytes = STAGE == SHIFTED ? kLine + 16 : kLine;
template <int STAGE, int S> constexpr int kTileBytes = S * kRowBytes<STAGE>;   // and of its steps of a piece
constexpr int kTiles = 4;   // of a warp: fwd gates and values of two pieces; bwd those of one, and dh of two
template <int STAGE> constexpr size_t kStageBytes = STAGE == PLAIN ? 0 : (size_t)kTiles * kScanPiece * kRowBytes<STAGE>;
// The warp's rows t0 .. t0 + S of a matrix with `stride` values a row, from
// column c0 on (the slab's first), into dst: of rows before n and columns before
// cols, zeros elsewhere.  ALL: every row and column is there.
template <typename T, int STAGE, int S, bool ALL>
__device__ __forceinline__ void copy_tile(uint32_t dst, const T* base, size_t stride, int t0, int n, int c0, int cols, int lane) {
  if constexpr (STAGE == SHIFTED) {
    constexpr int kPer = kRowBytes<STAGE> / 16, kAll = S * kPer;
    const uintptr_t any = reinterpret_cast<uintptr_t>(base) / 16 * 16;
    const int last = ALL ? c0 + 32 : min(c0 + 32, cols);   // nothing past the last channel is read
#pragma unroll
    for (int i = 0; i < kAll; i += 32) {
      const int q = i + lane, r = q / kPer;
      const uintptr_t row = reinterpret_cast<uintptr_t>(base + (size_t)(t0 + r) * stride);
      const uintptr_t src = (row + c0 * sizeof(T)) / 16 * 16 + q % kPer * 16, end = row + last * sizeof(T);
      const bool in = (ALL || t0 + r < n) && src < end;
      if (q < kAll)
        copy_async<16>(dst + q * 16, reinterpret_cast<const void*>(in ? src : any), in ? (uint32_t)min(end - src, (uintptr_t)16) : 0);
    }
  } else {
    constexpr int kPer = STAGE == CHUNKS ? 16 : 4, kLanes = kLine / kPer, kRows = 32 / kLanes;   // lanes a row, rows at a time
    const int c = c0 + lane % kLanes * (kPer / (int)sizeof(T)), r0 = lane / kLanes;
    const T* src = base + (size_t)(t0 + r0) * stride + c;
    dst += r0 * kLine + lane % kLanes * kPer;
#pragma unroll
    for (int r = 0; r < S; r += kRows) {
      const bool in = ALL || (t0 + r0 + r < n && c < cols);
      copy_async<kPer>(dst + r * kLine, in ? src : base, in ? kPer : 0);
      src += kRows * stride;
    }
  }
}
// Where a row's first channel lies in its 16 bytes (SHIFTED), for the rows of a
// tile, which starts at a multiple of 8 rows; row: the matrix's first one's.
struct Shift {
  uint32_t first, stride;
  template <typename T> __device__ __forceinline__ Shift(const T* row, int values)
      : first((uint32_t)(reinterpret_cast<uintptr_t>(row) % 16)), stride(values * (uint32_t)sizeof(T)) {}
};
// The lane's word of the i-th row of a tile.
template <typename W, int STAGE>
__device__ __forceinline__ W staged(const uint8_t* tile, int i, const Shift& s, int lane) {
  tile += i * kRowBytes<STAGE>;
  if constexpr (STAGE == SHIFTED) tile += (s.first + i * s.stride) % 16;
  return reinterpret_cast<const W*>(tile)[lane];
}

// ----------------------------------------------------------------------------- blocks
// A thread's place: its sequence, its channels (c; the slab's first is c0).
struct Place {
  int b, c0, c, n, end, rank, ranks, pieces;   // n: the sequence's steps, for every lane; end: those of gv, 0 past the last channel
  bool on, full;                               // its channels exist, all the slab's do
};
template <int CH>
__device__ __forceinline__ Place place_of(const ScanArgs& a, int ranks) {
  Place p;
  p.ranks = ranks;
  p.rank = blockIdx.x % ranks;
  p.b = blockIdx.y;
  p.c0 = blockIdx.x / ranks * 32 * CH;
  p.c = p.c0 + (threadIdx.x & 31) * CH;
  p.on = p.c < a.width;
  p.full = p.c0 + 32 * CH <= a.width;
  p.n = length_of(a, p.b, blockIdx.x == 0 && threadIdx.x == 0);
  p.end = p.on ? a.steps : 0;
  p.pieces = (a.steps + kScanPiece - 1) / kScanPiece;
  return p;
}
template <int CH>
__device__ __forceinline__ Val<CH> load_state(const float* s, bool on) {   // null: zeros
  Val<CH> x(0.f);
  if (s != nullptr && on) {
#pragma unroll
    for (int c = 0; c < CH; ++c) x.set(c, s[c]);
  }
  return x;
}
template <int CH>
__device__ __forceinline__ void store_state(float* s, Val<CH> x) {
#pragma unroll
  for (int c = 0; c < CH; ++c) s[c] = x.get(c);
}

// The maps of the blocks of a cluster, [rank][lane], exchanged: each block
// writes its own into every block's shared memory, where the bytes that arrive
// complete a phase of a barrier, so that nobody waits for anything but the maps (a
// cluster barrier's release waits for the outputs on their way to memory as well:
// 16384 x 256 in bf16 on clusters of 8 52 us instead of 33).  Two buffers and barriers are used in turn:
// who sends the next but one has had the next from every block, and they sent it
// after they had read this one.
template <int CH>
__device__ __forceinline__ void send_map(uint32_t at, uint32_t bar, const Map<CH, 2>& m) {
  if constexpr (CH == 2)
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                 "f"(m.v[0].get(0)), "f"(m.v[0].get(1)), "f"(m.v[1].get(0)), "f"(m.v[1].get(1)), "r"(bar)
                 : "memory");
  else
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                 "f"(m.v[0].get(0)), "f"(m.v[1].get(0)), "r"(bar)
                 : "memory");
}
// late: whether an earlier wait of the block has run out, after which none is
// waited for.
__device__ __forceinline__ bool wait_maps(uint64_t* bar, uint32_t parity, const volatile uint32_t* late,
                                          uint64_t limit_ns = kWaitLimitNs) {
  const uint32_t a = smem_u32(bar);
  auto arrived = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (arrived()) return true;
  if (*late != 0) return false;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (arrived()) return true;
    if ((unsigned long long)(clock64() - t0) > 2ull * limit_ns) return false;
  }
}
// By one warp.  round: how often this has been called before.  A wait that runs out
// is reported and noted after the barriers, and the results are wrong.  Returns
// where the round's maps are.
template <int CH>
__device__ __forceinline__ const Map<CH, 2> (*exchange(Map<CH, 2> (*ring)[32], uint64_t* bars, const Map<CH, 2>& mine, const Place& p,
                                                       int lane, int round, int* status))[32] {
  uint64_t* bar = bars + (round & 1);
  Map<CH, 2>(*to)[32] = ring + (round & 1) * p.ranks;
  if (lane == 0) mbar_arrive_expect_tx(bar, p.ranks * 32 * (uint32_t)sizeof(Map<CH, 2>));
  const uint32_t at = smem_u32(&to[p.rank][lane]), at_bar = smem_u32(bar);
#pragma unroll 4
  for (int r = 0; r < p.ranks; ++r) send_map<CH>(mapa_shared(at, r), mapa_shared(at_bar, r), mine);
  volatile uint32_t* late = reinterpret_cast<volatile uint32_t*>(bars + 2);
  if (!wait_maps(bar, round >> 1 & 1, late)) {
    *late = 1;
    atomicOr(status, DEV_TIMEOUT);
  }
  return to;
}
// Before the first exchange: every block's shared memory is there, and its
// barriers are.
__device__ __forceinline__ void open_cluster(uint64_t* bars) {
  if (threadIdx.x == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    *reinterpret_cast<volatile uint32_t*>(bars + 2) = 0;
    fence_mbar_init();
  }
  __syncwarp();
  cluster_sync();
}
// After the last one: no block's shared memory goes while another may write to it.
// A block whose wait has run out has not waited for all of the maps, which every
// block has sent by then: it stays until they have long arrived.
__device__ __forceinline__ void close_cluster(const uint64_t* bars) {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  if (*reinterpret_cast<const volatile uint32_t*>(bars + 2) != 0) __nanosleep(1000000);
}

// ----------------------------------------------------------------------------- forward
// Shared memory after the words: the warps' maps, the cluster's maps of two rounds, the state before the piece, two
// barriers, and whether a wait has run out.
template <int CH> constexpr size_t fwd_bytes(int ranks) {
  return (size_t)32 * CH * 4 * (2 * kWarps<kFwdSteps> + 2 * 2 * ranks + 1) + 32;
}
template <typename T, int CH, int STAGE>
__global__ void __launch_bounds__(kThreads<kFwdSteps>, 2) scan_fwd_kernel(const __grid_constant__ ScanArgs a, int ranks,
                                                                          const float* h0, T* __restrict__ h, float* last,
                                                                          float* __restrict__ states) {
  using W = Word<T, CH>;
  using V = Val<CH>;
  constexpr int S = kFwdSteps, kTile = kTileBytes<STAGE, S>;
  extern __shared__ __align__(16) uint8_t shared[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* stage = shared + warp * kTiles * kTile;   // [2][gate, value]
  auto maps = reinterpret_cast<Map<CH, 2>(*)[32]>(shared + kStageBytes<STAGE>);   // [warp][lane]
  auto ring = maps + kWarps<S>;                                                   // [2][rank][lane]
  V* begin = reinterpret_cast<V*>(ring + 2 * ranks);                              // [lane]
  uint64_t* bars = reinterpret_cast<uint64_t*>(begin + 32);
  const Place p = place_of<CH>(a, ranks);
  const size_t C = a.width;
  const T* gv = static_cast<const T*>(a.gv) + (size_t)p.b * a.steps * 2 * C;
  const Shift gs(gv + p.c0, 2 * a.width), vs(gv + C + p.c0, 2 * a.width);
  V carry(0.f);   // the first warp's
  if (warp == 0) carry = load_state<CH>(h0 != nullptr ? h0 + p.b * C + p.c : nullptr, p.on);

  auto fetch = [&](int piece, int buf) {
    const int t0 = piece * kScanPiece + warp * S;
    const uint32_t dst = smem_u32(stage) + buf * 2 * kTile;
    if (p.full && t0 + S <= p.n) {
      copy_tile<T, STAGE, S, true>(dst, gv, 2 * C, t0, 0, p.c0, 0, lane);
      copy_tile<T, STAGE, S, true>(dst + kTile, gv + C, 2 * C, t0, 0, p.c0, 0, lane);
    } else {
      copy_tile<T, STAGE, S, false>(dst, gv, 2 * C, t0, p.n, p.c0, a.width, lane);
      copy_tile<T, STAGE, S, false>(dst + kTile, gv + C, 2 * C, t0, p.n, p.c0, a.width, lane);
    }
    copy_commit();
  };
  if (p.ranks > 1) open_cluster(bars);
  if constexpr (STAGE != PLAIN)
    if (p.pieces > 0) fetch(p.rank, 0);
  for (int first = 0, round = 0; first < p.pieces; first += p.ranks, ++round) {
    const int piece = first + p.rank;
    const int t0 = piece * kScanPiece + warp * S;
    const bool all_in = p.full && t0 + S <= p.n;   // of the warp
    if constexpr (STAGE != PLAIN) {
      if (first + p.ranks < p.pieces) {
        fetch(piece + p.ranks, round & 1 ^ 1);
        copy_wait<1>();
      } else {
        copy_wait<0>();
      }
      __syncwarp();
    }
    V f[S], u[S];
    Map<CH, 2> m;
    m.v[0] = V(1.f);
    m.v[1] = V(0.f);
    auto read = [&](auto w) {
      constexpr bool whole = decltype(w)::value;
      const uint8_t* tile = stage + (round & 1) * 2 * kTile;
      const T* src = gv + (size_t)t0 * 2 * C + p.c;
      W gw[STAGE != PLAIN ? 1 : S], vw[STAGE != PLAIN ? 1 : S];
      if constexpr (STAGE == PLAIN) {
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (whole || (p.on && t0 + i < p.n)) {
            gw[i] = *reinterpret_cast<const W*>(src + (size_t)i * 2 * C);
            vw[i] = *reinterpret_cast<const W*>(src + (size_t)i * 2 * C + C);
          } else {
            gw[i] = vw[i] = W{};
          }
      }
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const W g = STAGE != PLAIN ? staged<W, STAGE>(tile, i, gs, lane) : gw[STAGE != PLAIN ? 0 : i];
        const W v = STAGE != PLAIN ? staged<W, STAGE>(tile + kTile, i, vs, lane) : vw[STAGE != PLAIN ? 0 : i];
        V k;
        sigmoid<CH>(g.get(), f[i], k);
        u[i] = mul(k, v.get());
        if (!whole && t0 + i >= p.n) {
          f[i] = V(1.f);
          u[i] = V(0.f);
        }
        m.v[0] = mul(m.v[0], f[i]);
        m.v[1] = fma(f[i], m.v[1], u[i]);
      }
    };
    if (all_in) read(std::true_type{});
    else read(std::false_type{});
    maps[warp][lane] = m;
    __syncthreads();
    if (warp == 0) {   // the map of what is before each warp's steps, and the state before the piece
      Map<CH, 2> all = maps[0][lane];
#pragma unroll
      for (int w = 1; w < kWarps<S>; ++w) {
        const Map<CH, 2> q = maps[w][lane];
        maps[w][lane] = all;
        all.v[1] = fma(q.v[0], all.v[1], q.v[1]);
        all.v[0] = mul(all.v[0], q.v[0]);
      }
      V x = carry;
      if (p.ranks > 1) {
        const auto at = exchange<CH>(ring, bars, all, p, lane, round, a.status);
#pragma unroll 4
        for (int r = 0; r < p.ranks; ++r) {
          if (r == p.rank) x = carry;
          carry = fma(at[r][lane].v[0], carry, at[r][lane].v[1]);
        }
      } else {
        carry = fma(all.v[0], x, all.v[1]);
      }
      begin[lane] = x;
      if (p.on && states != nullptr && piece < p.pieces)
        store_state<CH>(states + ((size_t)p.b * p.pieces + piece) * C + p.c, x);
    }
    __syncthreads();
    V x = begin[lane];
    if (warp > 0) x = fma(maps[warp][lane].v[0], x, maps[warp][lane].v[1]);
    T* to = h + ((size_t)p.b * a.steps + t0) * C + p.c;
    if (all_in) {
#pragma unroll
      for (int i = 0; i < S; ++i, to += C) {
        x = fma(f[i], x, u[i]);
        W o;
        o.put(x);
        *reinterpret_cast<W*>(to) = o;
      }
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i, to += C) {
        x = fma(f[i], x, u[i]);
        W o;
        o.put(t0 + i < p.n ? x : V(0.f));
        if (t0 + i < p.end) *reinterpret_cast<W*>(to) = o;
      }
    }
  }
  if (p.ranks > 1) close_cluster(bars);
  if (last != nullptr && p.on && p.rank == 0 && warp == 0) store_state<CH>(last + p.b * C + p.c, carry);
}

// ----------------------------------------------------------------------------- backward
// As fwd_bytes, with the maps of both directions, those of what is after each warp's steps, and the states before them.
template <int CH> constexpr size_t bwd_bytes(int ranks) {
  return (size_t)32 * CH * 4 * (6 * kWarps<kBwdSteps> + 2 * 2 * ranks + 1) + 32;
}
template <typename T, int CH, int STAGE>
__global__ void __launch_bounds__(kThreads<kBwdSteps>, 512 / kThreads<kBwdSteps>)
    scan_bwd_kernel(const __grid_constant__ ScanArgs a, int ranks, const T* __restrict__ dh, const float* __restrict__ states,
                    const float* __restrict__ dlast, T* __restrict__ dgv, float* __restrict__ dh0) {
  using W = Word<T, CH>;
  using V = Val<CH>;
  constexpr int S = kBwdSteps, kTile = kTileBytes<STAGE, S>;
  extern __shared__ __align__(16) uint8_t shared[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* stage = shared + warp * kTiles * kTile;   // gate, value, [2] dh
  auto ring = reinterpret_cast<Map<CH, 2>(*)[32]>(shared + kStageBytes<STAGE>);   // [2][rank][lane]
  auto maps = reinterpret_cast<Map<CH, 3>(*)[32]>(ring + 2 * ranks);              // [warp][lane]
  auto after = reinterpret_cast<Map<CH, 2>(*)[32]>(maps + kWarps<S>);             // [warp][lane]
  auto before = reinterpret_cast<V(*)[32]>(after + kWarps<S>);                    // [warp][lane]
  V* end = reinterpret_cast<V*>(before + kWarps<S>);                              // [lane]
  uint64_t* bars = reinterpret_cast<uint64_t*>(end + 32);
  const Place p = place_of<CH>(a, ranks);
  const size_t C = a.width;
  const T* gv = static_cast<const T*>(a.gv) + (size_t)p.b * a.steps * 2 * C;
  const Shift gs(gv + p.c0, 2 * a.width), vs(gv + C + p.c0, 2 * a.width);
  dh += (size_t)p.b * a.steps * C;
  const Shift ds(dh + p.c0, a.width);
  V carry(0.f);   // the first warp's: what reaches the state after the piece
  if (warp == 0) carry = load_state<CH>(dlast != nullptr ? dlast + p.b * C + p.c : nullptr, p.on);

  auto fetch_gv = [&](int piece) {
    const int t0 = piece * kScanPiece + warp * S;
    const uint32_t dst = smem_u32(stage);
    if (p.full && t0 + S <= p.n) {
      copy_tile<T, STAGE, S, true>(dst, gv, 2 * C, t0, 0, p.c0, 0, lane);
      copy_tile<T, STAGE, S, true>(dst + kTile, gv + C, 2 * C, t0, 0, p.c0, 0, lane);
    } else {
      copy_tile<T, STAGE, S, false>(dst, gv, 2 * C, t0, p.n, p.c0, a.width, lane);
      copy_tile<T, STAGE, S, false>(dst + kTile, gv + C, 2 * C, t0, p.n, p.c0, a.width, lane);
    }
  };
  auto fetch_dh = [&](int piece, int buf) {
    const int t0 = piece * kScanPiece + warp * S;
    const uint32_t dst = smem_u32(stage) + (2 + buf) * kTile;
    if (p.full && t0 + S <= p.n) copy_tile<T, STAGE, S, true>(dst, dh, C, t0, 0, p.c0, 0, lane);
    else copy_tile<T, STAGE, S, false>(dst, dh, C, t0, p.n, p.c0, a.width, lane);
  };
  const int groups = (p.pieces + p.ranks - 1) / p.ranks;
  if (p.ranks > 1) open_cluster(bars);
  if constexpr (STAGE != PLAIN)
    if (groups > 0) {
      fetch_gv((groups - 1) * p.ranks + p.rank);
      fetch_dh((groups - 1) * p.ranks + p.rank, 0);
      copy_commit();
    }
  for (int group = groups - 1, round = 0; group >= 0; --group, ++round) {
    const int piece = group * p.ranks + p.rank;
    const int t0 = piece * kScanPiece + warp * S;
    const bool all_in = p.full && t0 + S <= p.n;   // of the warp
    V state(0.f);   // the second warp's: before the piece
    if (warp == 1) state = load_state<CH>(states + ((size_t)p.b * p.pieces + piece) * C + p.c, p.on && piece < p.pieces);
    if constexpr (STAGE != PLAIN) {
      copy_wait<0>();
      __syncwarp();
    }
    V f[S], k[S], hv[S];
    W dw[STAGE != PLAIN ? 1 : S];
    auto dh_at = [&](int i) -> V {
      return STAGE != PLAIN ? staged<W, STAGE>(stage + (2 + (round & 1)) * kTile, i, ds, lane).get() : dw[STAGE != PLAIN ? 0 : i].get();
    };
    Map<CH, 3> m;
    m.v[0] = V(1.f);
    m.v[1] = m.v[2] = V(0.f);
    auto read = [&](auto w) {
      constexpr bool whole = decltype(w)::value;
      const T* src = gv + (size_t)t0 * 2 * C + p.c;
      W gw[STAGE != PLAIN ? 1 : S], vw[STAGE != PLAIN ? 1 : S];
      if constexpr (STAGE == PLAIN) {
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (whole || (p.on && t0 + i < p.n)) {
            gw[i] = *reinterpret_cast<const W*>(src + (size_t)i * 2 * C);
            vw[i] = *reinterpret_cast<const W*>(src + (size_t)i * 2 * C + C);
            dw[i] = *reinterpret_cast<const W*>(dh + (size_t)(t0 + i) * C + p.c);
          } else {
            gw[i] = vw[i] = dw[i] = W{};
          }
      }
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const W g = STAGE != PLAIN ? staged<W, STAGE>(stage, i, gs, lane) : gw[STAGE != PLAIN ? 0 : i];
        const W v = STAGE != PLAIN ? staged<W, STAGE>(stage + kTile, i, vs, lane) : vw[STAGE != PLAIN ? 0 : i];
        sigmoid<CH>(g.get(), f[i], k[i]);
        hv[i] = v.get();
        if (!whole && t0 + i >= p.n) {
          f[i] = V(1.f);
          k[i] = hv[i] = V(0.f);
        }
        m.v[0] = mul(m.v[0], f[i]);
        m.v[1] = fma(f[i], m.v[1], mul(k[i], hv[i]));
      }
#pragma unroll
      for (int i = S - 1; i >= 0; --i)
        if (whole || t0 + i < p.n) m.v[2] = mul(f[i], add(m.v[2], dh_at(i)));
    };
    if (all_in) read(std::true_type{});
    else read(std::false_type{});
    if constexpr (STAGE != PLAIN)
      if (group > 0) {   // the warp has its gates and values in registers, and has done with the dh of the piece before
        __syncwarp();
        fetch_gv(piece - p.ranks);
        fetch_dh(piece - p.ranks, round & 1 ^ 1);
        copy_commit();
      }
    maps[warp][lane] = m;
    __syncthreads();
    if (warp == 1) {   // the states before every warp's steps
#pragma unroll
      for (int w = 0; w < kWarps<S>; ++w) {
        before[w][lane] = state;
        state = fma(maps[w][lane].v[0], state, maps[w][lane].v[1]);
      }
    }
    if (warp == 0) {   // the map of what is after each warp's steps, and the gradient that reaches the piece's last state
      Map<CH, 2> all;
      all.v[0] = V(1.f);
      all.v[1] = V(0.f);
#pragma unroll
      for (int w = kWarps<S> - 1; w >= 0; --w) {
        after[w][lane] = all;
        all.v[1] = fma(maps[w][lane].v[0], all.v[1], maps[w][lane].v[2]);
        all.v[0] = mul(all.v[0], maps[w][lane].v[0]);
      }
      V l = carry;
      if (p.ranks > 1) {
        const auto at = exchange<CH>(ring, bars, all, p, lane, round, a.status);
#pragma unroll 4
        for (int r = p.ranks - 1; r >= 0; --r) {
          if (r == p.rank) l = carry;
          carry = fma(at[r][lane].v[0], carry, at[r][lane].v[1]);
        }
      } else {
        carry = fma(all.v[0], l, all.v[1]);
      }
      end[lane] = l;
    }
    __syncthreads();
    V x = before[warp][lane], l = fma(after[warp][lane].v[0], end[lane], after[warp][lane].v[1]);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const V v = hv[i];
      hv[i] = sub(x, v);
      x = fma(f[i], x, mul(k[i], v));
    }
    T* to = dgv + ((size_t)p.b * a.steps + t0 + S - 1) * 2 * C + p.c;
    if (all_in) {
#pragma unroll
      for (int i = S - 1; i >= 0; --i, to -= 2 * C) {
        const V d = add(l, dh_at(i)), dv = mul(d, k[i]);
        W o;
        o.put(mul(mul(dv, f[i]), hv[i]));
        *reinterpret_cast<W*>(to) = o;
        o.put(dv);
        *reinterpret_cast<W*>(to + C) = o;
        l = mul(f[i], d);
      }
    } else {
#pragma unroll
      for (int i = S - 1; i >= 0; --i, to -= 2 * C) {
        V dg(0.f), dv(0.f);
        if (t0 + i < p.n) {
          const V d = add(l, dh_at(i));
          dv = mul(d, k[i]);
          dg = mul(mul(dv, f[i]), hv[i]);
          l = mul(f[i], d);
        }
        W o;
        if (t0 + i < p.end) {
          o.put(dg);
          *reinterpret_cast<W*>(to) = o;
          o.put(dv);
          *reinterpret_cast<W*>(to + C) = o;
        }
      }
    }
  }
  if (p.ranks > 1) close_cluster(bars);
  if (dh0 != nullptr && p.on && p.rank == 0 && warp == 0) store_state<CH>(dh0 + p.b * C + p.c, carry);
}

// ----------------------------------------------------------------------------- few steps
// At most kFewSteps steps (serving: one), a thread for all steps of CH channels.
template <typename T, int CH>
__global__ void __launch_bounds__(kFewThreads) few_fwd_kernel(const __grid_constant__ ScanArgs a, const float* h0,
                                                              T* __restrict__ h, float* last, float* __restrict__ states) {
  using W = Word<T, CH>;
  using V = Val<CH>;
  const int c = (blockIdx.x * kFewThreads + threadIdx.x) * CH, b = blockIdx.y;
  if (c >= a.width) return;
  const int n = length_of(a, b, c == 0);
  const size_t C = a.width, at = (size_t)b * C + c;
  const T* gv = static_cast<const T*>(a.gv) + (size_t)b * a.steps * 2 * C + c;
  T* to = h + (size_t)b * a.steps * C + c;
  V x = load_state<CH>(h0 != nullptr ? h0 + at : nullptr, true);
  if (states != nullptr && a.steps > 0) store_state<CH>(states + at, x);
#pragma unroll 4
  for (int t = 0; t < a.steps; ++t) {
    W o;
    o.put(V(0.f));
    if (t < n) {
      const W g = *reinterpret_cast<const W*>(gv + t * 2 * C), v = *reinterpret_cast<const W*>(gv + t * 2 * C + C);
      V f, k;
      sigmoid<CH>(g.get(), f, k);
      x = fma(f, x, mul(k, v.get()));
      o.put(x);
    }
    *reinterpret_cast<W*>(to + t * C) = o;
  }
  if (last != nullptr) store_state<CH>(last + at, x);
}
template <typename T, int CH>
__global__ void __launch_bounds__(kFewThreads) few_bwd_kernel(const __grid_constant__ ScanArgs a, const T* __restrict__ dh,
                                                              const float* __restrict__ states,
                                                              const float* __restrict__ dlast, T* __restrict__ dgv,
                                                              float* __restrict__ dh0) {
  using W = Word<T, CH>;
  using V = Val<CH>;
  const int c = (blockIdx.x * kFewThreads + threadIdx.x) * CH, b = blockIdx.y;
  if (c >= a.width) return;
  const int n = length_of(a, b, c == 0);
  const size_t C = a.width, at = (size_t)b * C + c;
  const T* gv = static_cast<const T*>(a.gv) + (size_t)b * a.steps * 2 * C + c;
  T* to = dgv + (size_t)b * a.steps * 2 * C + c;
  dh += (size_t)b * a.steps * C + c;
  V l = load_state<CH>(dlast != nullptr ? dlast + at : nullptr, true);
  V x = load_state<CH>(states + at, a.steps > 0), f[kFewSteps], k[kFewSteps], hv[kFewSteps];
#pragma unroll
  for (int t = 0; t < kFewSteps; ++t)
    if (t < n) {
      const W g = *reinterpret_cast<const W*>(gv + t * 2 * C), v = *reinterpret_cast<const W*>(gv + t * 2 * C + C);
      sigmoid<CH>(g.get(), f[t], k[t]);
      hv[t] = sub(x, v.get());
      x = fma(f[t], x, mul(k[t], v.get()));
    }
#pragma unroll
  for (int t = kFewSteps - 1; t >= 0; --t)
    if (t < a.steps) {
      V dg(0.f), dv(0.f);
      if (t < n) {
        const V d = add(l, reinterpret_cast<const W*>(dh + t * C)->get());
        dv = mul(d, k[t]);
        dg = mul(mul(dv, f[t]), hv[t]);
        l = mul(f[t], d);
      }
      W o;
      o.put(dg);
      *reinterpret_cast<W*>(to + t * 2 * C) = o;
      o.put(dv);
      *reinterpret_cast<W*>(to + t * 2 * C + C) = o;
    }
  if (dh0 != nullptr) store_state<CH>(dh0 + at, l);
}

// ----------------------------------------------------------------------------- self test
// A wait for maps that nobody sends.
__global__ void wait_maps_kernel(int* status, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ uint32_t late;
  if (threadIdx.x == 0) {
    late = 0;
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (!wait_maps(&bar, 0, &late, limit_ns)) atomicOr(status, DEV_TIMEOUT);
}

// ----------------------------------------------------------------------------- launch
constexpr size_t kAloneBytes = 120 << 10;   // of shared memory, more than any launch takes: no two blocks on one SM
// How a kernel fills a device: the clusters of each size that run at once.
struct Resident {
  DeviceOnce once;
  int clusters[kMaxDevices][kMaxCluster + 1], alone[kMaxDevices][kMaxCluster + 1];   // alone: with one block an SM
};

// bytes: shared memory beside the words, by the blocks of a cluster.
template <int CH, int STAGE, typename K, typename... A>
cudaError_t launch(K kern, int threads, size_t (*bytes)(int), const ScanArgs& a, Resident& res, cudaStream_t s, A... args) {
  const size_t stage = kStageBytes<STAGE>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto size = [&](int ranks) {
    attr[0].val.clusterDim.x = ranks;
    cfg.dynamicSmemBytes = stage + bytes(ranks);
  };
  int dev = 0;
  cudaError_t e = res.once.run([&](int d) {
    cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAloneBytes);
    if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int k = 1; k <= kMaxCluster && r == cudaSuccess; ++k) {
      size(k);
      cfg.gridDim = dim3(k * 1024);
      bool ok = cudaOccupancyMaxActiveClusters(&res.clusters[d][k], kern, &cfg) == cudaSuccess;
      cfg.dynamicSmemBytes = kAloneBytes;
      ok = ok && cudaOccupancyMaxActiveClusters(&res.alone[d][k], kern, &cfg) == cudaSuccess;
      if (!ok) {
        res.clusters[d][k] = res.alone[d][k] = 0;
        cudaGetLastError();   // a size that this device does not take
      }
    }
    return r;
  }, &dev);
  if (e != cudaSuccess) return e;
  // The blocks of a cluster, by what their rounds of pieces should take: the clusters go in waves, each with its rounds
  // and about two to begin and end, or one where nothing is staged; a round is shorter where each block has an SM of its
  // own.  Measured forward, clusters of 1 | 2 | 4 | 8 blocks: 1 x 73728 x 1024 in bf16 673 | 406 | 207 | 166 us (12: 118, 13:
  // 121), 3 x 4609 x 777 in fp32 53 | 33 | 42 | 39, 64 x 300 x 2048 in fp16 50 | 82, 5 x 2048 x 1024 in bf16 22 | 21 | 19 | 20
  // (3: 18), 4 x 4000 x 777 in bf16 (PLAIN) 50 | 34 | 34 | 31.
  const int slabs = (a.width + 32 * CH - 1) / (32 * CH), pieces = (a.steps + kScanPiece - 1) / kScanPiece;
  const double chains = (double)slabs * a.batch;
  int ranks = 1;
  double least = -1.0;
  for (int k = 1; k <= kMaxCluster && k <= pieces; ++k) {
    if (res.clusters[dev][k] < 1) continue;
    const double waves = ceil(chains / res.clusters[dev][k]);
    const int rounds = (pieces + k - 1) / k + (STAGE == PLAIN ? 1 : 2);
    const double time = waves * rounds * (STAGE != PLAIN && chains <= res.alone[dev][k] ? 0.6 : 1.0);
    if (least < 0.0 || time < least) {
      least = time;
      ranks = k;
    }
  }
  size(ranks);
  cfg.gridDim = dim3(slabs * ranks, a.batch);
  return cudaLaunchKernelEx(&cfg, kern, a, ranks, args...);
}

dim3 few_grid(const ScanArgs& a, int ch) {
  return dim3((a.width + ch * kFewThreads - 1) / (ch * kFewThreads), a.batch);
}

template <typename T, int CH, int STAGE>
cudaError_t fwd_t(const ScanArgs& a, const float* h0, void* h, float* last, float* states, cudaStream_t s) {
  if (a.steps <= kFewSteps) {
    few_fwd_kernel<T, CH><<<few_grid(a, CH), kFewThreads, 0, s>>>(a, h0, (T*)h, last, states);
    return cudaGetLastError();
  }
  static Resident res;
  return launch<CH, STAGE>(scan_fwd_kernel<T, CH, STAGE>, kThreads<kFwdSteps>, fwd_bytes<CH>, a, res, s, h0, (T*)h, last, states);
}
template <typename T, int CH, int STAGE>
cudaError_t bwd_t(const ScanArgs& a, const void* dh, const float* states, const float* dlast, void* dgv, float* dh0,
                  cudaStream_t s) {
  if (a.steps <= kFewSteps) {
    few_bwd_kernel<T, CH><<<few_grid(a, CH), kFewThreads, 0, s>>>(a, (const T*)dh, states, dlast, (T*)dgv, dh0);
    return cudaGetLastError();
  }
  static Resident res;
  return launch<CH, STAGE>(scan_bwd_kernel<T, CH, STAGE>, kThreads<kBwdSteps>, bwd_bytes<CH>, a, res, s, (const T*)dh, states,
                           dlast, (T*)dgv, dh0);
}

// How rows can be copied: 16 bytes at a time, 4, or not at all.
int stage_of(const ScanArgs& a, const void* x, const void* y) {
  const size_t row = (size_t)a.width * (a.dtype == DTYPE_F32 ? 4 : 2);
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.gv) | reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y) | row;
  return all % 16 == 0 ? CHUNKS : (all % 4 == 0 ? WORDS : PLAIN);
}

}  // namespace

cudaError_t gated_scan_wait_selftest(int* status, uint64_t limit_ns, cudaStream_t s) {
  wait_maps_kernel<<<1, 32, 0, s>>>(status, limit_ns);
  return cudaGetLastError();
}

cudaError_t gated_scan_fwd(const ScanArgs& a, const float* h0, void* h, float* last, float* states, cudaStream_t s) {
  if (a.batch == 0) return cudaSuccess;
  const int st = stage_of(a, h, nullptr);
#define CALL(T, CH, STAGE) fwd_t<T, CH, STAGE>(a, h0, h, last, states, s)
#define TYPES                                                                                                       \
  if (a.dtype == DTYPE_F32) return st == CHUNKS ? CALL(float, 1, CHUNKS) : CALL(float, 1, SHIFTED);                  \
  if (a.dtype == DTYPE_F16)                                                                                         \
    return st == CHUNKS ? CALL(__half, 2, CHUNKS) : (st == WORDS ? CALL(__half, 2, WORDS) : CALL(__half, 1, PLAIN)); \
  return st == CHUNKS ? CALL(__nv_bfloat16, 2, CHUNKS)                                                              \
                      : (st == WORDS ? CALL(__nv_bfloat16, 2, WORDS) : CALL(__nv_bfloat16, 1, PLAIN));
  TYPES
#undef CALL
}

cudaError_t gated_scan_bwd(const ScanArgs& a, const void* dh, const float* states, const float* dlast, void* dgv,
                           float* dh0, cudaStream_t s) {
  if (a.batch == 0) return cudaSuccess;
  const int st = stage_of(a, dh, dgv);
#define CALL(T, CH, STAGE) bwd_t<T, CH, STAGE>(a, dh, states, dlast, dgv, dh0, s)
  TYPES
#undef CALL
#undef TYPES
}

}  // namespace jepa
