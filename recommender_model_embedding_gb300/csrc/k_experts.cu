// Rows sorted by expert and brought back (the data movement of a sparsely gated mixture of
// experts): n rows choose k experts each, slot q = i * k + j being row i's j-th choice.
//
//   sort      stable by (expert, q); slots without an expert last:
//             order[p] = q, pos[q] = p (or -1 - p for a dropped slot), offsets[e] = first p of e
//   dispatch  xs[p] = x[order[p] / k], zero past offsets[E]
//   combine   out[i] = sum over kept j of w[i][j] * ys[pos[i k + j]]
//   backward  dx[i] = sum over kept j of dxs[pos],  dys[pos] = w * dout[i] (zero past
//             offsets[E]),  dw[i][j] = dout[i] . ys[pos] (zero when dropped)
//
// Everything is data movement, so every kernel walks the unsorted rows: x and dout are read once,
// the sorted side is touched one whole row at a time through pos, and no output needs an atomic
// (fixed order of summation: results repeat bit for bit).  Dispatch, combine and the gradients
// are bound by HBM bandwidth.  Measured in bf16: dispatch 262144 x 4 rows of 512, 1.34 GB in
// 193 us (6.95 TB/s), combine the same 1.34 GB in 206 us (6.5), its gradient 262144 x 2, 1.34 GB in
// 208 us (6.4), dispatch's gradient 0.81 GB in 128 us (6.3).
#include "rows_common.cuh"

namespace emb {

// ---- sort: a stable counting sort, keys 0..E (E: dropped) ----
// Each CTA takes a contiguous chunk of slots and each of its warps a contiguous part of it, so
// a slot's place is base(expert) + earlier chunks + earlier warps + earlier slots of the warp.
// A first launch counts each chunk's keys; the last (started early: it waits for the first only
// where it reads the counts) sums those counts over the chunks (every CTA reads all of them
// from L2; a launch between the two does it where they are many), scans them over the experts
// and places the slots.  A single chunk needs no first launch (3000 slots: 4.5 us in one launch,
// 4.8 in two).  Up to 16 chunks exchanging their counts through the shared memory of a cluster,
// in one launch, gained little with few experts (6.1 us for 16384 slots of 64, two launches 6.3)
// and lost with many (15.4 us for 32768 slots of 1024, two launches 9.9).
// Bound by instructions and latency, not bytes (1M slots of 128 experts: 15 us, 2M of 64: 27; the
// placing kernel issues in 56% of the cycles with half the warps there are): a chunk is as short
// as one CTA an SM allows, a warp loads the ids of eight groups of 32 slots at once, and where
// that is all of its part (KEEP: chunks of up to 8192 slots) keys and ranks stay in registers
// from counting to placing and the chunk is put in order in shared memory first, so that its
// places are written in runs (1M slots: 23 -> 21 us).  Lanes with equal keys find each other by
// ballots over the key's bits: __match_any_sync, which works through the distinct keys, took
// 29 us where this took 23 (1M slots of 128 experts, before the staged writes).
constexpr int kSortWarps = 32, kSortThreads = kSortWarps * 32;
constexpr int kSortDepth = 8;       // groups of 32 ids a warp loads at once
constexpr int kSortSingle = 4096;   // slots of one CTA alone, at most
constexpr int kSortFewWarps = 8;    // of that CTA, for up to 2048 slots
constexpr int kSortScan = 32768;    // counts (chunks x keys) above which a launch sums them
constexpr int kSortMaxKeep = 1024;  // chunks, at most, of the size that stays in registers

// Keys of up to eight groups of 32 slots of a warp's part, from group g0 on; E + 1 past its end.
__device__ __forceinline__ void load_keys(const int64_t* ids, int64_t w0, int64_t g0, int64_t groups,
                                          int64_t end, int E, uint32_t (&key)[kSortDepth]) {
#pragma unroll
  for (int u = 0; u < kSortDepth; ++u) {
    const int64_t q = w0 + (g0 + u) * 32 + (threadIdx.x & 31);
    key[u] = (uint32_t)E + 1u;
    if (g0 + u < groups && q < end) {
      const uint64_t id = (uint64_t)ids[q];
      key[u] = id < (uint64_t)E ? (uint32_t)id : (uint32_t)E;
    }
  }
}

// The lanes of the warp with this lane's key, of `bits` bits (all lanes call; four bits a step:
// those above the key are zero in every lane and match).
__device__ __forceinline__ uint32_t same_key(uint32_t key, int bits) {
  uint32_t peers = 0xFFFFFFFFu;
  for (int b0 = 0; b0 < bits; b0 += 4, key >>= 4) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const bool set = key & (1u << b);
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, set);
      peers &= set ? m : ~m;
    }
  }
  return peers;
}

// A slot's rank among the warp's earlier ones of its key, counted up in `mine` (all lanes call).
__device__ __forceinline__ uint32_t take_rank(uint32_t* mine, uint32_t key, int E, int bits) {
  const int lane = threadIdx.x & 31;
  const uint32_t peers = same_key(key, bits);
  const bool in = key <= (uint32_t)E;
  const uint32_t at = in ? mine[key] : 0u;
  __syncwarp();
  if (in && lane == __ffs(peers) - 1) mine[key] = at + __popc(peers);
  __syncwarp();
  return at + __popc(peers & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kSortThreads) k_expert_count(const int64_t* ids, int64_t S, int E,
                                                               int64_t chunk, uint32_t* hist) {
  extern __shared__ uint32_t sm_count[];
  wait_for_earlier();
  let_next_start();  // not before: the placing kernel reads the ids before it waits for this one
  const int64_t c0 = (int64_t)blockIdx.x * chunk;
  const int64_t c1 = c0 + chunk < S ? c0 + chunk : S;
  const int64_t groups = (c1 - c0 + kSortThreads - 1) / kSortThreads;
  const int64_t w0 = c0 + (threadIdx.x >> 5) * groups * 32;
  uint32_t key[kSortDepth];
  load_keys(ids, w0, 0, groups, c1, E, key);
  for (int e = threadIdx.x; e <= E; e += kSortThreads) sm_count[e] = 0;
  __syncthreads();
  for (int64_t g0 = 0; g0 < groups; g0 += kSortDepth) {
    if (g0) load_keys(ids, w0, g0, groups, c1, E, key);
#pragma unroll
    for (int u = 0; u < kSortDepth; ++u) {
      if (g0 + u >= groups) break;
      if (key[u] <= (uint32_t)E) atomicAdd(sm_count + key[u], 1u);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortThreads)
    hist[(int64_t)blockIdx.x * (E + 1) + e] = sm_count[e];
}

// The counts of all chunks, summed over the chunks before each (in place), and their totals after
// the last chunk's: one warp a key.
__global__ void __launch_bounds__(256) k_expert_scan(uint32_t* hist, int chunks, int K) {
  let_next_start();
  wait_for_earlier();
  const int lane = threadIdx.x & 31, e = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (e >= K) return;
  uint32_t run = 0;
  for (int g0 = 0; g0 < chunks; g0 += 32 * 4) {
    uint32_t c[4];  // four groups of 32 chunks loaded together
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int g = g0 + u * 32 + lane;
      c[u] = g < chunks ? __ldcg(hist + (int64_t)g * K + e) : 0u;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int g = g0 + u * 32 + lane;
      uint32_t incl = c[u];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      if (g < chunks) hist[(int64_t)g * K + e] = run + incl - c[u];
      run += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
  }
  if (lane == 0) hist[(int64_t)chunks * K + e] = run;
}

// KEEP: keys and ranks stay in registers (chunks of WARPS * 256 slots); STAGE: the chunk is put in
// order in shared memory.  The other chunks' counts come from hist (SCANNED: k_expert_scan's
// sums); NULL: one chunk.
template <int WARPS, bool KEEP, bool STAGE, bool SCANNED>
__global__ void __launch_bounds__(WARPS * 32)
    k_expert_place(const int64_t* ids, int64_t S, int E, int64_t chunk, const uint32_t* hist,
                   int32_t* order, int32_t* pos, int32_t* offsets) {
  constexpr int THREADS = WARPS * 32;
  constexpr int PER = (EMB_EXPERT_MAX + THREADS) / THREADS;  // keys of a thread, at most
  // [warps][E + 1] places within the chunk; [E + 1] totals, then bases; [E + 1] earlier chunks, then
  // how far the places are from the chunk's own order; KEEP: [8192] slots and keys in that order
  extern __shared__ uint32_t sm_place[];
  let_next_start();
  if (!hist) wait_for_earlier();
  __shared__ uint32_t warp_tot[2][WARPS];
  const int K = E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bits = 32 - __clz(E + 1);
  uint32_t* total = sm_place + WARPS * K;
  uint32_t* before = total + K;
  uint32_t* mine = sm_place + warp * K;
  uint32_t* by_slot = before + K;
  uint16_t* by_key = reinterpret_cast<uint16_t*>(by_slot + kSortDepth * THREADS);
  const int64_t c0 = (int64_t)blockIdx.x * chunk;
  const int64_t c1 = c0 + chunk < S ? c0 + chunk : S;
  const int64_t groups = (c1 - c0 + THREADS - 1) / THREADS;
  const int64_t w0 = c0 + warp * groups * 32;
  uint32_t key[kSortDepth], rank[kSortDepth];
  load_keys(ids, w0, 0, groups, c1, E, key);
  for (int e = threadIdx.x; e < (WARPS + 2) * K; e += THREADS) sm_place[e] = 0;
  __syncthreads();
  for (int64_t g0 = 0; g0 < groups; g0 += kSortDepth) {
    if (g0) load_keys(ids, w0, g0, groups, c1, E, key);
#pragma unroll
    for (int u = 0; u < kSortDepth; ++u)
      if (g0 + u < groups) rank[u] = take_rank(mine, key[u], E, bits);
  }
  if (hist) {
    wait_for_earlier();
    if (SCANNED)
      for (int e = threadIdx.x; e < K; e += THREADS) {
        before[e] = __ldcg(hist + (int64_t)blockIdx.x * K + e);
        total[e] = __ldcg(hist + (int64_t)gridDim.x * K + e);
      }
    else
    for (int e = lane; e < K; e += 32) {  // warp w: chunks w, w + 32, ...
      uint32_t t = 0, b = 0;
      for (uint32_t g0 = warp; g0 < gridDim.x; g0 += WARPS * 5) {
        uint32_t c[5];  // loaded together: one trip to L2 for up to 160 chunks
#pragma unroll
        for (int u = 0; u < 5; ++u) {
          const uint32_t g = g0 + u * WARPS;
          c[u] = g < gridDim.x ? __ldcg(hist + (int64_t)g * K + e) : 0u;
        }
#pragma unroll
        for (int u = 0; u < 5; ++u) {
          t += c[u];
          b += g0 + u * WARPS < blockIdx.x ? c[u] : 0u;
        }
      }
      if (t) atomicAdd(total + e, t);
      if (b) atomicAdd(before + e, b);
    }
  }
  __syncthreads();
  // per key: earlier warps' counts, its first place (earlier keys' totals + earlier chunks), and
  // its first place in the chunk's own order (earlier keys' counts in the chunk)
  const int per = (K + THREADS - 1) / THREADS;  // keys of a thread (consecutive)
  uint32_t sum = 0, own = 0, mine_of[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = threadIdx.x * per + i;
    if (i >= per || e >= K) break;
    uint32_t run = 0;
#pragma unroll
    for (int w0 = 0; w0 < WARPS; w0 += 8) {
      uint32_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = sm_place[(w0 + w) * K + e];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        sm_place[(w0 + w) * K + e] = run;
        run += c[w];
      }
    }
    if (!hist) total[e] = run;
    sum += total[e];
    own += mine_of[i] = run;
  }
  uint32_t incl = sum, incl_own = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o), w = __shfl_up_sync(0xFFFFFFFFu, incl_own, o);
    if (lane >= o) incl += v, incl_own += w;
  }
  if (lane == 31) warp_tot[0][warp] = incl, warp_tot[1][warp] = incl_own;
  __syncthreads();
  uint32_t first = lane < warp ? warp_tot[0][lane] : 0u, place = lane < warp ? warp_tot[1][lane] : 0u;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    first += __shfl_xor_sync(0xFFFFFFFFu, first, o);
    place += __shfl_xor_sync(0xFFFFFFFFu, place, o);
  }
  first += incl - sum, place += incl_own - own;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = threadIdx.x * per + i;
    if (i >= per || e >= K) break;
    const uint32_t t = total[e];
    if (blockIdx.x == 0) offsets[e] = (int32_t)first;
    total[e] = first + before[e];
    before[e] = total[e] - place;
    first += t, place += mine_of[i];
  }
  __syncthreads();
  for (int64_t g0 = 0; g0 < groups; g0 += kSortDepth) {
    if (!KEEP) load_keys(ids, w0, g0, groups, c1, E, key);
#pragma unroll
    for (int u = 0; u < kSortDepth; ++u) {
      if (g0 + u >= groups) break;
      uint32_t p;
      if (KEEP) p = (key[u] <= (uint32_t)E ? mine[key[u]] : 0u) + rank[u];
      else p = take_rank(mine, key[u], E, bits);
      if (key[u] <= (uint32_t)E) {
        const int64_t q = w0 + (g0 + u) * 32 + lane;
        p += total[key[u]];
        pos[q] = key[u] < (uint32_t)E ? (int32_t)p : ~(int32_t)p;
        if (STAGE) {
          const uint32_t l = p - before[key[u]];
          by_slot[l] = (uint32_t)q;
          by_key[l] = (uint16_t)key[u];
        } else {
          order[p] = (int32_t)q;
        }
      }
    }
  }
  if (STAGE) {  // in the chunk's own order, so that neighbouring threads write neighbouring places
    __syncthreads();
    for (int l = threadIdx.x; l < (int)(c1 - c0); l += THREADS)
      order[l + before[by_key[l]]] = (int32_t)by_slot[l];
  }
}

struct SortPlan {
  int64_t chunk, chunks;
  bool keep, scan;
};

// One chunk an SM, or as many of the size that stays in registers as it takes.
static SortPlan sort_plan(int64_t S, int E, int sms) {
  SortPlan p{kSortSingle, 1, true, false};
  if (S <= kSortSingle) return p;
  const int64_t most = kSortDepth * kSortThreads, even = (S + sms - 1) / sms;
  p.keep = (S + most - 1) / most <= kSortMaxKeep;
  p.chunk = p.keep && even > most ? most : (even + kSortThreads - 1) / kSortThreads * kSortThreads;
  p.chunks = (S + p.chunk - 1) / p.chunk;
  p.scan = p.chunks * (E + 1) > kSortScan;
  return p;
}

int64_t expert_sort_workspace(int64_t S, int E) {
  const SortPlan p = sort_plan(S, E, device_sms());
  return p.chunks <= 1 ? 0 : (p.chunks + 1) * (E + 1) * (int64_t)sizeof(uint32_t);
}

cudaError_t launch_expert_sort(const int64_t* ids, int64_t S, int E, int32_t* order, int32_t* pos,
                               int32_t* offsets, void* ws, cudaStream_t s) {
  const SortPlan p = sort_plan(S, E, device_sms());
  const int G = (int)p.chunks;
  uint32_t* hist = G > 1 ? static_cast<uint32_t*>(ws) : nullptr;
  const uint32_t* sums = hist;
  const int staged = p.keep && hist ? kSortDepth * kSortThreads * 6 : 0;
  const auto smem = [&](int warps) { return (warps + 2) * (E + 1) * (int)sizeof(uint32_t) + staged; };
  if (!hist) {  // an empty batch still writes offsets
    const bool few = S <= kSortFewWarps * 32 * kSortDepth;
    constexpr auto small = k_expert_place<kSortFewWarps, true, false, false>;
    constexpr auto big = k_expert_place<kSortWarps, true, false, false>;
    const cudaError_t e = few ? prepare_kernel<small>() : prepare_kernel<big>();
    if (e != cudaSuccess) return e;
    const int warps = few ? kSortFewWarps : kSortWarps;
    return launch_early(few ? small : big, 1, warps * 32, smem(warps), s, ids, S, E, p.chunk, sums, order,
                        pos, offsets);
  }
  cudaError_t e = launch_early(k_expert_count, G, kSortThreads, (E + 1) * (int)sizeof(uint32_t), s, ids, S, E,
                               p.chunk, hist);
  if (e == cudaSuccess && p.scan)
    e = launch_early(k_expert_scan, (E + 1 + 7) / 8, 256, 0, s, hist, G, E + 1);
  if (e != cudaSuccess) return e;
  const auto place = [&](auto keep, auto scanned) {
    constexpr bool K = decltype(keep)::value;
    constexpr auto kern = k_expert_place<kSortWarps, K, K, decltype(scanned)::value>;
    const cudaError_t f = prepare_kernel<kern>();
    return f != cudaSuccess ? f
                            : launch_early(kern, G, kSortThreads, smem(kSortWarps), s, ids, S, E, p.chunk, sums,
                                           order, pos, offsets);
  };
  if (p.keep) return p.scan ? place(std::true_type{}, std::true_type{}) : place(std::true_type{}, std::false_type{});
  return p.scan ? place(std::false_type{}, std::true_type{}) : place(std::false_type{}, std::false_type{});
}

// ---- rows to and from their sorted places ----
// A task is a row, or a part of one: `lanes` neighbouring threads (a power of two, up to 32), each
// with UN units of the row `lanes` apart, all loaded before the first is used.  A unit is 16
// bytes where every row start and the row length are multiples of 16, else 4 or 2: the row's
// addresses are worked out once a task, so that narrow units cost little more (16411 x 3 rows of
// 479 fp32: dispatch 34 -> 19 us, combine 54 -> 24 us, against a division an element).  Narrow
// rows take few threads (but a 32-byte sector's worth) with several units each, so that a warp
// has several rows in flight (177877 x 1 rows of 40 fp32, both gradients: 68 -> 31 us); with too
// few rows to fill the device that way, more threads.  Units of 16 bytes go at most two a
// thread: with eight, dispatch of 262144 x 4 rows of 512 bf16 took 8 us more.
constexpr int kMoveThreads = 256;

struct MoveShape {
  uint32_t tasks, n;
  int U, lanes, shift;  // units of a row; threads of a task, and their log2
  FastDiv segs;         // tasks of a row
};

// UN (a power of two, at most `most`) and the shape for it.
static int move_shape(MoveShape& m, int64_t n, int units, int unit_bytes, int most) {
  const int64_t enough = (int64_t)device_sms() * 1024;
  m.n = (uint32_t)n, m.U = units, m.lanes = unit_bytes < 32 ? 32 / unit_bytes : 1, m.shift = 0;
  while (m.lanes > 1 && m.lanes / 2 >= units) m.lanes /= 2;
  while (m.lanes < 32 && m.lanes < units && (m.lanes * most < units || n * m.lanes < enough)) m.lanes *= 2;
  while ((1 << m.shift) < m.lanes) ++m.shift;
  int un = 1;
  while (un < most && un * m.lanes < units) un *= 2;
  m.segs = FastDiv((uint32_t)((units + un * m.lanes - 1) / (un * m.lanes)));
  m.tasks = m.n * m.segs.d;
  return un;
}

static unsigned move_grid(const MoveShape& m) {
  return (unsigned)(((int64_t)m.tasks * m.lanes + kMoveThreads - 1) / kMoveThreads);
}

// This thread's task: its row and first unit (false: none).
__device__ __forceinline__ bool move_task(const MoveShape& m, int un, uint32_t& row, int& unit) {
  const uint32_t task =
      (uint32_t)(((uint64_t)blockIdx.x * kMoveThreads + threadIdx.x) >> m.shift);
  if (task >= m.tasks) return false;
  row = m.segs.div(task);
  unit = (int)(task - row * m.segs.d) * un * m.lanes + (threadIdx.x & (m.lanes - 1));
  return true;
}

template <int UB>
struct Unit;
template <>
struct Unit<16> {
  using T = uint4;
  static __device__ __forceinline__ T zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Unit<4> {
  using T = uint32_t;
  static __device__ __forceinline__ T zero() { return 0u; }
};
template <>
struct Unit<2> {
  using T = uint16_t;
  static __device__ __forceinline__ T zero() { return 0; }
};

template <int UB, int UN>
__global__ void __launch_bounds__(kMoveThreads)
    k_expert_dispatch(const char* x, uint32_t x_st, const int32_t* pos, int k, MoveShape m, char* xs,
                      uint32_t xs_st) {
  using V = typename Unit<UB>::T;
  let_next_start();
  wait_for_earlier();
  uint32_t row;
  int unit;
  if (!move_task(m, UN, row, unit)) return;
  const uint32_t S = m.n * (uint32_t)k;
  const char* src = x + ((uint64_t)row * x_st + (uint32_t)unit * UB);
  V v[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (unit + u * m.lanes < m.U) v[u] = *reinterpret_cast<const V*>(src + u * m.lanes * UB);
  const int32_t* ps = pos + (uint64_t)row * k;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int32_t p = ps[j];
    const uint32_t to = (uint32_t)(p >= 0 ? p : ~p);
    if (to >= S) continue;
    char* dst = xs + ((uint64_t)to * xs_st + (uint32_t)unit * UB);
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (unit + u * m.lanes < m.U)
        *reinterpret_cast<V*>(dst + u * m.lanes * UB) = p >= 0 ? v[u] : Unit<UB>::zero();
  }
}

template <int UB>
static cudaError_t dispatch_units(const void* x, uint32_t x_st, const int32_t* pos, int64_t n, int k,
                           int row, void* xs, uint32_t xs_st, cudaStream_t s) {
  MoveShape m;
  const int un = move_shape(m, n, row / UB, UB, UB == 16 ? 2 : 8);
  const unsigned grid = move_grid(m);
  const char* in = static_cast<const char*>(x);
  char* out = static_cast<char*>(xs);
  const auto run = [&](auto kern) {
    return launch_early(kern, grid, kMoveThreads, 0, s, in, x_st, pos, k, m, out, xs_st);
  };
  if (un == 1) return run(k_expert_dispatch<UB, 1>);
  if constexpr (UB < 16)
    if (un >= 4) return un == 4 ? run(k_expert_dispatch<UB, 4>) : run(k_expert_dispatch<UB, 8>);
  return run(k_expert_dispatch<UB, 2>);
}

cudaError_t launch_expert_dispatch(const void* x, int64_t x_ld, const int32_t* pos, int64_t n, int k,
                                   int dim, int elem, void* xs, int64_t xs_ld, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const uint32_t x_st = (uint32_t)(x_ld * elem), xs_st = (uint32_t)(xs_ld * elem);
  const int row = dim * elem;
  const uint64_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(xs) | x_st | xs_st |
                       (uint64_t)row;
  if ((all & 15) == 0) return dispatch_units<16>(x, x_st, pos, n, k, row, xs, xs_st, s);
  if ((all & 3) == 0) return dispatch_units<4>(x, x_st, pos, n, k, row, xs, xs_st, s);
  return dispatch_units<2>(x, x_st, pos, n, k, row, xs, xs_st, s);
}

// Combine: KU sorted rows are loaded together (min(k, 4)); products and sums are fp32 whatever
// the rows' type, in the order of j, rounded once into out.
template <typename T, int EPU, int UN, int KU, bool WEIGHTED>
__global__ void __launch_bounds__(kMoveThreads, EPU * UN * KU > 48 ? 3 : 4)
    k_expert_combine(const T* ys, uint32_t ys_st, const int32_t* pos, const float* w, int k,
                     MoveShape m, T* out, uint32_t out_st) {
  constexpr int UB = EPU * (int)sizeof(T);
  let_next_start();
  wait_for_earlier();
  uint32_t row;
  int unit;
  if (!move_task(m, UN, row, unit)) return;
  const uint32_t S = m.n * (uint32_t)k;
  const uint64_t q0 = (uint64_t)row * k;
  float acc[UN][EPU];
#pragma unroll
  for (int u = 0; u < UN; ++u)
#pragma unroll
    for (int e = 0; e < EPU; ++e) acc[u][e] = 0.f;
  for (int j0 = 0; j0 < k; j0 += KU) {
    Pack<T, EPU> v[KU][UN];
    uint32_t p[KU];
    float g[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j) {
      p[j] = j0 + j < k ? (uint32_t)pos[q0 + j0 + j] : ~0u;
      g[j] = WEIGHTED && j0 + j < k ? w[q0 + j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < KU; ++j)
      if (p[j] < S) {  // a dropped slot's place is negative: above S
        const char* src = reinterpret_cast<const char*>(ys) + ((uint64_t)p[j] * ys_st + (uint32_t)unit * UB);
#pragma unroll
        for (int u = 0; u < UN; ++u)
          if (unit + u * m.lanes < m.U) v[j][u].load(reinterpret_cast<const T*>(src + u * m.lanes * UB));
      }
#pragma unroll
    for (int j = 0; j < KU; ++j)
      if (p[j] < S) {
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          if (unit + u * m.lanes >= m.U) continue;
          float f[EPU];
          v[j][u].get(f);
#pragma unroll
          for (int e = 0; e < EPU; ++e) acc[u][e] = WEIGHTED ? fmaf(g[j], f[e], acc[u][e]) : acc[u][e] + f[e];
        }
      }
  }
  char* dst = reinterpret_cast<char*>(out) + ((uint64_t)row * out_st + (uint32_t)unit * UB);
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (unit + u * m.lanes < m.U) {
      Pack<T, EPU> o;
      o.set(acc[u]);
      o.store(reinterpret_cast<T*>(dst + u * m.lanes * UB));
    }
}

template <typename T, int EPU, int UN, bool WEIGHTED>
static cudaError_t combine_un(const T* ys, uint32_t ys_st, const int32_t* pos, const float* w, int k,
                              const MoveShape& m, T* out, uint32_t out_st, cudaStream_t s) {
  const auto run = [&](auto kern) {
    return launch_early(kern, move_grid(m), kMoveThreads, 0, s, ys, ys_st, pos, w, k, m, out, out_st);
  };
  return k == 1   ? run(k_expert_combine<T, EPU, UN, 1, WEIGHTED>)
         : k == 2 ? run(k_expert_combine<T, EPU, UN, 2, WEIGHTED>)
         : k == 3 ? run(k_expert_combine<T, EPU, UN, 3, WEIGHTED>)
                  : run(k_expert_combine<T, EPU, UN, 4, WEIGHTED>);
}

template <typename T, int EPU>
static cudaError_t combine_units(const void* ys, uint32_t ys_st, const int32_t* pos, const float* w,
                                 int64_t n, int k, int dim, void* out, uint32_t out_st, cudaStream_t s) {
  MoveShape m;
  const int un = move_shape(m, n, dim / EPU, EPU * (int)sizeof(T), EPU > 2 ? 2 : 8 / EPU);
  const T* y = static_cast<const T*>(ys);
  T* o = static_cast<T*>(out);
  const auto run = [&](auto unc) {
    constexpr int UN = decltype(unc)::value;
    return w ? combine_un<T, EPU, UN, true>(y, ys_st, pos, w, k, m, o, out_st, s)
             : combine_un<T, EPU, UN, false>(y, ys_st, pos, w, k, m, o, out_st, s);
  };
  if (un == 1) return run(std::integral_constant<int, 1>{});
  if constexpr (EPU <= 2)
    if (un >= 4) {
      if constexpr (EPU == 1)
        if (un == 8) return run(std::integral_constant<int, 8>{});
      return run(std::integral_constant<int, 4>{});
    }
  return run(std::integral_constant<int, 2>{});
}

// w NULL: weights of one (the gradient of dispatch)
cudaError_t launch_expert_combine(const void* ys, int64_t ys_ld, const int32_t* pos, const float* w,
                                  int64_t n, int k, int dim, int bf16, void* out, int64_t out_ld,
                                  cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int elem = bf16 ? 2 : 4;
  const uint32_t ys_st = (uint32_t)(ys_ld * elem), out_st = (uint32_t)(out_ld * elem);
  const uint64_t all = reinterpret_cast<uintptr_t>(ys) | reinterpret_cast<uintptr_t>(out) | ys_st |
                       out_st | (uint64_t)(dim * elem);
  using H = __nv_bfloat16;
  if (bf16) {
    if ((all & 15) == 0) return combine_units<H, 8>(ys, ys_st, pos, w, n, k, dim, out, out_st, s);
    if ((all & 3) == 0) return combine_units<H, 2>(ys, ys_st, pos, w, n, k, dim, out, out_st, s);
    return combine_units<H, 1>(ys, ys_st, pos, w, n, k, dim, out, out_st, s);
  }
  if ((all & 15) == 0) return combine_units<float, 4>(ys, ys_st, pos, w, n, k, dim, out, out_st, s);
  return combine_units<float, 1>(ys, ys_st, pos, w, n, k, dim, out, out_st, s);
}

// ---- gradient of combine: dys and dw in one pass over dout and the sorted rows ----
// `tpr` threads share a row (a power of two): each unit of dout is loaded once, multiplied into
// the row's k sorted places and dotted with their rows; the k dot products are summed over
// the threads at the end.  A warp takes a row (less where 32 units are more than the row);
// batches too small to fill the device that way take up to a CTA a row, whose warps add
// their parts in shared memory.  UN units are in flight a thread, for each of the k rows.
constexpr int kCombThreads = 256;

template <typename T, int EPU, int KM, int UN>
__global__ void __launch_bounds__(kCombThreads)
    k_expert_combine_bwd(const T* dout, uint32_t dout_st, const T* ys, uint32_t ys_st,
                         const int32_t* pos, const float* w, uint32_t n, int k, int U, int shift,
                         T* dys, uint32_t dys_st, float* dw) {
  constexpr int UB = EPU * (int)sizeof(T);
  let_next_start();
  wait_for_earlier();
  __shared__ float part[KM][kCombThreads / 32];
  const int tpr = 1 << shift, sub = threadIdx.x & (tpr - 1);
  const uint32_t row = blockIdx.x * (kCombThreads >> shift) + (threadIdx.x >> shift);
  const bool live = row < n;
  const uint32_t S = n * (uint32_t)k;
  const uint64_t q0 = (uint64_t)row * k;
  int32_t p[KM];
  float g[KM], dot[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    dot[j] = g[j] = 0.f;
    p[j] = live && j < k ? pos[q0 + j] : (int32_t)0x80000000;  // a place no slot has
  }
#pragma unroll
  for (int j = 0; j < KM; ++j)
    if (p[j] >= 0) g[j] = w[q0 + j];
  const char* gr = reinterpret_cast<const char*>(dout) + (uint64_t)row * dout_st;
  if (live)
    for (int c0 = sub; c0 < U; c0 += tpr * UN) {
      Pack<T, EPU> d[UN], y[KM][UN];
#pragma unroll
      for (int u = 0; u < UN; ++u)
        if (c0 + u * tpr < U) d[u].load(reinterpret_cast<const T*>(gr + (uint32_t)(c0 + u * tpr) * UB));
#pragma unroll
      for (int j = 0; j < KM; ++j)
        if ((uint32_t)p[j] < S) {
          const char* src = reinterpret_cast<const char*>(ys) + ((uint64_t)(uint32_t)p[j] * ys_st + (uint32_t)c0 * UB);
#pragma unroll
          for (int u = 0; u < UN; ++u)
            if (c0 + u * tpr < U) y[j][u].load(reinterpret_cast<const T*>(src + u * tpr * UB));
        }
#pragma unroll
      for (int j = 0; j < KM; ++j) {
        const bool kept = p[j] >= 0;
        const uint32_t to = (uint32_t)(kept ? p[j] : ~p[j]);
        if (to >= S) continue;
        char* dst = reinterpret_cast<char*>(dys) + ((uint64_t)to * dys_st + (uint32_t)c0 * UB);
#pragma unroll
        for (int u = 0; u < UN; ++u) {
          if (c0 + u * tpr >= U) continue;
          Pack<T, EPU> o;
          if (kept) {
            float f[EPU], v[EPU];
            d[u].get(f);
            y[j][u].get(v);
#pragma unroll
            for (int e = 0; e < EPU; ++e) {
              dot[j] = fmaf(f[e], v[e], dot[j]);
              f[e] *= g[j];
            }
            o.set(f);
          } else {
            o.zero();
          }
          o.store(reinterpret_cast<T*>(dst + u * tpr * UB));
        }
      }
    }
#pragma unroll
  for (int j = 0; j < KM; ++j) dot[j] = lanes_sum(dot[j], tpr < 32 ? tpr : 32);
  if (tpr > 32) {
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int j = 0; j < KM; ++j) part[j][threadIdx.x >> 5] = dot[j];
    __syncthreads();
    const int w0 = (threadIdx.x >> shift) << (shift - 5);
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      dot[j] = 0.f;
      for (int i = 0; i < tpr / 32; ++i) dot[j] += part[j][w0 + i];
    }
  }
  if (live && sub == 0)
#pragma unroll
    for (int j = 0; j < KM; ++j)
      if (j < k) dw[q0 + j] = dot[j];
}

template <typename T, int EPU>
static cudaError_t combine_bwd_units(const void* dout, uint32_t dout_st, const void* ys, uint32_t ys_st,
                              const int32_t* pos, const float* w, int64_t n, int k, int dim,
                              void* dys, uint32_t dys_st, float* dw, cudaStream_t s) {
  const int U = dim / EPU;
  // threads of a row: so many that UN units each cover it, up to a warp, and more while that leaves
  // under 32 warps an SM (up to a CTA) and the row has units for them
  const int64_t enough = (int64_t)device_sms() * 32 * 32;
  const int un = k == 1 ? 4 : k == 2 || (k <= 4 && EPU <= 2) ? 2 : 1;
  int shift = 0;
  while ((1 << shift) < U && ((shift < 5 && (un << shift) < U) || (shift < 8 && (n << shift) < enough))) ++shift;
  const unsigned grid = (unsigned)(((n << shift) + kCombThreads - 1) / kCombThreads);
  const auto run = [&](auto kern) {
    return launch_early(kern, grid, kCombThreads, 0, s, static_cast<const T*>(dout), dout_st,
                        static_cast<const T*>(ys), ys_st, pos, w, (uint32_t)n, k, U, shift,
                        static_cast<T*>(dys), dys_st, dw);
  };
  return k == 1   ? run(k_expert_combine_bwd<T, EPU, 1, 4>)
         : k == 2 ? run(k_expert_combine_bwd<T, EPU, 2, 2>)
         : k <= 4 ? run(k_expert_combine_bwd<T, EPU, 4, (EPU > 2 ? 1 : 2)>)
         : k <= 8 ? run(k_expert_combine_bwd<T, EPU, 8, 1>)
                  : run(k_expert_combine_bwd<T, EPU, 16, 1>);
}

cudaError_t launch_expert_combine_bwd(const void* dout, int64_t dout_ld, const void* ys,
                                      int64_t ys_ld, const int32_t* pos, const float* w, int64_t n,
                                      int k, int dim, int bf16, void* dys, int64_t dys_ld, float* dw,
                                      cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int elem = bf16 ? 2 : 4;
  const uint32_t g_st = (uint32_t)(dout_ld * elem), y_st = (uint32_t)(ys_ld * elem),
                 o_st = (uint32_t)(dys_ld * elem);
  const uint64_t all = reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(ys) |
                       reinterpret_cast<uintptr_t>(dys) | g_st | y_st | o_st | (uint64_t)(dim * elem);
  using H = __nv_bfloat16;
  if (bf16) {
    if ((all & 15) == 0) return combine_bwd_units<H, 8>(dout, g_st, ys, y_st, pos, w, n, k, dim, dys, o_st, dw, s);
    if ((all & 3) == 0) return combine_bwd_units<H, 2>(dout, g_st, ys, y_st, pos, w, n, k, dim, dys, o_st, dw, s);
    return combine_bwd_units<H, 1>(dout, g_st, ys, y_st, pos, w, n, k, dim, dys, o_st, dw, s);
  }
  if ((all & 15) == 0) return combine_bwd_units<float, 4>(dout, g_st, ys, y_st, pos, w, n, k, dim, dys, o_st, dw, s);
  return combine_bwd_units<float, 1>(dout, g_st, ys, y_st, pos, w, n, k, dim, dys, o_st, dw, s);
}

}  // namespace emb
