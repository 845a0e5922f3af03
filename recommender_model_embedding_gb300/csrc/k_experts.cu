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
// Everything is data movement, so every kernel is row-major over the unsorted rows: x and dout
// are read once, the sorted side is touched one whole row at a time through pos, and no
// output needs an atomic (fixed order of summation: results repeat bit for bit).
#include "rows_common.cuh"

namespace emb {

// ---- sort: a stable counting sort, keys 0..E (E: dropped) ----
// Each CTA takes a contiguous chunk of slots and each of its warps a contiguous part of it, so
// a slot's place is base(expert) + earlier chunks + earlier warps + earlier slots of the warp.
// A first launch counts each chunk's keys; the second sums those counts (every CTA reads all
// of them: a few hundred KB from L2), scans them over the experts and places the slots.  A
// single chunk needs no first launch.
constexpr int kSortWarps = 16;
constexpr int kSortChunk = 4096;  // slots of a chunk, at least

__device__ __forceinline__ uint32_t expert_key(const int64_t* ids, int64_t q, int64_t end, int E) {
  if (q >= end) return (uint32_t)E + 1u;  // no slot: matches only its like
  const uint64_t id = (uint64_t)ids[q];
  return id < (uint64_t)E ? (uint32_t)id : (uint32_t)E;
}

__global__ void __launch_bounds__(kSortWarps * 32) k_expert_count(const int64_t* ids, int64_t S,
                                                                  int E, int64_t chunk,
                                                                  uint32_t* hist) {
  extern __shared__ uint32_t sm_count[];
  for (int e = threadIdx.x; e <= E; e += blockDim.x) sm_count[e] = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t c0 = (int64_t)blockIdx.x * chunk;
  const int64_t c1 = c0 + chunk < S ? c0 + chunk : S;
  for (int64_t b = c0 + (threadIdx.x & ~31); b < c1; b += blockDim.x) {
    const uint32_t key = expert_key(ids, b + lane, c1, E);
    const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key);
    if (key <= (uint32_t)E && lane == __ffs(peers) - 1) atomicAdd(sm_count + key, __popc(peers));
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x)
    hist[(int64_t)blockIdx.x * (E + 1) + e] = sm_count[e];
}

__global__ void __launch_bounds__(kSortWarps * 32)
    k_expert_place(const int64_t* ids, int64_t S, int E, int64_t chunk, const uint32_t* hist,
                   int32_t* order, int32_t* pos, int32_t* offsets) {
  extern __shared__ uint32_t sm_place[];  // [warps][E + 1] places within the chunk, [E + 1] bases
  __shared__ uint32_t warp_tot[kSortWarps];
  const int K = E + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* base = sm_place + kSortWarps * K;
  uint32_t* mine = sm_place + warp * K;
  for (int e = threadIdx.x; e < kSortWarps * K; e += blockDim.x) sm_place[e] = 0;
  __syncthreads();
  const int64_t c0 = (int64_t)blockIdx.x * chunk;
  const int64_t c1 = c0 + chunk < S ? c0 + chunk : S;
  const int64_t groups = (c1 - c0 + kSortWarps * 32 - 1) / (kSortWarps * 32);  // of 32, per warp
  const int64_t w0 = c0 + warp * groups * 32;
  for (int64_t g = 0; g < groups; ++g) {
    const uint32_t key = expert_key(ids, w0 + g * 32 + lane, c1, E);
    const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key);
    if (key <= (uint32_t)E && lane == __ffs(peers) - 1) mine[key] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  // per key: earlier warps' counts, the chunk's place among the chunks, the total
  const int per = (K + blockDim.x - 1) / blockDim.x;  // keys of a thread (consecutive)
  uint32_t sum = 0;
  for (int i = 0; i < per; ++i) {
    const int e = threadIdx.x * per + i;
    if (e >= K) break;
    uint32_t run = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = sm_place[w * K + e];
      sm_place[w * K + e] = run;
      run += c;
    }
    uint32_t before = 0, total = run;
    if (hist) {
      total = 0;
#pragma unroll 8
      for (uint32_t g = 0; g < gridDim.x; ++g) {
        const uint32_t c = hist[(int64_t)g * K + e];
        if (g < blockIdx.x) before += c;
        total += c;
      }
    }
    base[e] = sum + before;  // the keys before this thread's are added below
    if (blockIdx.x == 0) offsets[e] = (int32_t)sum;
    sum += total;
  }
  uint32_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  uint32_t pre = incl - sum;
  for (int w = 0; w < warp; ++w) pre += warp_tot[w];
  for (int i = 0; i < per; ++i) {
    const int e = threadIdx.x * per + i;
    if (e >= K) break;
    base[e] += pre;
    if (blockIdx.x == 0) offsets[e] += (int32_t)pre;
  }
  __syncthreads();
  for (int64_t g = 0; g < groups; ++g) {
    const int64_t q = w0 + g * 32 + lane;
    const uint32_t key = expert_key(ids, q, c1, E);
    const uint32_t peers = __match_any_sync(0xFFFFFFFFu, key);
    const bool in = key <= (uint32_t)E;
    const uint32_t first = in ? mine[key] : 0u;
    __syncwarp();
    if (in && lane == __ffs(peers) - 1) mine[key] = first + __popc(peers);
    __syncwarp();
    if (in) {
      const uint32_t p = base[key] + first + __popc(peers & ((1u << lane) - 1u));
      pos[q] = key < (uint32_t)E ? (int32_t)p : -1 - (int32_t)p;
      order[p] = (int32_t)q;
    }
  }
}

static int64_t sort_chunk(int64_t S, int sms) {
  const int64_t even = (S + sms - 1) / sms;
  const int64_t c = even > kSortChunk ? even : kSortChunk;
  return (c + kSortWarps * 32 - 1) / (kSortWarps * 32) * (kSortWarps * 32);
}

int64_t expert_sort_workspace(int64_t S, int E) {
  const int64_t chunk = sort_chunk(S, device_sms());
  const int64_t G = (S + chunk - 1) / chunk;
  return G <= 1 ? 0 : G * (E + 1) * (int64_t)sizeof(uint32_t);
}

cudaError_t launch_expert_sort(const int64_t* ids, int64_t S, int E, int32_t* order, int32_t* pos,
                               int32_t* offsets, void* ws, cudaStream_t s) {
  const int64_t chunk = sort_chunk(S, device_sms());
  const int G = S > 0 ? (int)((S + chunk - 1) / chunk) : 1;  // an empty batch still writes offsets
  uint32_t* hist = G > 1 ? static_cast<uint32_t*>(ws) : nullptr;
  const int smem = (kSortWarps + 1) * (E + 1) * (int)sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute(k_expert_place, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (hist)
    k_expert_count<<<G, kSortWarps * 32, (E + 1) * sizeof(uint32_t), s>>>(ids, S, E, chunk, hist);
  k_expert_place<<<G, kSortWarps * 32, smem, s>>>(ids, S, E, chunk, hist, order, pos, offsets);
  return cudaGetLastError();
}

// ---- dispatch: rows copied to their sorted places, in units of UB bytes ----
// A CTA takes a tile of rows; its threads step through the tile's (row, unit) items, four loads
// in flight each, and store every unit to the row's k places.
constexpr int kMoveThreads = 256, kMoveItems = 4;

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

struct MoveTile {
  int64_t n, tiles;
  int R;        // rows of a tile
  FastDiv U;    // units of a row
};

static MoveTile move_tile(int64_t n, int64_t units) {
  MoveTile t;
  t.n = n;
  t.U = FastDiv((uint32_t)units);
  const int64_t per = kMoveThreads * kMoveItems;
  t.R = (int)(units >= per ? 1 : per / units);
  t.tiles = (n + t.R - 1) / t.R;
  return t;
}

static int move_grid(const MoveTile& t) {
  const int64_t cap = (int64_t)device_sms() * 64;
  return (int)(t.tiles < cap ? t.tiles : cap);
}

template <int UB>
__global__ void __launch_bounds__(kMoveThreads) k_expert_dispatch(const char* x, int64_t x_step,
                                                                  const int32_t* pos, int k,
                                                                  MoveTile t, char* xs,
                                                                  int64_t xs_step) {
  using V = typename Unit<UB>::T;
  const int64_t S = t.n * k;
  for (int64_t tile = blockIdx.x; tile < t.tiles; tile += gridDim.x) {
    const int64_t row0 = tile * t.R;
    const int rows = (int)(t.n - row0 < t.R ? t.n - row0 : t.R);
    const uint32_t items = (uint32_t)rows * t.U.d;
    for (uint32_t i0 = threadIdx.x; i0 < items; i0 += kMoveThreads * kMoveItems) {
      V v[kMoveItems];
#pragma unroll
      for (int u = 0; u < kMoveItems; ++u) {
        const uint32_t i = i0 + u * kMoveThreads;
        if (i < items) {
          const uint32_t r = t.U.div(i), c = i - r * t.U.d;
          v[u] = *reinterpret_cast<const V*>(x + (row0 + r) * x_step + (int64_t)c * UB);
        }
      }
#pragma unroll
      for (int u = 0; u < kMoveItems; ++u) {
        const uint32_t i = i0 + u * kMoveThreads;
        if (i < items) {
          const uint32_t r = t.U.div(i), c = i - r * t.U.d;
          const int32_t* ps = pos + (row0 + r) * k;
          for (int j = 0; j < k; ++j) {
            const int32_t p = ps[j];
            const int64_t to = p >= 0 ? (int64_t)p : -1 - (int64_t)p;
            if (to < S)
              *reinterpret_cast<V*>(xs + to * xs_step + (int64_t)c * UB) = p >= 0 ? v[u] : Unit<UB>::zero();
          }
        }
      }
    }
  }
}

cudaError_t launch_expert_dispatch(const void* x, int64_t x_ld, const int32_t* pos, int64_t n, int k,
                                   int dim, int elem, void* xs, int64_t xs_ld, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int64_t xb = x_ld * elem, sb = xs_ld * elem, row = (int64_t)dim * elem;
  const uint64_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(xs) |
                       (uint64_t)xb | (uint64_t)sb | (uint64_t)row;
  const char* xc = static_cast<const char*>(x);
  char* xsc = static_cast<char*>(xs);
  // the widest unit that every row start and the row length are multiples of
  if ((all & 15) == 0) {
    const MoveTile t = move_tile(n, row / 16);
    k_expert_dispatch<16><<<move_grid(t), kMoveThreads, 0, s>>>(xc, xb, pos, k, t, xsc, sb);
  } else if ((all & 3) == 0) {
    const MoveTile t = move_tile(n, row / 4);
    k_expert_dispatch<4><<<move_grid(t), kMoveThreads, 0, s>>>(xc, xb, pos, k, t, xsc, sb);
  } else {
    const MoveTile t = move_tile(n, row / 2);
    k_expert_dispatch<2><<<move_grid(t), kMoveThreads, 0, s>>>(xc, xb, pos, k, t, xsc, sb);
  }
  return cudaGetLastError();
}

// ---- combine: each row gathers its kept sorted rows, fp32 sum in the order of j ----
// KU sorted rows are loaded together (min(k, 4)); the products and sums are fp32 whatever the
// rows' type, rounded once into out.
template <typename T, int EPU, int KU, bool WEIGHTED>
__global__ void __launch_bounds__(kMoveThreads) k_expert_combine(const T* ys, int64_t ys_ld,
                                                                 const int32_t* pos, const float* w,
                                                                 int k, MoveTile t, T* out,
                                                                 int64_t out_ld) {
  const int64_t S = t.n * k;
  for (int64_t tile = blockIdx.x; tile < t.tiles; tile += gridDim.x) {
    const int64_t row0 = tile * t.R;
    const int rows = (int)(t.n - row0 < t.R ? t.n - row0 : t.R);
    const uint32_t items = (uint32_t)rows * t.U.d;
    for (uint32_t i = threadIdx.x; i < items; i += kMoveThreads) {
      const uint32_t r = t.U.div(i), c = i - r * t.U.d;
      const int64_t q0 = (row0 + r) * k;
      float acc[EPU];
#pragma unroll
      for (int m = 0; m < EPU; ++m) acc[m] = 0.f;
      for (int j0 = 0; j0 < k; j0 += KU) {
        Pack<T, EPU> v[KU];
        bool in[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
          const int64_t p = j0 + j < k ? (int64_t)pos[q0 + j0 + j] : -1;
          in[j] = p >= 0 && p < S;
          if (in[j]) v[j].load(ys + p * ys_ld + (int64_t)c * EPU);
        }
#pragma unroll
        for (int j = 0; j < KU; ++j)
          if (in[j]) {
            float f[EPU];
            v[j].get(f);
            const float g = WEIGHTED ? w[q0 + j0 + j] : 1.f;
#pragma unroll
            for (int m = 0; m < EPU; ++m) acc[m] = WEIGHTED ? fmaf(g, f[m], acc[m]) : acc[m] + f[m];
          }
      }
      Pack<T, EPU> o;
      o.set(acc);
      o.store(out + (row0 + r) * out_ld + (int64_t)c * EPU);
    }
  }
}

template <typename T, int EPU>
static void combine_k(const void* ys, int64_t ys_ld, const int32_t* pos, const float* w, int64_t n,
                      int k, int dim, void* out, int64_t out_ld, cudaStream_t s) {
  const MoveTile t = move_tile(n, dim / EPU);
  const int grid = move_grid(t);
  const T* y = static_cast<const T*>(ys);
  T* o = static_cast<T*>(out);
#define EMB_COMBINE(KU)                                                                          \
  (w ? k_expert_combine<T, EPU, KU, true><<<grid, kMoveThreads, 0, s>>>(y, ys_ld, pos, w, k, t, o, out_ld) \
     : k_expert_combine<T, EPU, KU, false><<<grid, kMoveThreads, 0, s>>>(y, ys_ld, pos, w, k, t, o, out_ld))
  if (k == 1) EMB_COMBINE(1);
  else if (k == 2) EMB_COMBINE(2);
  else EMB_COMBINE(4);
#undef EMB_COMBINE
}

// w NULL: weights of one (the gradient of dispatch)
cudaError_t launch_expert_combine(const void* ys, int64_t ys_ld, const int32_t* pos, const float* w,
                                  int64_t n, int k, int dim, int bf16, void* out, int64_t out_ld,
                                  cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int elem = bf16 ? 2 : 4;
  const bool vec = rows16(ys, ys_ld, elem) && rows16(out, out_ld, elem) && dim * elem % 16 == 0;
  if (bf16) {
    if (vec) combine_k<__nv_bfloat16, 8>(ys, ys_ld, pos, w, n, k, dim, out, out_ld, s);
    else combine_k<__nv_bfloat16, 1>(ys, ys_ld, pos, w, n, k, dim, out, out_ld, s);
  } else {
    if (vec) combine_k<float, 4>(ys, ys_ld, pos, w, n, k, dim, out, out_ld, s);
    else combine_k<float, 1>(ys, ys_ld, pos, w, n, k, dim, out, out_ld, s);
  }
  return cudaGetLastError();
}

// ---- gradient of combine: dys and dw in one pass over dout and the sorted rows ----
// `tpr` threads share a row (a power of two, at least 4): each pack of dout is loaded once,
// multiplied into the row's k sorted places and dotted with their rows; the k dot products
// are summed over the threads at the end.  Rows of more than 32 threads are summed through
// shared memory.
constexpr int kCombThreads = 256;

template <typename T, int EPU, int KM>
__global__ void __launch_bounds__(kCombThreads)
    k_expert_combine_bwd(const T* dout, int64_t dout_ld, const T* ys, int64_t ys_ld,
                         const int32_t* pos, const float* w, int64_t n, int k, int U, int tpr,
                         T* dys, int64_t dys_ld, float* dw) {
  __shared__ float part[KM][kCombThreads / 32];
  const int rpb = kCombThreads / tpr, sub = threadIdx.x % tpr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t S = n * k;
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < n; r0 += (int64_t)gridDim.x * rpb) {
    const int64_t row = r0 + threadIdx.x / tpr;
    const bool live = row < n;
    int64_t to[KM];
    bool kept[KM];
    float g[KM], dot[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
      dot[j] = 0.f;
      g[j] = 0.f;
      to[j] = S;
      kept[j] = false;
      if (live && j < k) {
        const int32_t p = pos[row * k + j];
        kept[j] = p >= 0 && p < S;
        to[j] = p >= 0 ? (int64_t)p : -1 - (int64_t)p;
        if (kept[j]) g[j] = w[row * k + j];
      }
    }
    if (live)
      for (int c = sub; c < U; c += tpr) {
        Pack<T, EPU> d, y[KM];
        d.load(dout + row * dout_ld + (int64_t)c * EPU);
#pragma unroll
        for (int j = 0; j < KM; ++j)
          if (kept[j]) y[j].load(ys + to[j] * ys_ld + (int64_t)c * EPU);
        float f[EPU];
        d.get(f);
#pragma unroll
        for (int j = 0; j < KM; ++j) {
          if (to[j] >= S) continue;
          float o[EPU];
          Pack<T, EPU> out;
          if (kept[j]) {
            float v[EPU];
            y[j].get(v);
#pragma unroll
            for (int m = 0; m < EPU; ++m) {
              dot[j] = fmaf(f[m], v[m], dot[j]);
              o[m] = g[j] * f[m];
            }
            out.set(o);
          } else {
            out.zero();
          }
          out.store(dys + to[j] * dys_ld + (int64_t)c * EPU);
        }
      }
#pragma unroll
    for (int j = 0; j < KM; ++j) dot[j] = lanes_sum(dot[j], tpr < 32 ? tpr : 32);
    if (tpr > 32) {
      __syncthreads();
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < KM; ++j) part[j][warp] = dot[j];
      __syncthreads();
      const int w0 = threadIdx.x / tpr * (tpr / 32);
#pragma unroll
      for (int j = 0; j < KM; ++j) {
        dot[j] = 0.f;
        for (int i = 0; i < tpr / 32; ++i) dot[j] += part[j][w0 + i];
      }
    }
    if (live && sub == 0)
#pragma unroll
      for (int j = 0; j < KM; ++j)
        if (j < k) dw[row * k + j] = dot[j];
  }
}

template <typename T, int EPU>
static void combine_bwd_k(const void* dout, int64_t dout_ld, const void* ys, int64_t ys_ld,
                          const int32_t* pos, const float* w, int64_t n, int k, int dim, void* dys,
                          int64_t dys_ld, float* dw, cudaStream_t s) {
  const int U = dim / EPU;
  int tpr = 4;
  while (tpr < kCombThreads && tpr < U) tpr *= 2;
  const int rpb = kCombThreads / tpr;
  const int64_t blocks = (n + rpb - 1) / rpb, cap = (int64_t)device_sms() * 64;
  const int grid = (int)(blocks < cap ? blocks : cap);
#define EMB_COMBINE_BWD(KM)                                                                  \
  k_expert_combine_bwd<T, EPU, KM><<<grid, kCombThreads, 0, s>>>(                            \
      static_cast<const T*>(dout), dout_ld, static_cast<const T*>(ys), ys_ld, pos, w, n, k, U, \
      tpr, static_cast<T*>(dys), dys_ld, dw)
  if (k == 1) EMB_COMBINE_BWD(1);
  else if (k == 2) EMB_COMBINE_BWD(2);
  else if (k <= 4) EMB_COMBINE_BWD(4);
  else if (k <= 8) EMB_COMBINE_BWD(8);
  else EMB_COMBINE_BWD(16);
#undef EMB_COMBINE_BWD
}

cudaError_t launch_expert_combine_bwd(const void* dout, int64_t dout_ld, const void* ys,
                                      int64_t ys_ld, const int32_t* pos, const float* w, int64_t n,
                                      int k, int dim, int bf16, void* dys, int64_t dys_ld, float* dw,
                                      cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int elem = bf16 ? 2 : 4;
  const bool vec = rows16(dout, dout_ld, elem) && rows16(ys, ys_ld, elem) &&
                   rows16(dys, dys_ld, elem) && dim * elem % 16 == 0;
  if (bf16) {
    if (vec) combine_bwd_k<__nv_bfloat16, 8>(dout, dout_ld, ys, ys_ld, pos, w, n, k, dim, dys, dys_ld, dw, s);
    else combine_bwd_k<__nv_bfloat16, 1>(dout, dout_ld, ys, ys_ld, pos, w, n, k, dim, dys, dys_ld, dw, s);
  } else {
    if (vec) combine_bwd_k<float, 4>(dout, dout_ld, ys, ys_ld, pos, w, n, k, dim, dys, dys_ld, dw, s);
    else combine_bwd_k<float, 1>(dout, dout_ld, ys, ys_ld, pos, w, n, k, dim, dys, dys_ld, dw, s);
  }
  return cudaGetLastError();
}

}  // namespace emb
