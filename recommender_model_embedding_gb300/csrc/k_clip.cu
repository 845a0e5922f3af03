// Global gradient norm over a list of tensors, and clipping: norm = sqrt(sum of g^2 over all
// of them), out = g * min(1, max_norm / norm).
//
// Bound by HBM bandwidth: one read for the norm, then one read and one write for the scaled
// tensors.  Measured, 1 GB of bf16 in 40 tensors: the norm 149 us (6.75 TB/s), the scaling 304 us
// (6.6 TB/s), 477 us a call back to back.  The list is cut into tiles of equal size, dealt to the
// CTAs in turn whatever the tensors' sizes (neighbouring CTAs read neighbouring tiles: one
// contiguous share for each CTA took 505 us); the tensors' addresses travel as kernel
// parameters, so nothing is staged or kept.  Two launches serve short lists too: a cluster of
// 16 CTAs that did both passes in one took 6.3 us for 1024 elements and 10.7 for 524,288 where
// two launches take 5.6 and 8.0.  Squares are summed in fp32 over at most 16
// elements, those sums in fp64: a thread's, the CTA's and the list's, all in a fixed order, so
// the norm repeats bit for bit.  A group of elements whose fp32 sum overflows, or is so
// small that squares may have been lost, is summed again in fp64, so the norm is right for
// gradients of any finite size.
#include "rows_common.cuh"

namespace emb {

constexpr int kClipThreads = 256;
constexpr int kClipShort = 32, kClipLong = 256;  // tensors of one launch: lists up to 32, longer ones
constexpr int kClipCtasPerSm = 8;                // CTAs of the norm's launch, at most, per SM
constexpr int kClipScaleCtasPerSm = 4;           // of the scaling launch (64 registers a thread)
constexpr int kClipTile = 16384, kClipTileMin = 2048;  // elements

template <int N>
struct ClipList {
  const void* src[N];
  void* dst[N];
  int64_t numel[N];
  int64_t first[N + 1];  // first tile of each tensor
  uint8_t bf16[N];
  uint8_t vec[N];  // 16-byte accesses
  int count;
  int tile;  // elements of a tile
};

// Sum of squares of N values: fp32 where that is exact enough, else fp64.
template <int N>
__device__ __forceinline__ double square_sum(const float (&v)[N]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(v[i], v[i], s);
  if (s < 1e37f && s > 1e-30f) return (double)s;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) any |= __float_as_uint(v[i]) << 1;
  if (any == 0) return 0.0;
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) d += (double)v[i] * (double)v[i];
  return d;
}

// The last tensor whose first tile is at or before `tile` (tensors without tiles are passed over).
template <int N>
__device__ __forceinline__ int clip_tensor(const ClipList<N>& l, int64_t tile) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int THREADS, typename T, int EPU>
__device__ __forceinline__ double tile_squares(const T* p, int64_t n) {
  constexpr int U = EPU == 8 ? 2 : 4;  // 16 elements a group (4 where they come one by one)
  double acc = 0.0;
  const int64_t packs = n / EPU;
  for (int64_t c0 = threadIdx.x; c0 < packs; c0 += THREADS * U) {
    Pack<T, EPU> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u].zero();
      if (c0 + u * THREADS < packs) v[u].load(p + (c0 + u * THREADS) * EPU);
    }
    float f[U * EPU];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float e[EPU];
      v[u].get(e);
#pragma unroll
      for (int m = 0; m < EPU; ++m) f[u * EPU + m] = e[m];
    }
    acc += square_sum(f);
  }
  if (EPU > 1)
    for (int64_t i = packs * EPU + threadIdx.x; i < n; i += THREADS) {
      Pack<T, 1> v;
      v.load(p + i);
      float f[1];
      v.get(f);
      acc += square_sum(f);
    }
  return acc;
}

// Sum over the CTA, in thread 0.  fp64 additions are scarce (two lanes a cycle and SM), so one
// warp adds the others' values up and reduces once: 12 warp additions for 256 threads, where
// a shuffle tree in each of the 8 warps would take 40, and a few more to join them.
template <int THREADS>
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double sh[THREADS];
  sh[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
#pragma unroll 8
    for (int w = 1; w < THREADS / 32; ++w) v += sh[w * 32 + threadIdx.x];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// Sum of squares of tiles t0, t0 + step, ... over this thread.
template <int THREADS, int N>
__device__ __forceinline__ double share_squares(const ClipList<N>& l, int64_t t0, int64_t step) {
  double acc = 0.0;
  const int64_t tiles = l.first[l.count];
  for (int64_t t = t0; t < tiles; t += step) {
    const int i = clip_tensor(l, t);
    const int64_t at = (t - l.first[i]) * l.tile;
    const int64_t n = l.numel[i] - at < l.tile ? l.numel[i] - at : l.tile;
    if (l.bf16[i]) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(l.src[i]) + at;
      acc += l.vec[i] ? tile_squares<THREADS, __nv_bfloat16, 8>(p, n) : tile_squares<THREADS, __nv_bfloat16, 1>(p, n);
    } else {
      const float* p = static_cast<const float*>(l.src[i]) + at;
      acc += l.vec[i] ? tile_squares<THREADS, float, 4>(p, n) : tile_squares<THREADS, float, 1>(p, n);
    }
  }
  return acc;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtasPerSm)
    k_clip_norm(const __grid_constant__ ClipList<N> l, double* part) {
  let_next_start();
  wait_for_earlier();
  const double acc = cta_sum<kClipThreads>(share_squares<kClipThreads>(l, blockIdx.x, gridDim.x));
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// The factor as c * back, back a power of two: one so small that fp32 would hold it with few bits
// or as zero is carried by c near one, and the product's exponent by back, applied last.
struct Factor {
  float c, back;
  __device__ __forceinline__ float operator()(float v) const { return v * c * back; }
};

template <int THREADS, typename T, int EPU>
__device__ __forceinline__ void tile_scale(const T* p, T* o, int64_t n, Factor c) {
  constexpr int U = 4;
  const int64_t packs = n / EPU;
  for (int64_t c0 = threadIdx.x; c0 < packs; c0 += THREADS * U) {
    Pack<T, EPU> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * THREADS < packs) v[u].load(p + (c0 + u * THREADS) * EPU);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + u * THREADS < packs) {
        float f[EPU];
        v[u].get(f);
#pragma unroll
        for (int m = 0; m < EPU; ++m) f[m] = c(f[m]);
        v[u].set(f);
        v[u].store(o + (c0 + u * THREADS) * EPU);
      }
  }
  if (EPU > 1)
    for (int64_t i = packs * EPU + threadIdx.x; i < n; i += THREADS) {
      Pack<T, 1> v;
      v.load(p + i);
      float f[1];
      v.get(f);
      f[0] = c(f[0]);
      v.set(f);
      v.store(o + i);
    }
}

// Tiles t0, t0 - step, ... scaled by c.
template <int THREADS, int N>
__device__ __forceinline__ void share_scale(const ClipList<N>& l, int64_t t0, int64_t step, Factor c) {
  for (int64_t t = t0; t >= 0; t -= step) {
    const int i = clip_tensor(l, t);
    const int64_t at = (t - l.first[i]) * l.tile;
    const int64_t n = l.numel[i] - at < l.tile ? l.numel[i] - at : l.tile;
    if (l.bf16[i]) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(l.src[i]) + at;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(l.dst[i]) + at;
      if (l.vec[i]) tile_scale<THREADS, __nv_bfloat16, 8>(p, o, n, c);
      else tile_scale<THREADS, __nv_bfloat16, 1>(p, o, n, c);
    } else {
      const float* p = static_cast<const float*>(l.src[i]) + at;
      float* o = static_cast<float*>(l.dst[i]) + at;
      if (l.vec[i]) tile_scale<THREADS, float, 4>(p, o, n, c);
      else tile_scale<THREADS, float, 1>(p, o, n, c);
    }
  }
}

// The factor of a sum of squares (negative: nothing is to be scaled).  A norm that is infinite
// or NaN scales nothing: the caller sees it and drops the step.  One thread's work (fp64).
__device__ __forceinline__ Factor clip_factor(double squares, float max_norm, float& norm) {
  const double n = sqrt(squares);
  norm = (float)n;
  if (!(n > (double)max_norm && isfinite(norm))) return {-1.f, 1.f};
  const double f = (double)max_norm / n;
  if (f >= 0x1p-64 || f == 0.0) return {(float)f, 1.f};
  int x;
  frexp(f, &x);  // f < 2^x, and 2^x is in fp32 from 2^-149 on
  if (x < -149) x = -149;
  return {(float)ldexp(f, -x), (float)ldexp(1.0, x)};
}

// Every CTA adds up all `parts` itself (a few KB from L2).  The tiles are taken from the last to
// the first: the norm's pass left the last ones in L2.
template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipScaleCtasPerSm)
    k_clip_scale(const __grid_constant__ ClipList<N> l, const double* part, int parts, float max_norm,
                 float* norm_out, int inplace) {
  __shared__ Factor factor;
  let_next_start();
  wait_for_earlier();
  double acc = 0.0;
#pragma unroll 5
  for (int i = threadIdx.x; i < parts; i += kClipThreads) acc += __ldcg(part + i);
  acc = cta_sum<kClipThreads>(acc);
  if (threadIdx.x == 0) {
    float norm;
    factor = clip_factor(acc, max_norm, norm);
    if (blockIdx.x == 0) *norm_out = norm;
  }
  __syncthreads();
  Factor c = factor;
  if (c.c < 0.f) {
    if (inplace) return;
    c.c = 1.f;
  }
  share_scale<kClipThreads>(l, l.first[l.count] - 1 - blockIdx.x, gridDim.x, c);
}

int64_t clip_grads_workspace(int64_t count) {
  const int64_t launches = count > 0 ? (count + kClipLong - 1) / kClipLong : 1;
  return launches * device_sms() * kClipCtasPerSm * (int64_t)sizeof(double);
}

template <int N>
static cudaError_t clip_lists(const emb_tensor* list, int64_t count, float max_norm, float* norm,
                              double* part, cudaStream_t s) {
  const int64_t sms = device_sms(), cap = sms * kClipCtasPerSm;
  ClipList<N> l;
  int64_t total = 0;
  int inplace = 1;
  for (int64_t i = 0; i < count; ++i) {
    total += list[i].numel;
    if (list[i].d_out != list[i].d_src) inplace = 0;
  }
  // the same number of rounds for every CTA, with tiles as large as that allows up to kClipTile
  const int64_t rounds = (total + cap * kClipTile - 1) / (cap * kClipTile);
  const int64_t even = rounds > 0 ? (total + cap * rounds - 1) / (cap * rounds) : 0;
  l.tile = even > kClipTileMin ? (int)((even + 511) / 512 * 512) : kClipTileMin;
  const auto fill = [&](int64_t i0) {
    l.count = (int)(count - i0 < N ? count - i0 : N);
    l.first[0] = 0;
    for (int i = 0; i < l.count; ++i) {
      const emb_tensor& t = list[i0 + i];
      l.src[i] = t.d_src, l.dst[i] = t.d_out, l.numel[i] = t.numel;
      l.bf16[i] = t.dtype == EMB_BF16;
      l.vec[i] = rows16(t.d_src, 0, 1) && rows16(t.d_out, 0, 1);
      l.first[i + 1] = l.first[i] + (t.numel + l.tile - 1) / l.tile;
    }
    const int64_t tiles = l.first[l.count];
    return (int)(tiles < 1 ? 1 : tiles < cap ? tiles : cap);
  };
  int parts = 0, grid = 1;
  int64_t i0 = 0;
  cudaError_t e = cudaSuccess;
  do {  // an empty list still gives its norm of zero
    grid = fill(i0);
    e = launch_early(k_clip_norm<N>, (unsigned)grid, kClipThreads, 0, s, l, part + parts);
    parts += grid;
    i0 += N;
  } while (i0 < count && e == cudaSuccess);
  const bool one = count <= N;
  for (i0 = 0; e == cudaSuccess && (i0 < count || i0 == 0); i0 += N) {
    if (!one) grid = fill(i0);
    const int64_t most = sms * kClipScaleCtasPerSm;
    e = launch_early(k_clip_scale<N>, (unsigned)(grid < most ? grid : most), kClipThreads, 0, s, l,
                     (const double*)part, parts, max_norm, norm, inplace);
  }
  return e;
}

cudaError_t launch_clip_grads(const emb_tensor* list, int64_t count, float max_norm, float* norm,
                              void* ws, cudaStream_t s) {
  double* part = static_cast<double*>(ws);
  return count <= kClipShort ? clip_lists<kClipShort>(list, count, max_norm, norm, part, s)
                             : clip_lists<kClipLong>(list, count, max_norm, norm, part, s);
}

}  // namespace emb
