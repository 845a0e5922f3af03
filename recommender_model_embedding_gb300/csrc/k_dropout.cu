// Dropout from a counter-based generator, with the residual's addition.
//
//   out = residual + x * keep / (1 - p)
//
// keep is a function of (seed, step, site, row, column) alone: Philox4x32-10 (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011) of the counter (column / 8, row, step, site)
// under the 64-bit seed gives 128 bits, 16 for each of eight columns (low half of word 0 first).  An
// element is dropped where its 16 bits are below round(p 2^16), and the rest are scaled for that
// probability, so the mean is exact.  No mask is stored: the backward asks for the same numbers.  Seed and
// step are read from device memory, so a captured graph draws new numbers when they change between replays.
//
// Bound by HBM bandwidth: a thread takes the eight columns of one counter, in 16-byte accesses where the
// rows allow them.  Sixteen bits an element instead of 32 halve the generator's arithmetic (20 wide products
// a counter), which would otherwise be above what the loads leave time for.  Measured: 262144 x 1024 bf16 added to
// an fp32 residual 2.68 GB in 0.386 ms, 6.95 TB/s (the measured copy rate is 6.78); 16 x 1024 2.9 us a call.
#include <algorithm>

#include "rows_common.cuh"

namespace emb {

namespace {

constexpr int kDropThreads = 256;

struct Words {
  uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int valid, bool vec, float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      Pack<T, 8> a;
      a.load(p);
      a.get(v);
    } else {
      Pack<T, 4> a, b;
      a.load(p);
      b.load(p + 4);
      float x[4], y[4];
      a.get(x);
      b.get(y);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = x[i], v[4 + i] = y[i];
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float one[1] = {0.f};
    if (i < valid) {
      Pack<T, 1> a;
      a.load(p + i);
      a.get(one);
    }
    v[i] = one[0];
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, int valid, bool vec, const float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 2) {
      Pack<T, 8> a;
      a.set(v);
      a.store(p);
    } else {
      const float x[4] = {v[0], v[1], v[2], v[3]}, y[4] = {v[4], v[5], v[6], v[7]};
      Pack<T, 4> a;
      a.set(x);
      a.store(p);
      a.set(y);
      a.store(p + 4);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < valid) {
      const float one[1] = {v[i]};
      Pack<T, 1> a;
      a.set(one);
      a.store(p + i);
    }
}

// T: x; O: residual and out
template <typename T, typename O, bool VEC, bool RES>
__global__ void __launch_bounds__(kDropThreads)
    k_dropout(const T* x, int64_t x_ld, const O* res, int64_t res_ld, O* out, int64_t out_ld, uint32_t n, int d, int shift,
              const int64_t* rng, uint32_t site, uint32_t cut, float scale) {
  wait_for_earlier();
  let_next_start();
  const uint32_t per = kDropThreads >> shift;
  const int units = (d + 7) / 8, sub = threadIdx.x & ((1 << shift) - 1);
  const uint64_t seed = (uint64_t)rng[0];
  const uint32_t step = (uint32_t)rng[1], k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (uint32_t r = blockIdx.x * per + (threadIdx.x >> shift); r < n; r += gridDim.x * per) {
    const T* xr = x + (int64_t)r * x_ld;
    const O* rr = RES ? res + (int64_t)r * res_ld : nullptr;
    O* to = out + (int64_t)r * out_ld;
    for (int u = sub; u < units; u += 1 << shift) {
      const int valid = d - u * 8;
      float v[8], b[8];
      load8<T>(xr + u * 8, valid, VEC, v);
      if (RES) load8<O>(rr + u * 8, valid, VEC, b);
      const Words bits = philox((uint32_t)u, r, step, site, k0, k1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t draw = i & 1 ? bits.w[i >> 1] >> 16 : bits.w[i >> 1] & 0xFFFFu;
        // (a dropped element adds nothing, whatever it holds)
        if (RES) v[i] = draw >= cut ? fmaf(v[i], scale, b[i]) : b[i];
        else v[i] = draw >= cut ? v[i] * scale : 0.f;
      }
      store8<O>(to + u * 8, valid, VEC, v);
    }
  }
}

template <typename T, typename O>
cudaError_t dropout_of(const emb_dropout_rows& a, uint32_t cut, float scale, cudaStream_t s) {
  const bool vec = a.dim % 8 == 0 && rows16(a.d_x, a.x_ld, sizeof(T)) && rows16(a.d_residual, a.residual_ld, sizeof(O)) &&
                   rows16(a.d_out, a.out_ld, sizeof(O));
  int shift = 0;
  while (shift < 8 && (1 << shift) < (a.dim + 7) / 8) ++shift;
  const int64_t per = kDropThreads >> shift;
  const unsigned grid = (unsigned)std::min<int64_t>((a.n + per - 1) / per, (int64_t)device_sms() * 64);
  const auto run = [&](auto kern) {
    return launch_early(kern, grid, kDropThreads, 0, s, static_cast<const T*>(a.d_x), a.x_ld,
                        static_cast<const O*>(a.d_residual), a.residual_ld, static_cast<O*>(a.d_out), a.out_ld, (uint32_t)a.n,
                        (int)a.dim, shift, a.d_rng, a.site, cut, scale);
  };
  if (a.d_residual) return vec ? run(k_dropout<T, O, true, true>) : run(k_dropout<T, O, false, true>);
  return vec ? run(k_dropout<T, O, true, false>) : run(k_dropout<T, O, false, false>);
}

}  // namespace

cudaError_t launch_dropout(const emb_dropout_rows& a, uint32_t cut, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  using H = __nv_bfloat16;
  const float scale = cut < 65536 ? 65536.f / (float)(65536 - cut) : 0.f;
  if (a.dtype == EMB_F32) return dropout_of<float, float>(a, cut, scale, s);
  return a.out_dtype == EMB_F32 ? dropout_of<H, float>(a, cut, scale, s) : dropout_of<H, H>(a, cut, scale, s);
}

}  // namespace emb
