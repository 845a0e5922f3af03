// A residual block's ends in one pass: the norm after the block, its gate and residual scale,
// and the norm before the next block.
//
//   a = y / rms(y)                      rms(v) = sqrt(mean(v^2) + eps) over the row
//   x_out = x + res_scale * sigmoid(gate) * (a * w_post)
//   h = x_out / rms(x_out) * w_pre
//
// Backward, from dx_out (the residual stream's gradient), dh, and x_out and y as they are
// stored (no statistics are kept: both row sums of squares come with the pass):
//   q = x_out / rms(x_out), m = mean(dh * w_pre * q)
//   t = dx_out + (dh * w_pre - q * m) / rms(x_out)              dx = t
//   u = t * res_scale * g * w_post, g = sigmoid(gate)
//   dy = (u - a * mean(u * a)) / rms(y)
//   dgate = t * res_scale * w_post * a * g * (1 - g)            (summed for one gate per row)
//   dw_pre = sum over rows of dh * q;   with T = sum over rows of t * g * a:
//   dw_post = res_scale * T, dres_scale = w_post * T
//
// Both are bound by HBM bandwidth.  A group of `tpr` threads takes a row, about eight elements a
// thread (V packs of EPU: 16 bytes a pack where everything is aligned, one element otherwise;
// with an fp32 stream beside bf16 blocks 4 elements, 16 and 8 bytes, so that neighbouring
// threads' accesses of either type are neighbours in memory), so a row costs each thread few shuffles per element.  CTAs are persistent; every thread
// copies its own packs of the next rows to shared memory asynchronously, kStages rows ahead,
// and reads back only what it copied itself, so the ring needs no barrier; the groups of
// a CTA run independently of each other (named barriers for the row sums, and only for rows
// of more than 32 threads).  The backward computes everything but dy in one sweep
// over the row, since only dy needs the second row sum: it keeps u in registers and y in the
// ring.  A thread has the same columns for all its rows, so the column sums stay in its
// registers until the end, when they go to the workspace and a second launch adds the CTAs'
// parts in a fixed order.
#include "rows_common.cuh"

namespace emb {

constexpr int kNormThreads = 256;  // of a CTA (8 elements a thread)
constexpr int kNormWide = 512;     // of a CTA whose rows take 16 elements a thread, at most
constexpr int kStages = 3;            // rows of the ring

struct NormArgs {
  uint32_t n;
  int dim, packs, tpr;  // packs of EPU elements of a row; threads of a row
  int rpb;              // rows side by side in a CTA
  int stages;           // of the ring: 1 .. kStages
  int gate_row;         // one gate for a row
  float eps, inv_dim;
  const char *x, *y, *gate, *dx_out, *dh;
  char *x_out, *h, *dx, *dy, *dgate;
  uint32_t x_st, y_st, gate_st, dx_out_st, dh_st, x_out_st, h_st, dx_st, dy_st, dgate_st;  // bytes
  const float *w_post, *res_scale, *w_pre;
  float *dw_post, *dres_scale, *dw_pre;
  float* part;  // [CTAs][2][dim] column sums (backward)
};

// ---- arithmetic on N elements a thread: two at a time (fp32 pairs) where N is even ----
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// d = a * b + c, with b a vector or one factor for all
template <int N>
__device__ __forceinline__ void v_fma(float (&d)[N], const float (&a)[N], const float (&b)[N],
                                      const float (&c)[N]) {
  if constexpr (N == 1) d[0] = fmaf(a[0], b[0], c[0]);
  else
#pragma unroll
    for (int m = 0; m < N; m += 2)
      fma2(d[m], d[m + 1], a[m], a[m + 1], b[m], b[m + 1], c[m], c[m + 1]);
}
template <int N>
__device__ __forceinline__ void v_fma(float (&d)[N], const float (&a)[N], float b, const float (&c)[N]) {
  if constexpr (N == 1) d[0] = fmaf(a[0], b, c[0]);
  else
#pragma unroll
    for (int m = 0; m < N; m += 2) fma2(d[m], d[m + 1], a[m], a[m + 1], b, b, c[m], c[m + 1]);
}
template <int N>
__device__ __forceinline__ void v_mul(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
  if constexpr (N == 1) d[0] = a[0] * b[0];
  else
#pragma unroll
    for (int m = 0; m < N; m += 2) mul2(d[m], d[m + 1], a[m], a[m + 1], b[m], b[m + 1]);
}
template <int N>
__device__ __forceinline__ void v_mul(float (&d)[N], const float (&a)[N], float b) {
  if constexpr (N == 1) d[0] = a[0] * b;
  else
#pragma unroll
    for (int m = 0; m < N; m += 2) mul2(d[m], d[m + 1], a[m], a[m + 1], b, b);
}
// s += sum of a * b, in two halves
template <int N>
__device__ __forceinline__ void v_dot(float (&s)[2], const float (&a)[N], const float (&b)[N]) {
  if constexpr (N == 1) s[0] = fmaf(a[0], b[0], s[0]);
  else
#pragma unroll
    for (int m = 0; m < N; m += 2) fma2(s[0], s[1], a[m], a[m + 1], b[m], b[m + 1], s[0], s[1]);
}

// g = sigmoid(z) = 1 / (1 + e) and rest = 1 - g, with e = exp(-z), both to a few units in the
// last place: rest is taken as e g where that difference would cancel (z >= 0).
__device__ __forceinline__ void sigmoid2(float z, float& g, float& rest) {
  float e;  // the product's rounding moves e by less than |z| units, where e is at most that small
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(1.f + e));
  rest = z < 0.f ? 1.f - g : e * g;
}

// The ring: for each matrix and pack a plane of one place per thread.
template <typename T, int EPU>
struct Slot {
  static constexpr int kBytes = EPU * (int)sizeof(T);
  static_assert(kBytes <= 16, "a pack is one access");

  // starts the copy of the pack at p to this thread's place `to`
  static __device__ __forceinline__ void fetch(uint32_t to, const char* p) {
    if constexpr (kBytes == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
    } else if constexpr (kBytes >= 4) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(p), "n"(kBytes) : "memory");
    } else {  // one bf16: too small for an asynchronous copy
      const uint16_t v = *reinterpret_cast<const uint16_t*>(p);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(v) : "memory");
    }
  }
  static __device__ __forceinline__ void zero(uint32_t to) {
#pragma unroll
    for (int b = 0; b < kBytes; b += 2)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + b), "h"((uint16_t)0) : "memory");
  }
  static __device__ __forceinline__ void read(uint32_t from, float* v) {
    if constexpr (kBytes >= 4) {
      uint32_t w[kBytes / 4];
      if constexpr (kBytes == 16)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from) : "memory");
      else if constexpr (kBytes == 8)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(from) : "memory");
      else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(from) : "memory");
#pragma unroll
      for (int i = 0; i < EPU; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
        else v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      }
    } else {
      uint16_t w;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(from) : "memory");
      v[0] = __uint_as_float((uint32_t)w << 16);
    }
  }
};

template <int N>
__device__ __forceinline__ void ring_wait_n() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// waits until at most `stages - 1` of this thread's copies (one group a row) are in flight
__device__ __forceinline__ void ring_wait(int stages) {
  if (stages == 3) ring_wait_n<2>();
  else if (stages == 2) ring_wait_n<1>();
  else ring_wait_n<0>();
}
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// The threads of one row: group `id` of the CTA, thread `sub` of tpr.
struct RowGroup {
  int tpr, id, sub;
  // Sums of NS (1 or 3) values over the group, the same in every thread.  `red`: the group's own
  // NS * 16 floats, 16-byte aligned, zero past its warps and not used again before another
  // sum of the group has passed its barrier.
  template <int NS>
  __device__ __forceinline__ void sum(float (&v)[NS], float* red) const {
    static_assert(NS == 1 || NS == 3, "one or three sums");
    if (tpr < 32) {
#pragma unroll
      for (int i = 0; i < NS; ++i) v[i] = lanes_sum(v[i], tpr);
      return;
    }
    const int lane = threadIdx.x & 31;
    float r = v[0];
    if constexpr (NS == 3) {
      // three sums in one: lanes 0-7, 16-23 and 8-15 (24-31) end with v[0], v[1] and v[2]
      const bool up = lane & 16, odd = lane & 8;
      r = (up ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[0] : v[1], 16);
      const float c = v[2] + __shfl_xor_sync(0xFFFFFFFFu, v[2], 16);
      r = (odd ? c : r) + __shfl_xor_sync(0xFFFFFFFFu, odd ? r : c, 8);
    } else {
      r += __shfl_xor_sync(0xFFFFFFFFu, r, 16);
      r += __shfl_xor_sync(0xFFFFFFFFu, r, 8);
    }
    r += __shfl_xor_sync(0xFFFFFFFFu, r, 4);
    r += __shfl_xor_sync(0xFFFFFFFFu, r, 2);
    r += __shfl_xor_sync(0xFFFFFFFFu, r, 1);
    if (tpr == 32) {
      v[0] = __shfl_sync(0xFFFFFFFFu, r, 0);
      if constexpr (NS == 3) {
        v[1] = __shfl_sync(0xFFFFFFFFu, r, 16);
        v[2] = __shfl_sync(0xFFFFFFFFu, r, 8);
      }
      return;
    }
    if (lane == 0) red[sub >> 5] = r;
    if constexpr (NS == 3) {
      if (lane == 16) red[16 + (sub >> 5)] = r;
      if (lane == 8) red[32 + (sub >> 5)] = r;
    }
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(tpr) : "memory");
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float4* q = reinterpret_cast<const float4*>(red + i * 16);
      float4 f = q[0];
      v[i] = (f.x + f.y) + (f.z + f.w);
      for (int w = 1; w * 128 < tpr; ++w) {
        f = q[w];
        v[i] += (f.x + f.y) + (f.z + f.w);
      }
    }
  }
};

template <int EPU>
__device__ __forceinline__ void load_cols(const float* w, int col, float* v) {
  if constexpr (EPU >= 4) {
#pragma unroll
    for (int m = 0; m < EPU; m += 4) {
      const float4 f = w ? __ldg(reinterpret_cast<const float4*>(w + col + m))
                         : make_float4(1.f, 1.f, 1.f, 1.f);
      v[m] = f.x, v[m + 1] = f.y, v[m + 2] = f.z, v[m + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int m = 0; m < EPU; ++m) v[m] = w ? __ldg(w + col + m) : 1.f;
  }
}

// Which packs of a row a thread has: first, first + step, ... (V of them).  WARP: the row takes
// whole warps, each V * 32 packs in a row, so that the step is known to the compiler (addresses
// of a thread's packs differ by constants); else the threads of the row deal its packs in turn.
template <int V, bool WARP>
struct Share {
  int first, tpr;
  __device__ __forceinline__ Share(int sub, int tpr_)
      : first(WARP ? (sub & ~31) * V + (sub & 31) : sub), tpr(tpr_) {}
  __device__ __forceinline__ int step(int i) const { return WARP ? i * 32 : i * tpr; }
};

// How a thread's V packs of EPU elements are taken: in NC chunks of C elements (PP packs), the
// unit of arithmetic.
template <int EPU, int V>
struct Chunks {
  static constexpr int EPT = V * EPU, C = EPT < 8 ? EPT : 8, NC = EPT / C, PP = C / EPU;
};

// res_scale * w_post and w_pre of a thread's columns: in registers for all its rows when it has
// one chunk, else loaded where they are used (from L1).  Zero past the row's end.
template <int EPU, int V, bool WARP>
struct ColWeights {
  using K = Chunks<EPU, V>;
  float rw[K::C], wq[K::C];
  __device__ __forceinline__ void load(const NormArgs& a, const Share<V, WARP>& sh, int chunk) {
    float wp[K::C];
#pragma unroll
    for (int p = 0; p < K::PP; ++p) {
      const int c = sh.first + sh.step(chunk * K::PP + p);
#pragma unroll
      for (int m = 0; m < EPU; ++m) rw[p * EPU + m] = wq[p * EPU + m] = wp[p * EPU + m] = 0.f;
      if (c < a.packs) {
        load_cols<EPU>(a.w_post, c * EPU, wp + p * EPU);
        load_cols<EPU>(a.res_scale, c * EPU, rw + p * EPU);
        load_cols<EPU>(a.w_pre, c * EPU, wq + p * EPU);
      }
    }
    v_mul(rw, rw, wp);
  }
  __device__ __forceinline__ void init(const NormArgs& a, const Share<V, WARP>& sh) {
    if constexpr (K::NC == 1) load(a, sh, 0);
  }
  __device__ __forceinline__ void use(const NormArgs& a, const Share<V, WARP>& sh, int chunk) {
    if constexpr (K::NC > 1) load(a, sh, chunk);
  }
};

// Bytes of one ring stage for one thread: XS matrices of XT and BS of BT.
template <typename XT, typename BT, int EPU, int V, int XS, int BS>
constexpr int kRingBytes = V * EPU * (XS * (int)sizeof(XT) + BS * (int)sizeof(BT));

// One matrix's part of the ring, and its rows in memory: offsets and strides in bytes.
template <typename T, int EPU, int V, bool WARP>
struct Lane {
  using S = Slot<T, EPU>;
  using Sh = Share<V, WARP>;
  using K = Chunks<EPU, V>;
  uint32_t at, plane;  // this thread's place of the matrix in stage 0; bytes of a plane
  __device__ __forceinline__ uint32_t pack(uint32_t stage, int i) const {
    return at + stage + i * plane;
  }
  // the thread's packs of a row, into the ring (`left`: packs of the row from this thread's on)
  __device__ __forceinline__ void fetch(uint32_t stage, const char* row, int left, const Sh& sh) const {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (sh.step(i) < left) S::fetch(pack(stage, i), row + sh.step(i) * S::kBytes);
  }
  __device__ __forceinline__ void zero_tail(uint32_t stage, int left, const Sh& sh) const {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (sh.step(i) >= left) S::zero(pack(stage, i));
  }
  __device__ __forceinline__ void read(uint32_t stage, int chunk, float (&v)[K::C]) const {
#pragma unroll
    for (int p = 0; p < K::PP; ++p) S::read(pack(stage, chunk * K::PP + p), v + p * EPU);
  }
  static __device__ __forceinline__ void store(char* row, int chunk, const float (&v)[K::C], int left,
                                               const Sh& sh) {
#pragma unroll
    for (int p = 0; p < K::PP; ++p) {
      const int i = chunk * K::PP + p;
      if (sh.step(i) < left) {
        float f[EPU];
#pragma unroll
        for (int m = 0; m < EPU; ++m) f[m] = v[p * EPU + m];
        Pack<T, EPU> o;
        o.set(f);
        o.store(reinterpret_cast<T*>(row + sh.step(i) * S::kBytes));
      }
    }
  }
};

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// a thread's place in a row: base + row * step + ofs (one 32 x 32 + 64-bit multiply-add and a sum)
template <typename P>
__device__ __forceinline__ P at_row(P base, uint32_t row, uint32_t step, uint64_t ofs = 0) {
  return base + ((uint64_t)row * step + ofs);
}

// The vectors' gradients of column k from its sums of dh q and t g a.
__device__ __forceinline__ void put_cols(const NormArgs& a, int k, float pre, float t) {
  if (a.dw_pre) a.dw_pre[k] = pre;
  if (a.dw_post) a.dw_post[k] = (a.res_scale ? a.res_scale[k] : 1.f) * t;
  if (a.dres_scale) a.dres_scale[k] = (a.w_post ? a.w_post[k] : 1.f) * t;
}

template <typename BT>
__device__ __forceinline__ void row_gate(const NormArgs& a, uint32_t row, float& g, float& rest) {
  Pack<BT, 1> p;
  float z[1];
  p.load(reinterpret_cast<const BT*>(at_row(a.gate, row, a.gate_st)));
  p.get(z);
  sigmoid2(z[0], g, rest);
}

// GATE: a gate for each element.
template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
__global__ void __launch_bounds__(V * EPU > 8 ? kNormWide : kNormThreads, V * EPU > 8 ? 1 : 4) k_gated_norm(NormArgs a) {
  let_next_start();
  wait_for_earlier();
  using K = Chunks<EPU, V>;
  using LX = Lane<XT, EPU, V, WARP>;
  using LB = Lane<BT, EPU, V, WARP>;
  extern __shared__ __align__(16) char ring[];
  __shared__ __align__(16) float red_all[8 * 2 * 16];
  for (int i = threadIdx.x; i < 8 * 2 * 16; i += blockDim.x) red_all[i] = 0.f;
  const RowGroup grp{a.tpr, (int)threadIdx.x / a.tpr, (int)threadIdx.x % a.tpr};
  float* red = red_all + (a.tpr > 32 ? grp.id : 0) * 2 * 16;
  const Share<V, WARP> sh(grp.sub, a.tpr);
  const int left = a.packs - sh.first, tpr = a.tpr;
  const uint32_t plx = blockDim.x * LX::S::kBytes, plb = blockDim.x * LB::S::kBytes;
  const uint32_t stage_bytes = blockDim.x * kRingBytes<XT, BT, EPU, V, 1, GATE ? 2 : 1>;
  const uint32_t tx = smem_at(ring) + threadIdx.x * LX::S::kBytes;
  const uint32_t tb = smem_at(ring) + threadIdx.x * LB::S::kBytes + V * plx;
  const LX lx{tx, plx};
  const LB ly{tb, plb}, lg{tb + V * plb, plb};
  const uint64_t cx = (uint32_t)sh.first * LX::S::kBytes, cb = (uint32_t)sh.first * LB::S::kBytes;

  auto fetch = [&](uint32_t row, uint32_t stage) {
    if (row < a.n) {
      lx.fetch(stage, at_row(a.x, row, a.x_st, cx), left, sh);
      if (a.y) ly.fetch(stage, at_row(a.y, row, a.y_st, cb), left, sh);
      if (GATE) lg.fetch(stage, at_row(a.gate, row, a.gate_st, cb), left, sh);
    }
    ring_commit();
  };
  const uint32_t step = gridDim.x * a.rpb, last = (a.stages - 1) * stage_bytes;
  uint32_t row = blockIdx.x * a.rpb + grp.id;
  for (int s = 0; s < a.stages - 1; ++s) fetch(row + s * step, s * stage_bytes);
  ColWeights<EPU, V, WARP> cw;
  cw.init(a, sh);
  for (int s = 0; s < a.stages; ++s) {
    lx.zero_tail(s * stage_bytes, left, sh);
    ly.zero_tail(s * stage_bytes, left, sh);
    if (GATE) lg.zero_tail(s * stage_bytes, left, sh);
  }
  __syncthreads();  // red_all is cleared
  uint32_t st = 0;
  // every group runs as many rounds as the CTA's first: shuffles and barriers stay whole
  for (uint32_t r0 = blockIdx.x * a.rpb; r0 < a.n; r0 += step, row += step) {
    const bool live = row < a.n;
    fetch(row + (a.stages - 1) * step, st == 0 ? last : st - stage_bytes);
    float g_row = 1.f, rest;
    if (!GATE && a.gate_row && live) row_gate<BT>(a, row, g_row, rest);
    ring_wait(a.stages);
    float f[K::NC][K::C];  // y, then x_out
    float s[1], s2[2] = {0.f, 0.f}, ry = 0.f;
    if (a.y) {
      if (live)
#pragma unroll
        for (int i = 0; i < K::NC; ++i) {
          ly.read(st, i, f[i]);
          v_dot(s2, f[i], f[i]);
        }
      s[0] = s2[0] + s2[1];
      grp.sum(s, red);
      ry = rsqrtf(s[0] * a.inv_dim + a.eps);
      s2[0] = s2[1] = 0.f;
    }
    if (live)
#pragma unroll
      for (int i = 0; i < K::NC; ++i) {
        float x[K::C];
        lx.read(st, i, x);
        if (a.y) {
          float g[K::C];
          cw.use(a, sh, i);
          v_mul(f[i], f[i], ry);
          if (GATE) {
            lg.read(st, i, g);
#pragma unroll
            for (int m = 0; m < K::C; ++m) sigmoid2(g[m], g[m], rest);
            v_mul(g, g, cw.rw);
          } else {
            v_mul(g, cw.rw, g_row);
          }
          v_fma(x, g, f[i], x);
          LX::store(at_row(a.x_out, row, a.x_out_st, cx), i, x, left, sh);
        }
        v_dot(s2, x, x);
#pragma unroll
        for (int m = 0; m < K::C; ++m) f[i][m] = x[m];
      }
    if (a.h) {
      s[0] = s2[0] + s2[1];
      grp.sum(s, red + 16);
      const float rx = rsqrtf(s[0] * a.inv_dim + a.eps);
      if (live)
#pragma unroll
        for (int i = 0; i < K::NC; ++i) {
          cw.use(a, sh, i);
          v_mul(f[i], f[i], rx);
          v_mul(f[i], f[i], cw.wq);
          LB::store(at_row(a.h, row, a.h_st, cb), i, f[i], left, sh);
        }
    }
    // a call with one sum a row leaves no second barrier between its uses of `red`
    if ((!a.y || !a.h) && tpr > 32) asm volatile("bar.sync %0, %1;" ::"r"(grp.id + 1), "r"(tpr) : "memory");
    st = st == last ? 0 : st + stage_bytes;
  }
}

template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
__global__ void __launch_bounds__(V * EPU > 8 ? kNormWide : kNormThreads, V * EPU > 8 ? 1 : 3) k_gated_norm_bwd(NormArgs a) {
  let_next_start();
  wait_for_earlier();
  using K = Chunks<EPU, V>;
  using LX = Lane<XT, EPU, V, WARP>;
  using LB = Lane<BT, EPU, V, WARP>;
  extern __shared__ __align__(16) char ring[];
  __shared__ __align__(16) float red_all[8 * 4 * 16];
  for (int i = threadIdx.x; i < 8 * 4 * 16; i += blockDim.x) red_all[i] = 0.f;
  const RowGroup grp{a.tpr, (int)threadIdx.x / a.tpr, (int)threadIdx.x % a.tpr};
  float* red = red_all + (a.tpr > 32 ? grp.id : 0) * 4 * 16;
  const Share<V, WARP> sh(grp.sub, a.tpr);
  const int left = a.packs - sh.first, tpr = a.tpr;
  const uint32_t plx = blockDim.x * LX::S::kBytes, plb = blockDim.x * LB::S::kBytes;
  const uint32_t stage_bytes = blockDim.x * kRingBytes<XT, BT, EPU, V, 2, GATE ? 3 : 2>;
  const uint32_t mx = V * plx, mb = V * plb;  // of a matrix
  const uint32_t tx = smem_at(ring) + threadIdx.x * LX::S::kBytes;
  const uint32_t tb = smem_at(ring) + threadIdx.x * LB::S::kBytes + 2 * mx;
  const LX lx{tx, plx}, lt{tx + mx, plx};
  const LB ld{tb, plb}, ly{tb + mb, plb}, lg{tb + 2 * mb, plb};
  const uint64_t cx = (uint32_t)sh.first * LX::S::kBytes, cb = (uint32_t)sh.first * LB::S::kBytes;
  float col_pre[K::NC][K::C], col_t[K::NC][K::C];
#pragma unroll
  for (int i = 0; i < K::NC; ++i)
#pragma unroll
    for (int m = 0; m < K::C; ++m) col_pre[i][m] = col_t[i][m] = 0.f;

  auto fetch = [&](uint32_t row, uint32_t stage) {
    if (row < a.n) {
      lx.fetch(stage, at_row(a.x_out, row, a.x_out_st, cx), left, sh);
      if (a.dx_out) lt.fetch(stage, at_row(a.dx_out, row, a.dx_out_st, cx), left, sh);
      if (a.dh) ld.fetch(stage, at_row(a.dh, row, a.dh_st, cb), left, sh);
      if (a.y) ly.fetch(stage, at_row(a.y, row, a.y_st, cb), left, sh);
      if (GATE) lg.fetch(stage, at_row(a.gate, row, a.gate_st, cb), left, sh);
    }
    ring_commit();
  };
  const uint32_t step = gridDim.x * a.rpb, last = (a.stages - 1) * stage_bytes;
  uint32_t row = blockIdx.x * a.rpb + grp.id;
  for (int s = 0; s < a.stages - 1; ++s) fetch(row + s * step, s * stage_bytes);
  ColWeights<EPU, V, WARP> cw;
  cw.init(a, sh);
  for (int s = 0; s < a.stages; ++s) {
    lx.zero_tail(s * stage_bytes, left, sh);
    lt.zero_tail(s * stage_bytes, left, sh);
    ld.zero_tail(s * stage_bytes, left, sh);
    ly.zero_tail(s * stage_bytes, left, sh);
    if (GATE) lg.zero_tail(s * stage_bytes, left, sh);
  }
  __syncthreads();  // red_all is cleared
  uint32_t st = 0;
  for (uint32_t r0 = blockIdx.x * a.rpb; r0 < a.n; r0 += step, row += step) {
    const bool live = row < a.n;
    fetch(row + (a.stages - 1) * step, st == 0 ? last : st - stage_bytes);
    float g_row = 1.f, rest_row = 0.f;
    if (!GATE && a.gate_row && live) row_gate<BT>(a, row, g_row, rest_row);
    ring_wait(a.stages);
    float sx[2] = {0.f, 0.f}, sd[2] = {0.f, 0.f}, sy[2] = {0.f, 0.f};
    if (live)
#pragma unroll
      for (int i = 0; i < K::NC; ++i) {
        float x[K::C], d[K::C];
        lx.read(st, i, x);
        v_dot(sx, x, x);
        if (a.dh) {
          cw.use(a, sh, i);
          ld.read(st, i, d);
          v_mul(d, d, cw.wq);
          v_dot(sd, d, x);
        }
        if (a.y) {
          ly.read(st, i, d);
          v_dot(sy, d, d);
        }
      }
    float s[3] = {sx[0] + sx[1], sd[0] + sd[1], sy[0] + sy[1]};
    grp.sum(s, red);
    const float rx = rsqrtf(s[0] * a.inv_dim + a.eps), ry = rsqrtf(s[2] * a.inv_dim + a.eps);
    const float xm = -rx * rx * (rx * s[1] * a.inv_dim);  // x_out * xm = -q mean(dh w_pre q) / rms
    float su2[2] = {0.f, 0.f}, su[1];
    float u[K::NC][K::C];
    if (live)
#pragma unroll
      for (int i = 0; i < K::NC; ++i) {
        float t[K::C];
        cw.use(a, sh, i);
        if (a.dx_out) lt.read(st, i, t);
        else
#pragma unroll
          for (int m = 0; m < K::C; ++m) t[m] = 0.f;
        if (a.dh) {
          float x[K::C], d[K::C];
          lx.read(st, i, x);
          ld.read(st, i, d);
          v_mul(d, d, rx);
          v_fma(t, d, cw.wq, t);
          v_fma(t, x, xm, t);
          v_fma(col_pre[i], d, x, col_pre[i]);
        }
        if (a.dx) LX::store(at_row(a.dx, row, a.dx_st, cx), i, t, left, sh);
        if (a.y) {
          float y[K::C], rest[K::C];
          ly.read(st, i, y);
          v_mul(y, y, ry);
          if (GATE) {
            float g[K::C];
            lg.read(st, i, g);
#pragma unroll
            for (int m = 0; m < K::C; ++m) sigmoid2(g[m], g[m], rest[m]);
            v_mul(t, t, g);
          } else {
            v_mul(t, t, g_row);
          }
          v_fma(col_t[i], t, y, col_t[i]);
          v_mul(u[i], t, cw.rw);
          v_dot(su2, u[i], y);
          if (GATE && a.dgate) {
            v_mul(y, u[i], y);
            v_mul(y, y, rest);
            LB::store(at_row(a.dgate, row, a.dgate_st, cb), i, y, left, sh);
          }
        }
      }
    if (a.y) {
      su[0] = su2[0] + su2[1];
      grp.sum(su, red + 3 * 16);
      // one gate a row: sum of t res_scale w_post a g, times 1 - g
      if (!GATE && a.gate_row && a.dgate && live && grp.sub == 0) {
        Pack<BT, 1> p;
        const float z[1] = {su[0] * rest_row};
        p.set(z);
        p.store(reinterpret_cast<BT*>(at_row(a.dgate, row, a.dgate_st)));
      }
      const float um = -ry * ry * su[0] * a.inv_dim;
      if (a.dy && live)
#pragma unroll
        for (int i = 0; i < K::NC; ++i) {
          float y[K::C];
          ly.read(st, i, y);
          v_mul(y, y, um);
          v_fma(y, u[i], ry, y);
          LB::store(at_row(a.dy, row, a.dy_st, cb), i, y, left, sh);
        }
    } else if (tpr > 32) {  // one sum a row: no second barrier between its uses of `red`
      asm volatile("bar.sync %0, %1;" ::"r"(grp.id + 1), "r"(tpr) : "memory");
    }
    st = st == last ? 0 : st + stage_bytes;
  }
  ring_wait_n<0>();
  // the CTA's column sums: a warp's groups by shuffles, then the slices (warps, or groups of whole
  // warps) side by side in shared memory
  const int slices = tpr < 32 ? (int)blockDim.x / 32 : a.rpb;
  const int slice = tpr < 32 ? (int)threadIdx.x / 32 : grp.id;
  const bool writes = tpr >= 32 || (int)(threadIdx.x & 31) < tpr;
  float* cols = reinterpret_cast<float*>(ring);  // [slices][2][dim], when there are several
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.dim;
  const bool alone = gridDim.x == 1;  // then there is nothing to add: the results themselves
  __syncthreads();  // the ring has been read
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int m = 0; m < EPU; ++m) {
      const int e = i * EPU + m;
      float p = col_pre[e / K::C][e % K::C], q = col_t[e / K::C][e % K::C];
      if (!WARP)
        for (int o = tpr; o < 32; o <<= 1) {
          p += __shfl_xor_sync(0xFFFFFFFFu, p, o);
          q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
        }
      if (writes && sh.step(i) < left) {
        const int k = (sh.first + sh.step(i)) * EPU + m;
        if (slices > 1) cols[slice * 2 * a.dim + k] = p, cols[(slice * 2 + 1) * a.dim + k] = q;
        else if (alone) put_cols(a, k, p, q);
        else out[k] = p, out[a.dim + k] = q;
      }
    }
  }
  if (slices == 1) return;
  __syncthreads();
  for (int k = threadIdx.x; k < a.dim; k += blockDim.x) {
    float p = 0.f, q = 0.f;
    for (int r = 0; r < slices; ++r) p += cols[r * 2 * a.dim + k], q += cols[(r * 2 + 1) * a.dim + k];
    if (alone) put_cols(a, k, p, q);
    else out[k] = p, out[a.dim + k] = q;
  }
}

// Sums the CTAs' parts: 32 columns a CTA, 32 threads a column over interleaved parts, then over
// the 32 in order.
__global__ void __launch_bounds__(1024) k_gated_norm_cols(NormArgs a, int parts) {
  __shared__ float sh[2][32][33];
  let_next_start();
  wait_for_earlier();
  const float* part = a.part;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, k = blockIdx.x * 32 + lane, dim = a.dim;
  float p = 0.f, t = 0.f;
  for (int g0 = slice; g0 < parts; g0 += 32 * 8) {  // 8 CTAs' parts loaded together
    float c[8], d[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = g0 + u * 32 < parts && k < dim;
      const float* q = part + (int64_t)(g0 + u * 32) * 2 * dim + k;
      c[u] = in ? __ldcg(q) : 0.f;
      d[u] = in ? __ldcg(q + dim) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) p += c[u], t += d[u];
  }
  sh[0][slice][lane] = p;
  sh[1][slice][lane] = t;
  __syncthreads();
  // warp c (of 32) sums column c: lane = slice
  const int col = blockIdx.x * 32 + slice;
  p = lanes_sum(sh[0][lane][slice], 32);
  t = lanes_sum(sh[1][lane][slice], 32);
  if (lane == 0 && col < dim) {
    put_cols(a, col, p, t);
  }
}

// ---- host ----

// Threads of a row: for 8 elements each (16 in rows of more than 2048), a power of two up to a
// warp, whole warps above.
static void norm_shape(NormArgs& a, int epu) {
  a.packs = a.dim / epu;
  const int each = a.dim > 8 * kNormThreads ? 16 : 8, want = (a.dim + each - 1) / each;
  int t = 4;
  while (t < want && t < 32) t *= 2;
  if (want > 32) t = (want + 31) / 32 * 32;
  a.tpr = t;
  a.rpb = t >= kNormThreads ? 1 : kNormThreads / t;
}

// CTAs an SM holds: `per` by registers (the kernels' launch bounds), fewer where shared memory
// (the ring, and up to 3 KB beside it) allows no more.
static int norm_fit(int per, int smem) {
  const int fit = 227 * 1024 / (smem + 3 * 1024);
  return fit < per ? fit : per;
}

// Ring stages and their bytes: kStages, but two where that puts more CTAs on an SM (as many rows
// are in flight either way, and more warps hide the arithmetic), and one for the widest rows.
static int norm_ring(NormArgs& a, int thread_bytes, int per) {
  const int bytes = a.rpb * a.tpr * thread_bytes;
  a.stages = kStages;
  while (a.stages > 1) {
    const int fit = norm_fit(per, a.stages * bytes);
    if (fit > 0 && (a.stages == 2 || fit == norm_fit(per, (a.stages - 1) * bytes))) break;
    --a.stages;
  }
  return a.stages * bytes;
}

static NormArgs norm_args(const emb_norm& p) {
  const int xe = p.x_dtype == EMB_BF16 ? 2 : 4, be = p.dtype == EMB_BF16 ? 2 : 4;
  const auto in = [](const void* q) { return static_cast<const char*>(q); };
  const auto out = [](void* q) { return static_cast<char*>(q); };
  NormArgs a{};
  a.n = (uint32_t)p.n, a.dim = p.dim, a.gate_row = p.d_gate && p.gate_cols == 1;
  a.eps = p.eps, a.inv_dim = 1.f / (float)p.dim;
  a.x = in(p.d_x), a.y = in(p.d_y), a.gate = in(p.d_gate), a.dx_out = in(p.d_dx_out), a.dh = in(p.d_dh);
  a.x_out = out(p.d_x_out), a.h = out(p.d_h), a.dx = out(p.d_dx), a.dy = out(p.d_dy);
  a.dgate = out(p.d_dgate);
  a.x_st = (uint32_t)(p.x_ld * xe), a.x_out_st = (uint32_t)(p.x_out_ld * xe);
  a.dx_out_st = (uint32_t)(p.dx_out_ld * xe), a.dx_st = (uint32_t)(p.dx_ld * xe);
  a.y_st = (uint32_t)(p.y_ld * be), a.gate_st = (uint32_t)(p.gate_ld * be);
  a.h_st = (uint32_t)(p.h_ld * be), a.dh_st = (uint32_t)(p.dh_ld * be);
  a.dy_st = (uint32_t)(p.dy_ld * be), a.dgate_st = (uint32_t)(p.dgate_ld * be);
  a.w_post = p.d_w_post, a.res_scale = p.d_res_scale, a.w_pre = p.d_w_pre;
  a.dw_post = p.d_dw_post, a.dres_scale = p.d_dres_scale, a.dw_pre = p.d_dw_pre;
  return a;
}

// Whether every matrix of the call (NULL: none) allows packs of more than one element.
static bool norm_vec(const emb_norm& p) {
  const int xe = p.x_dtype == EMB_BF16 ? 2 : 4, be = p.dtype == EMB_BF16 ? 2 : 4;
  const int epu = xe == 2 ? 8 : 4, bb = epu * be;  // elements of a pack, bytes of a block's
  return p.dim % epu == 0 && rows16(p.d_x, p.x_ld, xe) && rows_on(p.d_y, p.y_ld, be, bb) &&
         (p.gate_cols == 1 || rows_on(p.d_gate, p.gate_ld, be, bb)) &&
         rows16(p.d_x_out, p.x_out_ld, xe) && rows_on(p.d_h, p.h_ld, be, bb) &&
         rows16(p.d_dx_out, p.dx_out_ld, xe) && rows_on(p.d_dh, p.dh_ld, be, bb) &&
         rows16(p.d_dx, p.dx_ld, xe) && rows_on(p.d_dy, p.dy_ld, be, bb) &&
         (p.gate_cols == 1 || rows_on(p.d_dgate, p.dgate_ld, be, bb)) && rows16(p.d_w_post, 0, 4) &&
         rows16(p.d_res_scale, 0, 4) && rows16(p.d_w_pre, 0, 4);
}

template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
static cudaError_t norm_fwd_v(NormArgs& a, cudaStream_t s) {
  const int threads = a.rpb * a.tpr, per = V * EPU > 8 ? kNormWide / threads : 4;
  const int smem = norm_ring(a, kRingBytes<XT, BT, EPU, V, 1, GATE ? 2 : 1>, per);
  constexpr auto kern = k_gated_norm<XT, BT, EPU, V, GATE, WARP>;
  const int64_t blocks = ((int64_t)a.n + a.rpb - 1) / a.rpb, cap = (int64_t)device_sms() * norm_fit(per, smem);
  const cudaError_t e = prepare_kernel<kern>();
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)(blocks < cap ? blocks : cap), threads, smem, s, a);
}

// CTAs of the backward: a row a group up to one CTA an SM, then at least four rows a group up to
// `cap`, so that the column parts stay small beside the rows.
static int64_t norm_bwd_grid(int64_t n, int rpb, int64_t cap) {
  const int64_t sms = device_sms(), all = (n + rpb - 1) / rpb, four = (n + 4 * rpb - 1) / (4 * rpb);
  const int64_t blocks = all <= sms ? all : four > sms ? four : sms;
  return blocks < 1 ? 1 : blocks < cap ? blocks : cap;
}

constexpr int kNormCtasPerSm = 3;  // CTAs of the backward per SM, at most (wide rows: 160 threads and more)

int64_t gated_norm_bwd_workspace(int64_t n, int dim) {
  NormArgs a{};
  a.dim = dim;
  norm_shape(a, 1);
  return norm_bwd_grid(n, a.rpb, (int64_t)device_sms() * kNormCtasPerSm) * 2 * dim * (int64_t)sizeof(float);
}

template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
static cudaError_t norm_bwd_v(NormArgs& a, int* grid, cudaStream_t s) {
  const int threads = a.rpb * a.tpr, per = V * EPU > 8 ? kNormWide / threads : kNormCtasPerSm;
  int smem = norm_ring(a, kRingBytes<XT, BT, EPU, V, 2, GATE ? 3 : 2>, per);
  const int slices = a.tpr < 32 ? threads / 32 : a.rpb;
  const int cols = slices > 1 ? slices * 2 * a.dim * (int)sizeof(float) : 0;
  if (smem < cols) smem = cols;
  constexpr auto kern = k_gated_norm_bwd<XT, BT, EPU, V, GATE, WARP>;
  const cudaError_t e = prepare_kernel<kern>();
  if (e != cudaSuccess) return e;
  *grid = (int)norm_bwd_grid(a.n, a.rpb, (int64_t)device_sms() * norm_fit(per, smem));
  return launch_early(kern, (unsigned)*grid, threads, smem, s, a);
}

// The kernel of a call by packs per thread (1, 2, 4, 8 or 16: at most 16 elements), gate and
// threads per row.  Rows of 16 elements a thread always take whole warps.
template <typename XT, typename BT, int EPU, bool BWD, int V = 1>
static cudaError_t norm_t(NormArgs& a, int* grid, cudaStream_t s) {
  if constexpr (V == 1) norm_shape(a, EPU);
  if constexpr (V * EPU < 16)
    if ((a.packs + a.tpr - 1) / a.tpr > V) return norm_t<XT, BT, EPU, BWD, 2 * V>(a, grid, s);
  const auto run = [&](auto gate, auto warp) {
    constexpr bool G = decltype(gate)::value, W = decltype(warp)::value;
    if constexpr (BWD) return norm_bwd_v<XT, BT, EPU, V, G, W>(a, grid, s);
    else return norm_fwd_v<XT, BT, EPU, V, G, W>(a, s);
  };
  const bool gate = a.gate && !a.gate_row;
  if constexpr (V * EPU <= 8)
    if (a.tpr < 32 || V == 1) return gate ? run(std::true_type{}, std::false_type{}) : run(std::false_type{}, std::false_type{});
  if constexpr (V > 1) return gate ? run(std::true_type{}, std::true_type{}) : run(std::false_type{}, std::true_type{});
  return cudaErrorInvalidValue;  // not reached: one pack a thread was taken above
}

template <bool BWD>
static cudaError_t norm_call(const emb_norm& p, NormArgs& a, int* grid, cudaStream_t s) {
  const bool vec = norm_vec(p);
  using H = __nv_bfloat16;
  if (p.dtype == EMB_F32)
    return vec ? norm_t<float, float, 4, BWD>(a, grid, s) : norm_t<float, float, 1, BWD>(a, grid, s);
  if (p.x_dtype == EMB_F32)
    return vec ? norm_t<float, H, 4, BWD>(a, grid, s) : norm_t<float, H, 1, BWD>(a, grid, s);
  return vec ? norm_t<H, H, 8, BWD>(a, grid, s) : norm_t<H, H, 1, BWD>(a, grid, s);
}

cudaError_t launch_gated_norm(const emb_norm& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  NormArgs a = norm_args(p);
  return norm_call<false>(p, a, nullptr, s);
}

cudaError_t launch_gated_norm_bwd(const emb_norm& p, void* ws, cudaStream_t s) {
  NormArgs a = norm_args(p);
  a.part = static_cast<float*>(ws);
  int grid = 0;
  cudaError_t e = p.n > 0 ? norm_call<true>(p, a, &grid, s) : cudaSuccess;
  if (e != cudaSuccess || grid == 1 || !(p.d_dw_post || p.d_dres_scale || p.d_dw_pre)) return e;
  return launch_early(k_gated_norm_cols, (p.dim + 31) / 32, 1024, 0, s, a, grid);
}

}  // namespace emb
