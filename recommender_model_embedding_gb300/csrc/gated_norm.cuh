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
// Both are bound by HBM bandwidth while there are bytes enough for each row's chain of work (loads,
// two row sums one after the other, arithmetic), and by that chain where there are not: the forward
// takes about 300 warp instructions a warp's share of a row (8 elements a thread), the backward
// 530, with 24 warps an SM to hide one another's waits.  Measured with a gate for each element, 262144 x 1024: forward with
// an fp32 stream and bf16 blocks 3.76 GB in 0.555 ms (6.77 TB/s, the measured copy rate), backward
// all in bf16 4.29 GB in 0.679 ms (6.32 TB/s, 93%); with one gate a row the bf16 backward reaches
// 75% there and 59% at 65536 x 2048, where it issues in 64% of the cycles and has DRAM busy for
// 46%; fp32 reaches 90% at 262144 x 1024.
//
// A group of `tpr` threads takes a row, about eight elements a thread (V packs of EPU: 16 bytes
// a pack where everything is aligned, else 4 or one element; with an fp32 stream beside bf16
// blocks 4 elements, 16 and 8 bytes, so that neighbouring threads' accesses of either type are
// neighbours in memory: with 8, half-filled sectors took 0.72 ms, not 0.57), so a row costs each
// thread few shuffles per element.  CTAs are persistent; every thread copies its own packs of
// the next rows to shared memory asynchronously, up to two rows ahead, and reads back only what
// it copied itself, so the ring needs no barrier (a row loaded only when its turn came: 2.88 ms
// backward, 1.17 ms forward); the groups of a CTA run independently of each other (named
// barriers for the row sums, and only for rows of more than 32 threads).  Packs past the row's
// end are zero in the ring, which takes the place of masks.  The backward computes everything
// but dy in one sweep over the row, since only dy needs the second row sum: it keeps u in
// registers and y in the ring.  A thread has the same columns for all its rows, so the column
// sums stay in its registers until the end, when they go to the workspace and a second launch
// adds the CTAs' parts in a fixed order (6 us; a single CTA writes the results itself).
#pragma once

#include "rows_common.cuh"

namespace emb {

// Threads: a CTA of narrow rows has 256.  A row has 8 elements a thread while that takes up to
// kNormForward threads forward, and backward kNormBackward for packs of four elements and more (two
// such CTAs fill an SM's registers, 64 and 80 a thread), kNormThreads for narrower ones (128
// registers); 16 above.
constexpr int kNormThreads = 256, kNormForward = 512, kNormBackward = 384, kNormWide = 512;
constexpr int kStages = 3;  // rows of the ring

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
  // backward: [CTAs][2][dim] column sums, and whether any vector's gradient is asked for
  float* part;
  int cols;
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

// g = sigmoid(z) = 1 / (1 + e) and rest = 1 - g = e g, with e = exp(-z), to a few units in the last
// place at every z.  The fast exponential 2^t of t = -z / ln 2 alone would be off by the rounding
// of t, about z 2^-24 of itself (58 units of 2^-24 in g at z = -80); with d = -z - t ln 2, which
// is that rounding's size, e = 2^t exp(d) = 2^t (1 + d) to within d^2 < 2^-34.  z is held to where
// e neither overflows nor leaves infinities to subtract in d: from 104 on e is zero in fp32 anyway,
// and from -87.4 down g is zero, and rest too, which is only ever multiplied by g.  NaN stays.
// In pairs, and with no choice between 1 - g and e g by the sign of z, this costs the backward little
// (262144 x 1024 bf16 with a gate for each element: 666 us with 2^t alone, 678 so, 709 with expf).
template <int N>
__device__ __forceinline__ void v_sigmoid(const float (&gate)[N], float (&g)[N], float (&rest)[N]) {
  constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Rest = -1.90465421e-9f;
  constexpr int P = N < 2 ? 1 : 2;
#pragma unroll
  for (int m = 0; m < N; m += P) {
    float z[P], t[P], d[P], e[P], q[P], one[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(z[i]) : "f"(-gate[m + i]), "f"(-104.f));
      asm("min.NaN.f32 %0, %1, %2;" : "=f"(z[i]) : "f"(z[i]), "f"(88.f));
      one[i] = 1.f;
    }
    v_mul(t, z, kLog2e);
#pragma unroll
    for (int i = 0; i < P; ++i) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e[i]) : "f"(t[i]));
    v_fma(d, t, -kLn2, z);
    v_fma(d, t, -kLn2Rest, d);
    v_fma(e, e, d, e);
    v_fma(t, e, 1.f, one);
#pragma unroll
    for (int i = 0; i < P; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q[i]) : "f"(t[i]));
    v_mul(e, e, q);
#pragma unroll
    for (int i = 0; i < P; ++i) g[m + i] = q[i], rest[m + i] = e[i];
  }
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

// (Ordinary loads: an early-launched kernel is there before the work ahead of it has written its last,
// so nothing that it reads is read-only for as long as it runs.)
template <int EPU>
__device__ __forceinline__ void load_cols(const float* w, int col, float* v) {
  if constexpr (EPU >= 4) {
#pragma unroll
    for (int m = 0; m < EPU; m += 4) {
      const float4 f = w ? *reinterpret_cast<const float4*>(w + col + m)
                         : make_float4(1.f, 1.f, 1.f, 1.f);
      v[m] = f.x, v[m + 1] = f.y, v[m + 2] = f.z, v[m + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int m = 0; m < EPU; ++m) v[m] = w ? w[col + m] : 1.f;
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

// res_scale * w_post and w_pre of a thread's columns, zero past the row's end: in registers for all
// its rows when it has one chunk, else in shared memory for the CTA (in L1 they would be driven
// out by the rows).  shared: [2][threads of a row * elements of a thread].
template <int EPU, int V, bool WARP>
struct ColWeights {
  using K = Chunks<EPU, V>;
  static constexpr bool kShared = K::NC > 1;
  float rw[K::C], wq[K::C];
  uint32_t at;  // kShared: the shared copy
  __device__ __forceinline__ void init(const NormArgs& a, const Share<V, WARP>& sh, float* shared) {
    if constexpr (kShared) {
      const int n = a.tpr * K::EPT;  // a row a CTA: EPT columns a thread
#pragma unroll
      for (int j0 = 0; j0 < K::EPT; j0 += 8) {
        float wp[8], rs[8], wn[8];  // loaded together
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int k = threadIdx.x + (j0 + j) * a.tpr;
          const bool in = k < a.dim;
          wp[j] = in ? a.w_post ? a.w_post[k] : 1.f : 0.f;
          rs[j] = in ? a.res_scale ? a.res_scale[k] : 1.f : 0.f;
          wn[j] = in ? a.w_pre ? a.w_pre[k] : 1.f : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int k = threadIdx.x + (j0 + j) * a.tpr;
          shared[k] = wp[j] * rs[j];
          shared[n + k] = wn[j];
        }
      }
      at = (uint32_t)__cvta_generic_to_shared(shared + sh.first * EPU);
    } else {
      float wp[K::C];
#pragma unroll
      for (int p = 0; p < K::PP; ++p) {
        const int c = sh.first + sh.step(p);
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
  }
  __device__ __forceinline__ void read(uint32_t from, const Share<V, WARP>& sh, int chunk, float (&v)[K::C]) {
#pragma unroll
    for (int p = 0; p < K::PP; ++p) {
      const uint32_t q = from + (uint32_t)sh.step(chunk * K::PP + p) * (EPU * 4);
#pragma unroll
      for (int m = 0; m < EPU; m += EPU < 4 ? 1 : 4) {
        float* d = v + p * EPU + m;
        if constexpr (EPU < 4)
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(d[0]) : "r"(q + m * 4));
        else
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(q + m * 4));
      }
    }
  }
  __device__ __forceinline__ void use_rw(const NormArgs& a, const Share<V, WARP>& sh, int chunk) {
    if constexpr (kShared) read(at, sh, chunk, rw);
  }
  __device__ __forceinline__ void use_wq(const NormArgs& a, const Share<V, WARP>& sh, int chunk) {
    if constexpr (kShared) read(at + (uint32_t)(a.tpr * K::EPT) * 4, sh, chunk, wq);
  }
};

// Whether a thread's packs of the next row wait in registers instead of the ring, for small packs,
// up to 8 elements: there a ring would take two more instructions of the same pipe for every few
// bytes, and single bf16 elements have no asynchronous copy at all.  Packs of one element:
// forward of 16411 x 479 fp32 33 us through the ring, 27 so; of 83781 x 801 bf16 225 and 169,
// backward 466 and 339.  Packs of two, 83676 x 802 bf16: backward 275 and 240, but the forward,
// with more rows in flight through the ring, 140 and 148; wider packs lose in the backward too
// (262144 x 1024 bf16: 0.67 ms and 0.71, before the gate's error was carried along).
template <int EPU, int V>
constexpr bool kAheadForward = EPU == 1 && V <= 8;
template <int EPU, int V>
constexpr bool kAheadBackward = EPU <= 2 && V * EPU <= 8;

// Bytes of one ring stage for one thread: XS matrices of XT and BS of BT.
template <typename XT, typename BT, int EPU, int V, int XS, int BS>
constexpr int kRingBytes = V * EPU * (XS * (int)sizeof(XT) + BS * (int)sizeof(BT));

// One matrix's part of the ring, and its rows in memory: offsets and strides in bytes.
template <typename T, int EPU, int V, bool WARP, bool AHEAD>
struct Lane {
  using S = Slot<T, EPU>;
  using Sh = Share<V, WARP>;
  using K = Chunks<EPU, V>;
  uint32_t at, plane;  // this thread's place of the matrix in stage 0; bytes of a plane
  static constexpr int W = S::kBytes < 4 ? 1 : S::kBytes / 4;  // words of a pack
  uint32_t now[AHEAD ? V * W : 1], next[AHEAD ? V * W : 1];  // AHEAD: the packs
  __device__ __forceinline__ Lane(uint32_t at_, uint32_t plane_) : at(at_), plane(plane_) {}
  __device__ __forceinline__ uint32_t pack(uint32_t stage, int i) const {
    return at + stage + i * plane;
  }
  // the thread's packs of a row, into the ring (`left`: packs of the row from this thread's on)
  __device__ __forceinline__ void fetch(uint32_t stage, const char* row, int left, const Sh& sh) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (AHEAD) {
#pragma unroll
        for (int w = 0; w < W; ++w) next[i * W + w] = 0;
        if (sh.step(i) < left) {
          const char* p = row + sh.step(i) * S::kBytes;
          if constexpr (S::kBytes == 2) {
            next[i] = *reinterpret_cast<const uint16_t*>(p);
          } else if constexpr (S::kBytes == 4) {
            next[i] = *reinterpret_cast<const uint32_t*>(p);
          } else {
            static_assert(S::kBytes == 8, "packs of up to two elements");
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            next[i * 2] = q.x, next[i * 2 + 1] = q.y;
          }
        }
      } else if (sh.step(i) < left) {
        S::fetch(pack(stage, i), row + sh.step(i) * S::kBytes);
      }
    }
  }
  __device__ __forceinline__ void advance() {  // AHEAD: the row fetched last becomes the current one
#pragma unroll
    for (int i = 0; i < (AHEAD ? V * W : 0); ++i) now[i] = next[i];
  }
  __device__ __forceinline__ void zero_tail(uint32_t stage, int left, const Sh& sh) const {
    if constexpr (!AHEAD)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (sh.step(i) >= left) S::zero(pack(stage, i));
  }
  __device__ __forceinline__ void read(uint32_t stage, int chunk, float (&v)[K::C]) const {
#pragma unroll
    for (int p = 0; p < K::PP; ++p) {
      if constexpr (AHEAD) {
        const int i = (chunk * K::PP + p) * W;
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          if constexpr (sizeof(T) == 4) v[p * EPU + m] = __uint_as_float(now[i + m]);
          else v[p * EPU + m] = __uint_as_float(m % 2 ? now[i + m / 2] & 0xFFFF0000u : now[i + m / 2] << 16);
        }
      } else {
        S::read(pack(stage, chunk * K::PP + p), v + p * EPU);
      }
    }
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

// One gate for a row, loaded a round ahead of its use.
template <typename BT>
struct RowGate {
  Pack<BT, 1> next;
  __device__ __forceinline__ void fetch(const NormArgs& a, uint32_t row) {
    next.zero();
    if (a.gate_row && row < a.n) next.load(reinterpret_cast<const BT*>(at_row(a.gate, row, a.gate_st)));
  }
  // the gate fetched last, and 1 - gate; fetches the one of row `then`
  __device__ __forceinline__ void take(const NormArgs& a, uint32_t then, float& g, float& rest) {
    float z[1], gs[1], rs[1];
    next.get(z);
    fetch(a, then);
    g = 1.f, rest = 0.f;
    if (!a.gate_row) return;
    v_sigmoid(z, gs, rs);
    g = gs[0], rest = rs[0];
  }
};

// ---- host ----

// Threads of a row: for 8 elements each while that is at most `most` threads, else 16; a power of
// two up to a warp, whole warps above.
inline void norm_shape(NormArgs& a, int epu, int most) {
  a.packs = a.dim / epu;
  const int each = a.dim > 8 * most ? 16 : 8, want = (a.dim + each - 1) / each;
  int t = 4;
  while (t < want && t < 32) t *= 2;
  if (want > 32) t = (want + 31) / 32 * 32;
  a.tpr = t;
  a.rpb = t >= kNormThreads ? 1 : kNormThreads / t;
}

// CTAs an SM holds: `per` by registers (the kernels' launch bounds), fewer where shared memory
// (the ring, and up to 3 KB beside it) allows no more.
inline int norm_fit(int per, int smem) {
  const int fit = 227 * 1024 / (smem + 3 * 1024);
  return fit < per ? fit : per;
}

// Ring stages, and the bytes of shared memory with them: kStages, but two where that puts more
// CTAs on an SM (as many rows are in flight either way, and more warps hide the arithmetic),
// and one for the widest rows.  `extra`: bytes beside the ring.
inline int norm_ring(NormArgs& a, int thread_bytes, int per, int extra) {
  const int bytes = a.rpb * a.tpr * thread_bytes;
  a.stages = bytes ? kStages : 2;  // (in registers: the next row)
  while (a.stages > 1) {
    const int fit = norm_fit(per, a.stages * bytes + extra);
    if (fit > 0 && (a.stages == 2 || fit == norm_fit(per, (a.stages - 1) * bytes + extra))) break;
    --a.stages;
  }
  return a.stages * bytes + extra;
}

inline NormArgs norm_args(const emb_norm& p) {
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

// Elements of a pack: what every matrix of the call (NULL: none) allows, 16 bytes at most.
inline bool norm_allows(const emb_norm& p, int epu) {
  const int xe = p.x_dtype == EMB_BF16 ? 2 : 4, be = p.dtype == EMB_BF16 ? 2 : 4;
  const int xb = epu * xe, bb = epu * be, wb = epu < 4 ? epu * 4 : 16;
  return p.dim % epu == 0 && rows_on(p.d_x, p.x_ld, xe, xb) && rows_on(p.d_y, p.y_ld, be, bb) &&
         (p.gate_cols == 1 || rows_on(p.d_gate, p.gate_ld, be, bb)) &&
         rows_on(p.d_x_out, p.x_out_ld, xe, xb) && rows_on(p.d_h, p.h_ld, be, bb) &&
         rows_on(p.d_dx_out, p.dx_out_ld, xe, xb) && rows_on(p.d_dh, p.dh_ld, be, bb) &&
         rows_on(p.d_dx, p.dx_ld, xe, xb) && rows_on(p.d_dy, p.dy_ld, be, bb) &&
         (p.gate_cols == 1 || rows_on(p.d_dgate, p.dgate_ld, be, bb)) && rows_on(p.d_w_post, 0, 4, wb) &&
         rows_on(p.d_res_scale, 0, 4, wb) && rows_on(p.d_w_pre, 0, 4, wb);
}

// Call::run for a call, by packs per thread (1, 2, 4, 8 or 16: at most 16 elements), gate and
// threads per row.  Rows of 16 elements a thread always take whole warps.
template <typename Call, typename XT, typename BT, int EPU, int V = 1>
cudaError_t norm_t(NormArgs& a, Call call) {
  if constexpr (V == 1) norm_shape(a, EPU, Call::most(EPU));
  if constexpr (V * EPU < 16)
    if ((a.packs + a.tpr - 1) / a.tpr > V) return norm_t<Call, XT, BT, EPU, 2 * V>(a, call);
  const auto run = [&](auto gate, auto warp) {
    constexpr bool G = decltype(gate)::value, W = decltype(warp)::value;
    return call.template run<XT, BT, EPU, V, G, W>(a);
  };
  const bool gate = a.gate && !a.gate_row;
  if constexpr (V * EPU <= 8)
    if (a.tpr < 32 || V == 1) return gate ? run(std::true_type{}, std::false_type{}) : run(std::false_type{}, std::false_type{});
  if constexpr (V > 1) return gate ? run(std::true_type{}, std::true_type{}) : run(std::false_type{}, std::true_type{});
  return cudaErrorInvalidValue;  // not reached: one pack a thread was taken above
}

template <typename Call>
cudaError_t norm_call(const emb_norm& p, NormArgs& a, Call call) {
  using H = __nv_bfloat16;
  const bool bf = p.dtype == EMB_BF16, xbf = p.x_dtype == EMB_BF16;
  if (norm_allows(p, xbf ? 8 : 4))
    return !bf ? norm_t<Call, float, float, 4>(a, call)
           : !xbf ? norm_t<Call, float, H, 4>(a, call)
                  : norm_t<Call, H, H, 8>(a, call);
  if (bf && norm_allows(p, 2))
    return !xbf ? norm_t<Call, float, H, 2>(a, call) : norm_t<Call, H, H, 2>(a, call);
  return !bf ? norm_t<Call, float, float, 1>(a, call)
         : !xbf ? norm_t<Call, float, H, 1>(a, call)
                : norm_t<Call, H, H, 1>(a, call);
}

}  // namespace emb
