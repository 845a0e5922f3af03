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
// thread (V packs of EPU: 16 bytes a pack where everything is aligned, one element otherwise),
// so a row costs each thread few shuffles per element.  CTAs are persistent; every thread
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

constexpr int kNormThreads = 256;     // of a CTA, unless a row takes more
constexpr int kNormMaxThreads = 512;  // of a row
constexpr int kStages = 3;            // rows of the ring

struct NormArgs {
  int64_t n;
  int dim, packs, tpr;  // packs of EPU elements of a row; threads of a row
  int rpb;              // rows side by side in a CTA
  int stages;           // of the ring: 1 .. kStages
  int gate_cols;        // 0, 1 or dim
  float eps, inv_dim;
  const void *x, *y, *gate, *dx_out, *dh;
  void *x_out, *h, *dx, *dy, *dgate;
  int64_t x_ld, y_ld, gate_ld, dx_out_ld, dh_ld, x_out_ld, h_ld, dx_ld, dy_ld, dgate_ld;
  const float *w_post, *res_scale, *w_pre;
  float* part;  // [CTAs][2][dim] column sums (backward)
};

// sigmoid(z) and 1 - sigmoid(z), each to a few units in the last place at either end (the
// smaller of the two is e / (1 + e), not a difference); |z| e^-|z| < 1/2, so the fast
// exponential's argument error stays below one unit too.
__device__ __forceinline__ void sigmoid2(float z, float& g, float& rest) {
  const float e = __expf(-fabsf(z)), r = __fdividef(1.f, 1.f + e), er = e * r;
  g = z >= 0.f ? r : er;
  rest = z >= 0.f ? er : r;
}

// The ring: one plane of UB bytes a thread for each 16 bytes (or element) of a pack.
template <typename T, int EPU>
struct Slot {
  static constexpr int kBytes = EPU * (int)sizeof(T);
  static constexpr int UB = kBytes < 16 ? kBytes : 16, kPlanes = kBytes / UB;

  // starts the copy of the pack at p to this thread's place of the planes from `to` on
  static __device__ __forceinline__ void fetch(uint32_t to, uint32_t plane, const T* p) {
    if constexpr (UB >= 4) {
#pragma unroll
      for (int i = 0; i < kPlanes; ++i)
        if constexpr (UB == 16)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * plane),
                       "l"(reinterpret_cast<const char*>(p) + i * 16) : "memory");
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p) : "memory");
    } else {  // one bf16: too small for an asynchronous copy
      const uint16_t v = *reinterpret_cast<const uint16_t*>(p);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(v) : "memory");
    }
  }
  static __device__ __forceinline__ void read(uint32_t from, uint32_t plane, float (&v)[EPU]) {
    if constexpr (UB == 16) {
      uint32_t w[4 * kPlanes];
#pragma unroll
      for (int i = 0; i < kPlanes; ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(from + i * plane) : "memory");
#pragma unroll
      for (int i = 0; i < EPU; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
        else v[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      }
    } else if constexpr (UB == 4) {
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(from) : "memory");
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
  // Sums of NS values over the group, the same in every thread.  `red`: NS * 16 floats of the
  // group's own, not used again before another sum of the group has passed its barrier.
  template <int NS>
  __device__ __forceinline__ void sum(float (&v)[NS], float* red) const {
    const int width = tpr < 32 ? tpr : 32;
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = lanes_sum(v[i], width);
    if (tpr > 32) {
      const int lane = sub & 31, warp = sub >> 5, warps = tpr >> 5;
      if (lane == 0)
#pragma unroll
        for (int i = 0; i < NS; ++i) red[i * 16 + warp] = v[i];
      asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(tpr) : "memory");
      if (warps <= 4) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          v[i] = red[i * 16];
          for (int w = 1; w < warps; ++w) v[i] += red[i * 16 + w];
        }
      } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) v[i] = lanes_sum(lane < warps ? red[i * 16 + lane] : 0.f, 32);
      }
    }
  }
};

template <int EPU>
__device__ __forceinline__ void load_cols(const float* w, int col, float (&v)[EPU]) {
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

// res_scale * w_post and w_pre of a thread's columns: in registers for all its rows when it has
// one pack, else loaded where they are used (from L1).
template <int EPU, int V>
struct ColWeights {
  static constexpr bool kKeep = V == 1 || EPU == 1;
  static constexpr int N = kKeep ? V : 1;
  float rw[N][EPU], wq[N][EPU];
  __device__ __forceinline__ void load(const NormArgs& a, int i, int at) {
    float wp[EPU];
    load_cols<EPU>(a.w_post, at, wp);
    load_cols<EPU>(a.res_scale, at, rw[i]);
    load_cols<EPU>(a.w_pre, at, wq[i]);
#pragma unroll
    for (int m = 0; m < EPU; ++m) rw[i][m] *= wp[m];
  }
  __device__ __forceinline__ void init(const NormArgs& a, int sub) {
    if constexpr (kKeep)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (sub + i * a.tpr < a.packs) load(a, i, (sub + i * a.tpr) * EPU);
  }
  __device__ __forceinline__ int use(const NormArgs& a, int i, int at) {
    if constexpr (kKeep) return i;
    load(a, 0, at);
    return 0;
  }
};

// Bytes of one ring stage for one thread: XS matrices of XT and BS of BT.
template <typename XT, typename BT, int EPU, int V, int XS, int BS>
constexpr int kRingBytes = V * EPU * (XS * (int)sizeof(XT) + BS * (int)sizeof(BT));

__device__ __forceinline__ uint32_t smem_at(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

template <typename XT, typename BT, int EPU, int V>
__global__ void __launch_bounds__(kNormMaxThreads) k_gated_norm(NormArgs a) {
  using SX = Slot<XT, EPU>;
  using SB = Slot<BT, EPU>;
  extern __shared__ __align__(16) char ring[];
  __shared__ float red_all[2 * 16 * 16];
  const uint32_t plx = blockDim.x * SX::UB, plb = blockDim.x * SB::UB;  // bytes of a plane
  const RowGroup grp{a.tpr, (int)threadIdx.x / a.tpr, (int)threadIdx.x % a.tpr};
  float* red = red_all + (a.tpr > 32 ? grp.id : 0) * 2 * 16;
  const uint32_t stage_bytes = blockDim.x * kRingBytes<XT, BT, EPU, V, 1, 2>;
  const uint32_t ring0 = smem_at(ring);
  const uint32_t ofs_y = V * SX::kPlanes * plx, ofs_g = ofs_y + V * SB::kPlanes * plb;
  const uint32_t tx = ring0 + threadIdx.x * SX::UB, tb = ring0 + threadIdx.x * SB::UB;
  const int64_t step = (int64_t)gridDim.x * a.rpb;
  ColWeights<EPU, V> cw;
  cw.init(a, grp.sub);

  auto fetch = [&](int64_t row, int stage) {
    if (row < a.n) {
      const uint32_t sb = stage * stage_bytes;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = grp.sub + i * a.tpr;
        if (c < a.packs) {
          const int64_t at = (int64_t)c * EPU;
          SX::fetch(tx + sb + i * SX::kPlanes * plx, plx, static_cast<const XT*>(a.x) + row * a.x_ld + at);
          if (a.y)
            SB::fetch(tb + sb + ofs_y + i * SB::kPlanes * plb, plb,
                      static_cast<const BT*>(a.y) + row * a.y_ld + at);
          if (a.gate_cols > 1)
            SB::fetch(tb + sb + ofs_g + i * SB::kPlanes * plb, plb,
                      static_cast<const BT*>(a.gate) + row * a.gate_ld + at);
        }
      }
    }
    ring_commit();
  };
  int64_t row = (int64_t)blockIdx.x * a.rpb + grp.id;
  for (int s = 0; s < a.stages - 1; ++s) fetch(row + s * step, s);
  int st = 0;
  // every group runs as many rounds as the CTA's first: shuffles and barriers stay whole
  for (int64_t r0 = (int64_t)blockIdx.x * a.rpb; r0 < a.n; r0 += step, row += step) {
    const bool live = row < a.n;
    fetch(row + (a.stages - 1) * step, st == 0 ? a.stages - 1 : st - 1);
    float g_row = 1.f, rest;
    if (a.gate_cols == 1 && live) {
      Pack<BT, 1> p;
      float z[1];
      p.load(static_cast<const BT*>(a.gate) + row * a.gate_ld);
      p.get(z);
      sigmoid2(z[0], g_row, rest);
    }
    ring_wait(a.stages);
    const uint32_t sb = st * stage_bytes;
    float s[1] = {0.f}, ry = 0.f;
    float f[V][EPU];  // y, then x_out
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = grp.sub + i * a.tpr;
#pragma unroll
      for (int m = 0; m < EPU; ++m) f[i][m] = 0.f;
      if (a.y && live && c < a.packs) {
        SB::read(tb + sb + ofs_y + i * SB::kPlanes * plb, plb, f[i]);
#pragma unroll
        for (int m = 0; m < EPU; ++m) s[0] = fmaf(f[i][m], f[i][m], s[0]);
      }
    }
    if (a.y) {
      grp.sum(s, red);
      ry = rsqrtf(s[0] * a.inv_dim + a.eps);
    }
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = grp.sub + i * a.tpr;
      if (!live || c >= a.packs) continue;
      float x[EPU], z[EPU];
      SX::read(tx + sb + i * SX::kPlanes * plx, plx, x);
      if (a.y) {
        const int w = cw.use(a, i, c * EPU);
        if (a.gate_cols > 1) SB::read(tb + sb + ofs_g + i * SB::kPlanes * plb, plb, z);
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          float g = g_row;
          if (a.gate_cols > 1) sigmoid2(z[m], g, rest);
          x[m] = fmaf(cw.rw[w][m] * g, f[i][m] * ry, x[m]);
        }
        Pack<XT, EPU> o;
        o.set(x);
        o.store(static_cast<XT*>(a.x_out) + row * a.x_out_ld + (int64_t)c * EPU);
      }
#pragma unroll
      for (int m = 0; m < EPU; ++m) {
        f[i][m] = x[m];
        s[0] = fmaf(x[m], x[m], s[0]);
      }
    }
    if (a.h) {
      grp.sum(s, red + 16);
      const float rx = rsqrtf(s[0] * a.inv_dim + a.eps);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = grp.sub + i * a.tpr;
        if (!live || c >= a.packs) continue;
        const int w = cw.use(a, i, c * EPU);
        float o[EPU];
#pragma unroll
        for (int m = 0; m < EPU; ++m) o[m] = f[i][m] * rx * cw.wq[w][m];
        Pack<BT, EPU> p;
        p.set(o);
        p.store(static_cast<BT*>(a.h) + row * a.h_ld + (int64_t)c * EPU);
      }
    }
    // a call with one sum a row leaves no second barrier between its uses of `red`
    if ((!a.y || !a.h) && a.tpr > 32)
      asm volatile("bar.sync %0, %1;" ::"r"(grp.id + 1), "r"(a.tpr) : "memory");
    st = st + 1 == a.stages ? 0 : st + 1;
  }
}

template <typename XT, typename BT, int EPU, int V>
__global__ void __launch_bounds__(kNormMaxThreads) k_gated_norm_bwd(NormArgs a) {
  using SX = Slot<XT, EPU>;
  using SB = Slot<BT, EPU>;
  extern __shared__ __align__(16) char ring[];
  __shared__ float red_all[4 * 16 * 16];
  const uint32_t plx = blockDim.x * SX::UB, plb = blockDim.x * SB::UB;
  const RowGroup grp{a.tpr, (int)threadIdx.x / a.tpr, (int)threadIdx.x % a.tpr};
  float* red = red_all + (a.tpr > 32 ? grp.id : 0) * 4 * 16;
  const uint32_t stage_bytes = blockDim.x * kRingBytes<XT, BT, EPU, V, 2, 3>;
  const uint32_t ring0 = smem_at(ring);
  const uint32_t ofs_dx = V * SX::kPlanes * plx, ofs_dh = 2 * ofs_dx;
  const uint32_t ofs_y = ofs_dh + V * SB::kPlanes * plb, ofs_g = ofs_y + V * SB::kPlanes * plb;
  const uint32_t tx = ring0 + threadIdx.x * SX::UB, tb = ring0 + threadIdx.x * SB::UB;
  const int64_t step = (int64_t)gridDim.x * a.rpb;
  ColWeights<EPU, V> cw;
  cw.init(a, grp.sub);
  float col_pre[V][EPU], col_t[V][EPU];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int m = 0; m < EPU; ++m) col_pre[i][m] = col_t[i][m] = 0.f;

  auto fetch = [&](int64_t row, int stage) {
    if (row < a.n) {
      const uint32_t sb = stage * stage_bytes;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = grp.sub + i * a.tpr;
        if (c < a.packs) {
          const int64_t at = (int64_t)c * EPU;
          const uint32_t ix = tx + sb + i * SX::kPlanes * plx, ib = tb + sb + i * SB::kPlanes * plb;
          SX::fetch(ix, plx, static_cast<const XT*>(a.x_out) + row * a.x_out_ld + at);
          if (a.dx_out) SX::fetch(ix + ofs_dx, plx, static_cast<const XT*>(a.dx_out) + row * a.dx_out_ld + at);
          if (a.dh) SB::fetch(ib + ofs_dh, plb, static_cast<const BT*>(a.dh) + row * a.dh_ld + at);
          if (a.y) SB::fetch(ib + ofs_y, plb, static_cast<const BT*>(a.y) + row * a.y_ld + at);
          if (a.gate_cols > 1) SB::fetch(ib + ofs_g, plb, static_cast<const BT*>(a.gate) + row * a.gate_ld + at);
        }
      }
    }
    ring_commit();
  };
  int64_t row = (int64_t)blockIdx.x * a.rpb + grp.id;
  for (int s = 0; s < a.stages - 1; ++s) fetch(row + s * step, s);
  int st = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * a.rpb; r0 < a.n; r0 += step, row += step) {
    const bool live = row < a.n;
    fetch(row + (a.stages - 1) * step, st == 0 ? a.stages - 1 : st - 1);
    float g_row = 1.f, rest_row = 0.f;
    if (a.gate_cols == 1 && live) {
      Pack<BT, 1> p;
      float z[1];
      p.load(static_cast<const BT*>(a.gate) + row * a.gate_ld);
      p.get(z);
      sigmoid2(z[0], g_row, rest_row);
    }
    ring_wait(a.stages);
    const uint32_t sb = st * stage_bytes;
    float s[3] = {0.f, 0.f, 0.f};  // x_out^2, dh w_pre x_out, y^2
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = grp.sub + i * a.tpr;
      if (!live || c >= a.packs) continue;
      const uint32_t ix = tx + sb + i * SX::kPlanes * plx, ib = tb + sb + i * SB::kPlanes * plb;
      float x[EPU], d[EPU];
      SX::read(ix, plx, x);
#pragma unroll
      for (int m = 0; m < EPU; ++m) s[0] = fmaf(x[m], x[m], s[0]);
      if (a.dh) {
        const int w = cw.use(a, i, c * EPU);
        SB::read(ib + ofs_dh, plb, d);
#pragma unroll
        for (int m = 0; m < EPU; ++m) s[1] = fmaf(d[m] * cw.wq[w][m], x[m], s[1]);
      }
      if (a.y) {
        SB::read(ib + ofs_y, plb, d);
#pragma unroll
        for (int m = 0; m < EPU; ++m) s[2] = fmaf(d[m], d[m], s[2]);
      }
    }
    grp.sum(s, red);
    const float rx = rsqrtf(s[0] * a.inv_dim + a.eps), ry = rsqrtf(s[2] * a.inv_dim + a.eps);
    const float xm = rx * rx * (rx * s[1] * a.inv_dim);  // x_out * xm = q mean(dh w_pre q) / rms
    float su[1] = {0.f};
    float u[V][EPU];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = grp.sub + i * a.tpr;
      if (!live || c >= a.packs) continue;
      const int64_t at = (int64_t)c * EPU;
      const uint32_t ix = tx + sb + i * SX::kPlanes * plx, ib = tb + sb + i * SB::kPlanes * plb;
      const int w = cw.use(a, i, c * EPU);
      float t[EPU];
#pragma unroll
      for (int m = 0; m < EPU; ++m) t[m] = 0.f;
      if (a.dx_out) SX::read(ix + ofs_dx, plx, t);
      if (a.dh) {
        float x[EPU], d[EPU];
        SX::read(ix, plx, x);
        SB::read(ib + ofs_dh, plb, d);
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          const float dr = d[m] * rx;
          t[m] += dr * cw.wq[w][m] - x[m] * xm;
          col_pre[i][m] = fmaf(dr, x[m], col_pre[i][m]);
        }
      }
      if (a.dx) {
        Pack<XT, EPU> o;
        o.set(t);
        o.store(static_cast<XT*>(a.dx) + row * a.dx_ld + at);
      }
      if (a.y) {
        float y[EPU], z[EPU];
        SB::read(ib + ofs_y, plb, y);
        if (a.gate_cols > 1) SB::read(ib + ofs_g, plb, z);
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          float g = g_row, rest = 0.f;
          if (a.gate_cols > 1) sigmoid2(z[m], g, rest);
          const float yn = y[m] * ry, tg = t[m] * g;
          col_t[i][m] = fmaf(tg, yn, col_t[i][m]);
          u[i][m] = tg * cw.rw[w][m];
          const float uy = u[i][m] * yn;
          su[0] += uy;
          z[m] = uy * rest;
        }
        if (a.gate_cols > 1 && a.dgate) {
          Pack<BT, EPU> o;
          o.set(z);
          o.store(static_cast<BT*>(a.dgate) + row * a.dgate_ld + at);
        }
      }
    }
    if (a.y) {
      grp.sum(su, red + 3 * 16);
      // one gate a row: sum of t res_scale w_post a g, times 1 - g
      if (a.gate_cols == 1 && a.dgate && live && grp.sub == 0) {
        Pack<BT, 1> p;
        const float z[1] = {su[0] * rest_row};
        p.set(z);
        p.store(static_cast<BT*>(a.dgate) + row * a.dgate_ld);
      }
      const float um = ry * su[0] * a.inv_dim;
      if (a.dy)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = grp.sub + i * a.tpr;
          if (!live || c >= a.packs) continue;
          float y[EPU];
          SB::read(tb + sb + i * SB::kPlanes * plb + ofs_y, plb, y);
#pragma unroll
          for (int m = 0; m < EPU; ++m) y[m] = ry * (u[i][m] - y[m] * um);
          Pack<BT, EPU> o;
          o.set(y);
          o.store(static_cast<BT*>(a.dy) + row * a.dy_ld + (int64_t)c * EPU);
        }
    } else if (a.tpr > 32) {  // one sum a row: no second barrier between its uses of `red`
      asm volatile("bar.sync %0, %1;" ::"r"(grp.id + 1), "r"(a.tpr) : "memory");
    }
    st = st + 1 == a.stages ? 0 : st + 1;
  }
  ring_wait_n<0>();
  // the CTA's column sums: its groups are added one after another in shared memory
  float* cols = reinterpret_cast<float*>(ring);  // [2][dim], when a CTA has more than one group
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.dim;
  for (int r = 0; r < a.rpb; ++r) {
    if (a.rpb > 1) __syncthreads();
    if (grp.id != r) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = grp.sub + i * a.tpr;
      if (c >= a.packs) continue;
#pragma unroll
      for (int m = 0; m < EPU; ++m) {
        const int k = c * EPU + m;
        float p = col_pre[i][m], q = col_t[i][m];
        if (r > 0) p += cols[k], q += cols[a.dim + k];
        if (r < a.rpb - 1) cols[k] = p, cols[a.dim + k] = q;
        else out[k] = p, out[a.dim + k] = q;
      }
    }
  }
}

// Sums the CTAs' parts: 32 columns a CTA, 32 threads a column over interleaved parts, then over
// the 32 in order.
__global__ void __launch_bounds__(1024) k_gated_norm_cols(const float* part, int parts, int dim,
                                                          const float* w_post, const float* res_scale,
                                                          float* dw_post, float* dres_scale,
                                                          float* dw_pre) {
  __shared__ float sh[2][32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, k = blockIdx.x * 32 + lane;
  float p = 0.f, t = 0.f;
  if (k < dim) {
#pragma unroll 4
    for (int g = slice; g < parts; g += 32) {
      p += part[(int64_t)g * 2 * dim + k];
      t += part[(int64_t)g * 2 * dim + dim + k];
    }
  }
  sh[0][slice][lane] = p;
  sh[1][slice][lane] = t;
  __syncthreads();
  // warp c (of 32) sums column c: lane = slice
  const int col = blockIdx.x * 32 + slice;
  p = lanes_sum(sh[0][lane][slice], 32);
  t = lanes_sum(sh[1][lane][slice], 32);
  if (lane == 0 && col < dim) {
    if (dw_pre) dw_pre[col] = p;
    if (dw_post) dw_post[col] = (res_scale ? res_scale[col] : 1.f) * t;
    if (dres_scale) dres_scale[col] = (w_post ? w_post[col] : 1.f) * t;
  }
}

// ---- host ----

// Threads of a row: about eight elements each, a power of two up to a warp, whole warps above.
static void norm_shape(NormArgs& a, int epu) {
  a.packs = a.dim / epu;
  const int want = (a.dim + 7) / 8;
  int t = 4;
  while (t < want && t < 32) t *= 2;
  if (want > 32) t = (want + 31) / 32 * 32;
  a.tpr = t < kNormMaxThreads ? t : kNormMaxThreads;
  a.rpb = a.tpr >= kNormThreads ? 1 : kNormThreads / a.tpr;
}

// Ring stages that fit, and their bytes: up to kStages within a CTA's shared memory.
static int norm_ring(NormArgs& a, int thread_bytes) {
  const int per = a.rpb * a.tpr * thread_bytes, most = 220 * 1024;
  a.stages = kStages;
  while (a.stages > 1 && a.stages * per > most) --a.stages;
  return a.stages * per;
}

// CTAs of `kern` on the device at once.
template <typename K>
static int norm_ctas(K kern, int threads, int smem, cudaError_t* e) {
  int per = 0;
  *e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (*e == cudaSuccess)
    *e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, threads, smem);
  return (per < 1 ? 1 : per) * device_sms();
}

static NormArgs norm_args(const emb_norm& p) {
  NormArgs a{};
  a.n = p.n, a.dim = p.dim, a.gate_cols = p.d_gate ? p.gate_cols : 0;
  a.eps = p.eps, a.inv_dim = 1.f / (float)p.dim;
  a.x = p.d_x, a.y = p.d_y, a.gate = p.d_gate, a.dx_out = p.d_dx_out, a.dh = p.d_dh;
  a.x_out = p.d_x_out, a.h = p.d_h, a.dx = p.d_dx, a.dy = p.d_dy, a.dgate = p.d_dgate;
  a.x_ld = p.x_ld, a.y_ld = p.y_ld, a.gate_ld = p.gate_ld, a.dx_out_ld = p.dx_out_ld;
  a.dh_ld = p.dh_ld, a.x_out_ld = p.x_out_ld, a.h_ld = p.h_ld, a.dx_ld = p.dx_ld;
  a.dy_ld = p.dy_ld, a.dgate_ld = p.dgate_ld;
  a.w_post = p.d_w_post, a.res_scale = p.d_res_scale, a.w_pre = p.d_w_pre;
  return a;
}

// Whether every matrix of the call (NULL: none) allows packs of 16 bytes.
static bool norm_vec(const emb_norm& p) {
  const int xe = p.x_dtype == EMB_BF16 ? 2 : 4, be = p.dtype == EMB_BF16 ? 2 : 4;
  const int epu = be == 2 ? 8 : 4;
  return p.dim % epu == 0 && rows16(p.d_x, p.x_ld, xe) && rows16(p.d_y, p.y_ld, be) &&
         (p.gate_cols == 1 || rows16(p.d_gate, p.gate_ld, be)) && rows16(p.d_x_out, p.x_out_ld, xe) &&
         rows16(p.d_h, p.h_ld, be) && rows16(p.d_dx_out, p.dx_out_ld, xe) &&
         rows16(p.d_dh, p.dh_ld, be) && rows16(p.d_dx, p.dx_ld, xe) && rows16(p.d_dy, p.dy_ld, be) &&
         (p.gate_cols == 1 || rows16(p.d_dgate, p.dgate_ld, be)) && rows16(p.d_w_post, 0, 4) &&
         rows16(p.d_res_scale, 0, 4) && rows16(p.d_w_pre, 0, 4);
}

template <typename XT, typename BT, int EPU, int V>
static cudaError_t norm_fwd_v(NormArgs& a, cudaStream_t s) {
  const int smem = norm_ring(a, kRingBytes<XT, BT, EPU, V, 1, 2>), threads = a.rpb * a.tpr;
  cudaError_t e;
  const int64_t blocks = (a.n + a.rpb - 1) / a.rpb;
  const int64_t cap = norm_ctas(k_gated_norm<XT, BT, EPU, V>, threads, smem, &e);
  if (e != cudaSuccess) return e;
  k_gated_norm<XT, BT, EPU, V><<<(int)(blocks < cap ? blocks : cap), threads, smem, s>>>(a);
  return cudaGetLastError();
}

// CTAs of the backward: no more than `cap`, and at least four rows a group where that is fewer,
// so that the column parts stay small beside the rows.
static int64_t norm_bwd_grid(int64_t n, int rpb, int64_t cap) {
  const int64_t blocks = (n + 4 * rpb - 1) / (4 * rpb);
  return blocks < 1 ? 1 : blocks < cap ? blocks : cap;
}

constexpr int kNormCtasPerSm = 4;  // CTAs of the backward per SM, at most

int64_t gated_norm_bwd_workspace(int64_t n, int dim) {
  NormArgs a{};
  a.dim = dim;
  norm_shape(a, 1);
  return norm_bwd_grid(n, a.rpb, (int64_t)device_sms() * kNormCtasPerSm) * 2 * dim * (int64_t)sizeof(float);
}

template <typename XT, typename BT, int EPU, int V>
static cudaError_t norm_bwd_v(NormArgs& a, int* grid, cudaStream_t s) {
  int smem = norm_ring(a, kRingBytes<XT, BT, EPU, V, 2, 3>);
  const int threads = a.rpb * a.tpr, cols = a.rpb > 1 ? 2 * a.dim * (int)sizeof(float) : 0;
  if (smem < cols) smem = cols;
  cudaError_t e;
  int64_t cap = norm_ctas(k_gated_norm_bwd<XT, BT, EPU, V>, threads, smem, &e);
  if (e != cudaSuccess) return e;
  if (cap > (int64_t)device_sms() * kNormCtasPerSm) cap = (int64_t)device_sms() * kNormCtasPerSm;
  *grid = (int)norm_bwd_grid(a.n, a.rpb, cap);
  k_gated_norm_bwd<XT, BT, EPU, V><<<*grid, threads, smem, s>>>(a);
  return cudaGetLastError();
}

// The kernel of a call by packs per thread (1, 2, 4, 8 or 16: at most 16 elements).
template <typename XT, typename BT, int EPU, bool BWD, int V = 1>
static cudaError_t norm_t(NormArgs& a, int* grid, cudaStream_t s) {
  if constexpr (V == 1) norm_shape(a, EPU);
  if constexpr (V * EPU < 16)
    if ((a.packs + a.tpr - 1) / a.tpr > V) return norm_t<XT, BT, EPU, BWD, 2 * V>(a, grid, s);
  if constexpr (BWD) return norm_bwd_v<XT, BT, EPU, V>(a, grid, s);
  else return norm_fwd_v<XT, BT, EPU, V>(a, s);
}

template <bool BWD>
static cudaError_t norm_call(const emb_norm& p, NormArgs& a, int* grid, cudaStream_t s) {
  const bool vec = norm_vec(p);
  using H = __nv_bfloat16;
  if (p.dtype == EMB_F32)
    return vec ? norm_t<float, float, 4, BWD>(a, grid, s) : norm_t<float, float, 1, BWD>(a, grid, s);
  if (p.x_dtype == EMB_F32)
    return vec ? norm_t<float, H, 8, BWD>(a, grid, s) : norm_t<float, H, 1, BWD>(a, grid, s);
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
  if (e == cudaSuccess && (p.d_dw_post || p.d_dres_scale || p.d_dw_pre)) {
    k_gated_norm_cols<<<(p.dim + 31) / 32, 1024, 0, s>>>(a.part, grid, p.dim, p.d_w_post,
                                                         p.d_res_scale, p.d_dw_post, p.d_dres_scale,
                                                         p.d_dw_pre);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace emb
