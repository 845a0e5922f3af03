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
// Both are bound by HBM bandwidth.  `tpr` threads hold one row in registers as loaded (packs of
// 16 bytes, V of them a thread), so each matrix is read and written once; row sums are
// fp32, by shuffles and, above 32 threads a row, through shared memory.  The backward's CTAs
// are persistent: a thread keeps the same columns for all its rows, so the column sums stay in
// its registers until the end, when they go to the workspace and a second launch adds the
// CTAs' parts in a fixed order.
#include "rows_common.cuh"

namespace emb {

constexpr int kNormThreads = 256;     // of a CTA, unless a row takes more
constexpr int kNormMaxThreads = 512;  // of a row

struct NormArgs {
  int64_t n;
  int dim, packs, tpr;  // packs of EPU elements of a row; threads of a row
  int gate_cols;        // 0, 1 or dim
  float eps, inv_dim;
  const void *x, *y, *gate, *dx_out, *dh;
  void *x_out, *h, *dx, *dy, *dgate;
  int64_t x_ld, y_ld, gate_ld, dx_out_ld, dh_ld, x_out_ld, h_ld, dx_ld, dy_ld, dgate_ld;
  const float *w_post, *res_scale, *w_pre;
  float* part;  // [CTAs][2][dim] column sums (backward)
};

// sigmoid(z) and 1 - sigmoid(z), each to full relative precision at either end
__device__ __forceinline__ void sigmoid2(float z, float& g, float& rest) {
  const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
  g = z >= 0.f ? r : e * r;
  rest = z >= 0.f ? e * r : r;
}

// Sums of NS values over the threads of a row; every thread of the row gets them.  `red` holds
// 32 floats per value.  Called by all threads of the CTA.
template <int NS>
__device__ __forceinline__ void row_sum(float (&v)[NS], int tpr, float (*red)[32]) {
#pragma unroll
  for (int i = 0; i < NS; ++i) v[i] = lanes_sum(v[i], tpr < 32 ? tpr : 32);
  if (tpr > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) red[i][warp] = v[i];
    __syncthreads();
    const int wpr = tpr >> 5, w0 = threadIdx.x / tpr * wpr;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      v[i] = 0.f;
      for (int w = 0; w < wpr; ++w) v[i] += red[i][w0 + w];
    }
  }
}

template <int EPU>
__device__ __forceinline__ void load_cols(const float* w, int col, float (&v)[EPU]) {
#pragma unroll
  for (int m = 0; m < EPU; ++m) v[m] = w ? w[col + m] : 1.f;
}

template <typename XT, typename BT, int EPU, int V>
__global__ void __launch_bounds__(kNormMaxThreads) k_gated_norm(NormArgs a) {
  __shared__ float red[1][32];
  const int rpb = blockDim.x / a.tpr, sub = threadIdx.x % a.tpr;
  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.n; r0 += (int64_t)gridDim.x * rpb) {
    const int64_t row = r0 + threadIdx.x / a.tpr;
    const bool live = row < a.n;
    const XT* x = static_cast<const XT*>(a.x) + row * a.x_ld;
    const BT* y = static_cast<const BT*>(a.y) + row * a.y_ld;
    const BT* gate = static_cast<const BT*>(a.gate) + row * a.gate_ld;
    Pack<XT, EPU> px[V];
    Pack<BT, EPU> py[V], pg[V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * a.tpr;
      px[i].zero(), py[i].zero(), pg[i].zero();
      if (live && c < a.packs) {
        px[i].load(x + (int64_t)c * EPU);
        if (a.y) py[i].load(y + (int64_t)c * EPU);
        if (a.gate_cols > 1) pg[i].load(gate + (int64_t)c * EPU);
      }
    }
    if (a.y) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[EPU];
        py[i].get(f);
#pragma unroll
        for (int m = 0; m < EPU; ++m) s[0] = fmaf(f[m], f[m], s[0]);
      }
      row_sum(s, a.tpr, red);
    }
    const float ry = rsqrtf(s[0] * a.inv_dim + a.eps);
    float g_row = 1.f, rest;
    if (a.gate_cols == 1 && live) {
      Pack<BT, 1> p;
      float z[1];
      p.load(gate);
      p.get(z);
      sigmoid2(z[0], g_row, rest);
    }
    float xo[V][EPU];
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * a.tpr;
      px[i].get(xo[i]);
      if (a.y && live && c < a.packs) {
        float f[EPU], z[EPU], wp[EPU], rs[EPU];
        py[i].get(f);
        pg[i].get(z);
        load_cols<EPU>(a.w_post, c * EPU, wp);
        load_cols<EPU>(a.res_scale, c * EPU, rs);
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          float g = g_row;
          if (a.gate_cols > 1) sigmoid2(z[m], g, rest);
          xo[i][m] = fmaf(rs[m] * g, f[m] * ry * wp[m], xo[i][m]);
        }
        Pack<XT, EPU> o;
        o.set(xo[i]);
        o.store(static_cast<XT*>(a.x_out) + row * a.x_out_ld + (int64_t)c * EPU);
      }
#pragma unroll
      for (int m = 0; m < EPU; ++m) s[0] = fmaf(xo[i][m], xo[i][m], s[0]);
    }
    if (!a.h) continue;
    row_sum(s, a.tpr, red);
    const float rx = rsqrtf(s[0] * a.inv_dim + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * a.tpr;
      if (live && c < a.packs) {
        float w[EPU], f[EPU];
        load_cols<EPU>(a.w_pre, c * EPU, w);
#pragma unroll
        for (int m = 0; m < EPU; ++m) f[m] = xo[i][m] * rx * w[m];
        Pack<BT, EPU> o;
        o.set(f);
        o.store(static_cast<BT*>(a.h) + row * a.h_ld + (int64_t)c * EPU);
      }
    }
  }
}

// HOLD: the row stays in registers between the passes; otherwise (wide rows) each pass loads it
// again, from L1 or L2.
template <typename XT, typename BT, int EPU, int V, bool HOLD>
__global__ void __launch_bounds__(kNormMaxThreads) k_gated_norm_bwd(NormArgs a) {
  __shared__ float red[3][32];
  const int rpb = blockDim.x / a.tpr, sub = threadIdx.x % a.tpr;
  constexpr int VH = HOLD ? V : 1;
  float col_pre[V][EPU], col_t[V][EPU];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int m = 0; m < EPU; ++m) col_pre[i][m] = col_t[i][m] = 0.f;

  for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.n; r0 += (int64_t)gridDim.x * rpb) {
    const int64_t row = r0 + threadIdx.x / a.tpr;
    const bool live = row < a.n;
    Pack<XT, EPU> px[VH], pdx[VH];
    Pack<BT, EPU> py[VH], pg[VH], pdh[VH];
    auto fetch = [&](int i, int h) {  // packs of column step i into registers h
      const int c = sub + i * a.tpr;
      px[h].zero(), pdx[h].zero(), py[h].zero(), pg[h].zero(), pdh[h].zero();
      if (live && c < a.packs) {
        const int64_t at = (int64_t)c * EPU;
        px[h].load(static_cast<const XT*>(a.x_out) + row * a.x_out_ld + at);
        if (a.dx_out) pdx[h].load(static_cast<const XT*>(a.dx_out) + row * a.dx_out_ld + at);
        if (a.dh) pdh[h].load(static_cast<const BT*>(a.dh) + row * a.dh_ld + at);
        if (a.y) py[h].load(static_cast<const BT*>(a.y) + row * a.y_ld + at);
        if (a.gate_cols > 1) pg[h].load(static_cast<const BT*>(a.gate) + row * a.gate_ld + at);
      }
    };
    if (HOLD)
#pragma unroll
      for (int i = 0; i < V; ++i) fetch(i, i);
    float s[3] = {0.f, 0.f, 0.f};  // x_out^2, dh w_pre x_out, y^2
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * a.tpr, h = HOLD ? i : 0;
      if (!HOLD) fetch(i, 0);
      if (c >= a.packs) continue;
      float x[EPU], y[EPU], d[EPU], w[EPU];
      px[h].get(x), py[h].get(y), pdh[h].get(d);
      load_cols<EPU>(a.w_pre, c * EPU, w);
#pragma unroll
      for (int m = 0; m < EPU; ++m) {
        s[0] = fmaf(x[m], x[m], s[0]);
        s[1] = fmaf(d[m] * w[m], x[m], s[1]);
        s[2] = fmaf(y[m], y[m], s[2]);
      }
    }
    row_sum(s, a.tpr, red);
    const float rx = rsqrtf(s[0] * a.inv_dim + a.eps), ry = rsqrtf(s[2] * a.inv_dim + a.eps);
    const float rxm = rx * (rx * s[1] * a.inv_dim);  // mean(dh w_pre q) / rms
    float g_row = 1.f, rest_row = 0.f;
    if (a.gate_cols == 1 && live) {
      Pack<BT, 1> p;
      float z[1];
      p.load(static_cast<const BT*>(a.gate) + row * a.gate_ld);
      p.get(z);
      sigmoid2(z[0], g_row, rest_row);
    }
    // t of a pack, in fp32
    auto grad_t = [&](int h, const float (&x)[EPU], const float (&d)[EPU], const float (&w)[EPU],
                      float (&t)[EPU]) {
      pdx[h].get(t);
      if (a.dh)
#pragma unroll
        for (int m = 0; m < EPU; ++m) t[m] += rx * (d[m] * w[m]) - rxm * (x[m] * rx);
    };
    float u_sum[1] = {0.f};
    if (a.y) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = sub + i * a.tpr, h = HOLD ? i : 0;
        if (!HOLD) fetch(i, 0);
        if (c >= a.packs) continue;
        float x[EPU], y[EPU], d[EPU], z[EPU], w[EPU], wp[EPU], rs[EPU], t[EPU];
        px[h].get(x), py[h].get(y), pdh[h].get(d), pg[h].get(z);
        load_cols<EPU>(a.w_pre, c * EPU, w);
        load_cols<EPU>(a.w_post, c * EPU, wp);
        load_cols<EPU>(a.res_scale, c * EPU, rs);
        grad_t(h, x, d, w, t);
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          float g = g_row, rest;
          if (a.gate_cols > 1) sigmoid2(z[m], g, rest);
          u_sum[0] = fmaf(t[m] * rs[m] * (g * wp[m]), y[m] * ry, u_sum[0]);
        }
      }
      row_sum(u_sum, a.tpr, red);
      // one gate a row: sum of t res_scale w_post a g, times 1 - g
      if (a.gate_cols == 1 && a.dgate && live && sub == 0) {
        Pack<BT, 1> p;
        const float z[1] = {u_sum[0] * rest_row};
        p.set(z);
        p.store(static_cast<BT*>(a.dgate) + row * a.dgate_ld);
      }
    }
    const float um = u_sum[0] * a.inv_dim;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = sub + i * a.tpr, h = HOLD ? i : 0;
      if (!HOLD) fetch(i, 0);
      if (!live || c >= a.packs) continue;
      const int64_t at = (int64_t)c * EPU;
      float x[EPU], y[EPU], d[EPU], z[EPU], w[EPU], wp[EPU], rs[EPU], t[EPU];
      px[h].get(x), py[h].get(y), pdh[h].get(d), pg[h].get(z);
      load_cols<EPU>(a.w_pre, c * EPU, w);
      load_cols<EPU>(a.w_post, c * EPU, wp);
      load_cols<EPU>(a.res_scale, c * EPU, rs);
      grad_t(h, x, d, w, t);
#pragma unroll
      for (int m = 0; m < EPU; ++m) col_pre[i][m] = fmaf(d[m], x[m] * rx, col_pre[i][m]);
      if (a.dx) {
        Pack<XT, EPU> o;
        o.set(t);
        o.store(static_cast<XT*>(a.dx) + row * a.dx_ld + at);
      }
      if (a.y) {
        float dy[EPU], dz[EPU];
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          float g = g_row, rest = 0.f;
          if (a.gate_cols > 1) sigmoid2(z[m], g, rest);
          const float yn = y[m] * ry, tg = t[m] * g, rw = rs[m] * wp[m];
          col_t[i][m] = fmaf(tg, yn, col_t[i][m]);
          dy[m] = ry * (tg * rw - yn * um);
          dz[m] = tg * rw * yn * rest;
        }
        if (a.dy) {
          Pack<BT, EPU> o;
          o.set(dy);
          o.store(static_cast<BT*>(a.dy) + row * a.dy_ld + at);
        }
        if (a.gate_cols > 1 && a.dgate) {
          Pack<BT, EPU> o;
          o.set(dz);
          o.store(static_cast<BT*>(a.dgate) + row * a.dgate_ld + at);
        }
      }
    }
  }
  // the CTA's column sums: its rows side by side are added in shared memory, one after another
  extern __shared__ float cols[];  // [2][dim], when a CTA holds more than one row
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.dim;
  for (int r = 0; r < rpb; ++r) {
    if (threadIdx.x / a.tpr == r) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = sub + i * a.tpr;
        if (c >= a.packs) continue;
#pragma unroll
        for (int m = 0; m < EPU; ++m) {
          const int k = c * EPU + m;
          float p = col_pre[i][m], q = col_t[i][m];
          if (rpb > 1) {
            if (r > 0) p += cols[k], q += cols[a.dim + k];
            if (r < rpb - 1) cols[k] = p, cols[a.dim + k] = q;
          }
          if (r == rpb - 1) out[k] = p, out[a.dim + k] = q;
        }
      }
    }
    if (rpb > 1) __syncthreads();
  }
}

// Sums the CTAs' parts: 32 columns a CTA, 8 threads a column over interleaved parts, then over
// the 8 in order.
__global__ void __launch_bounds__(256) k_gated_norm_cols(const float* part, int parts, int dim,
                                                         const float* w_post, const float* res_scale,
                                                         float* dw_post, float* dres_scale,
                                                         float* dw_pre) {
  __shared__ float sh[2][8][32];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, k = blockIdx.x * 32 + lane;
  float p = 0.f, t = 0.f;
  if (k < dim)
    for (int g = slice; g < parts; g += 8) {
      p += part[(int64_t)g * 2 * dim + k];
      t += part[(int64_t)g * 2 * dim + dim + k];
    }
  sh[0][slice][lane] = p;
  sh[1][slice][lane] = t;
  __syncthreads();
  if (slice == 0 && k < dim) {
    for (int i = 1; i < 8; ++i) p += sh[0][i][lane], t += sh[1][i][lane];
    if (dw_pre) dw_pre[k] = p;
    if (dw_post) dw_post[k] = (res_scale ? res_scale[k] : 1.f) * t;
    if (dres_scale) dres_scale[k] = (w_post ? w_post[k] : 1.f) * t;
  }
}

// ---- host ----

// Threads of a row: a power of two, enough for one pack each up to `most`.
static int norm_tpr(int packs, int most) {
  int t = 4;
  while (t < packs && t < most) t *= 2;
  return t;
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

template <typename XT, typename BT, int EPU>
static cudaError_t norm_fwd_t(NormArgs a, cudaStream_t s) {
  a.packs = a.dim / EPU;
  a.tpr = norm_tpr(a.packs, kNormMaxThreads);
  const int threads = a.tpr > kNormThreads ? a.tpr : kNormThreads;
  const int rpb = threads / a.tpr, V = (a.packs + a.tpr - 1) / a.tpr;
  const int64_t blocks = (a.n + rpb - 1) / rpb, cap = (int64_t)device_sms() * 32;
  const int grid = (int)(blocks < cap ? blocks : cap);
  if (V <= 1) k_gated_norm<XT, BT, EPU, 1><<<grid, threads, 0, s>>>(a);
  else if (V <= 2) k_gated_norm<XT, BT, EPU, 2><<<grid, threads, 0, s>>>(a);
  else if constexpr (EPU < 8) {
    if (V <= 4) k_gated_norm<XT, BT, EPU, 4><<<grid, threads, 0, s>>>(a);
    else if constexpr (EPU == 1) {
      if (V <= 8) k_gated_norm<XT, BT, EPU, 8><<<grid, threads, 0, s>>>(a);
      else k_gated_norm<XT, BT, EPU, 16><<<grid, threads, 0, s>>>(a);
    }
  }
  return cudaGetLastError();
}

cudaError_t launch_gated_norm(const emb_norm& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  const NormArgs a = norm_args(p);
  const bool vec = norm_vec(p);
  if (p.dtype == EMB_F32) return vec ? norm_fwd_t<float, float, 4>(a, s) : norm_fwd_t<float, float, 1>(a, s);
  if (p.x_dtype == EMB_F32)
    return vec ? norm_fwd_t<float, __nv_bfloat16, 8>(a, s) : norm_fwd_t<float, __nv_bfloat16, 1>(a, s);
  return vec ? norm_fwd_t<__nv_bfloat16, __nv_bfloat16, 8>(a, s)
             : norm_fwd_t<__nv_bfloat16, __nv_bfloat16, 1>(a, s);
}

// CTAs of the backward: two per SM, fewer when there are few rows (at least four rows' work a
// CTA, so that the column parts stay small beside the rows).
static int norm_bwd_grid(int64_t n, int rpb) {
  const int64_t blocks = (n + 4 * rpb - 1) / (4 * rpb), cap = (int64_t)device_sms() * 2;
  return (int)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

int64_t gated_norm_bwd_workspace(int64_t n, int dim) {
  return (int64_t)norm_bwd_grid(n, 1) * 2 * dim * (int64_t)sizeof(float);
}

template <typename XT, typename BT, int EPU>
static cudaError_t norm_bwd_t(NormArgs a, int* grid_out, cudaStream_t s) {
  a.packs = a.dim / EPU;
  a.tpr = norm_tpr(a.packs, kNormMaxThreads);
  const int threads = a.tpr > kNormThreads ? a.tpr : kNormThreads;
  const int rpb = threads / a.tpr, V = (a.packs + a.tpr - 1) / a.tpr;
  const int grid = norm_bwd_grid(a.n, rpb);
  const int smem = rpb > 1 ? 2 * a.dim * (int)sizeof(float) : 0;
  *grid_out = grid;
  if (V <= 1) k_gated_norm_bwd<XT, BT, EPU, 1, true><<<grid, threads, smem, s>>>(a);
  else if (V <= 2) k_gated_norm_bwd<XT, BT, EPU, 2, (EPU < 8)><<<grid, threads, smem, s>>>(a);
  else if constexpr (EPU < 8) {
    if (V <= 4) k_gated_norm_bwd<XT, BT, EPU, 4, EPU == 1><<<grid, threads, smem, s>>>(a);
    else if constexpr (EPU == 1) {
      if (V <= 8) k_gated_norm_bwd<XT, BT, EPU, 8, false><<<grid, threads, smem, s>>>(a);
      else k_gated_norm_bwd<XT, BT, EPU, 16, false><<<grid, threads, smem, s>>>(a);
    }
  }
  return cudaGetLastError();
}

cudaError_t launch_gated_norm_bwd(const emb_norm& p, void* ws, cudaStream_t s) {
  NormArgs a = norm_args(p);
  a.part = static_cast<float*>(ws);
  int grid = 0;
  cudaError_t e = cudaSuccess;
  if (p.n > 0) {
    const bool vec = norm_vec(p);
    if (p.dtype == EMB_F32)
      e = vec ? norm_bwd_t<float, float, 4>(a, &grid, s) : norm_bwd_t<float, float, 1>(a, &grid, s);
    else if (p.x_dtype == EMB_F32)
      e = vec ? norm_bwd_t<float, __nv_bfloat16, 8>(a, &grid, s)
              : norm_bwd_t<float, __nv_bfloat16, 1>(a, &grid, s);
    else
      e = vec ? norm_bwd_t<__nv_bfloat16, __nv_bfloat16, 8>(a, &grid, s)
              : norm_bwd_t<__nv_bfloat16, __nv_bfloat16, 1>(a, &grid, s);
  }
  if (e == cudaSuccess && (p.d_dw_post || p.d_dres_scale || p.d_dw_pre)) {
    k_gated_norm_cols<<<(p.dim + 31) / 32, 256, 0, s>>>(a.part, grid, p.dim, p.d_w_post,
                                                        p.d_res_scale, p.d_dw_post, p.d_dres_scale,
                                                        p.d_dw_pre);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace emb
