// Gated norm, backward: the kernel, the sum of its column parts and their launches (formulas and
// design: gated_norm.cuh).
#include "gated_norm.cuh"

namespace emb {

template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
__global__ void __launch_bounds__(V * EPU > 8 ? kNormWide : kAheadBackward<EPU, V> ? kNormThreads : kNormBackward, V * EPU > 8 ? 1 : 2) k_gated_norm_bwd(NormArgs a) {
  let_next_start();
  wait_for_earlier();
  using K = Chunks<EPU, V>;
  using LX = Lane<XT, EPU, V, WARP, kAheadBackward<EPU, V>>;
  using LB = Lane<BT, EPU, V, WARP, kAheadBackward<EPU, V>>;
  extern __shared__ __align__(16) char ring[];
  __shared__ __align__(16) float red_all[8 * 4 * 16];
  for (int i = threadIdx.x; i < 8 * 4 * 16; i += blockDim.x) red_all[i] = 0.f;
  const RowGroup grp{a.tpr, (int)threadIdx.x / a.tpr, (int)threadIdx.x % a.tpr};
  float* red = red_all + (a.tpr > 32 ? grp.id : 0) * 4 * 16;
  const Share<V, WARP> sh(grp.sub, a.tpr);
  const int left = a.packs - sh.first, tpr = a.tpr;
  const uint32_t plx = blockDim.x * LX::S::kBytes, plb = blockDim.x * LB::S::kBytes;
  const uint32_t stage_bytes =
      kAheadBackward<EPU, V> ? 0 : blockDim.x * kRingBytes<XT, BT, EPU, V, 2, GATE ? 3 : 2>;
  const uint32_t mx = V * plx, mb = V * plb;  // of a matrix
  const uint32_t tx = smem_at(ring) + threadIdx.x * LX::S::kBytes;
  const uint32_t tb = smem_at(ring) + threadIdx.x * LB::S::kBytes + 2 * mx;
  LX lx(tx, plx), lt(tx + mx, plx);
  LB ld(tb, plb), ly(tb + mb, plb), lg(tb + 2 * mb, plb);
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
  RowGate<BT> row_gate;
  if (!GATE) row_gate.fetch(a, row);
  ColWeights<EPU, V, WARP> cw;
  cw.init(a, sh, reinterpret_cast<float*>(ring + a.stages * stage_bytes));
  for (int s = 0; s < a.stages; ++s) {
    lx.zero_tail(s * stage_bytes, left, sh);
    lt.zero_tail(s * stage_bytes, left, sh);
    ld.zero_tail(s * stage_bytes, left, sh);
    ly.zero_tail(s * stage_bytes, left, sh);
    if (GATE) lg.zero_tail(s * stage_bytes, left, sh);
  }
  __syncthreads();  // red_all is cleared, shared weights are there
  uint32_t st = 0;
  for (uint32_t r0 = blockIdx.x * a.rpb; r0 < a.n; r0 += step, row += step) {
    const bool live = row < a.n;
    if constexpr (kAheadBackward<EPU, V>) lx.advance(), lt.advance(), ld.advance(), ly.advance(), lg.advance();
    fetch(row + (a.stages - 1) * step, st == 0 ? last : st - stage_bytes);
    float g_row = 1.f, rest_row = 0.f;
    if (!GATE) row_gate.take(a, row + step, g_row, rest_row);
    ring_wait(a.stages);
    float sx[2] = {0.f, 0.f}, sd[2] = {0.f, 0.f}, sy[2] = {0.f, 0.f};
    if (live)
#pragma unroll
      for (int i = 0; i < K::NC; ++i) {
        float x[K::C], d[K::C];
        lx.read(st, i, x);
        v_dot(sx, x, x);
        if (a.dh) {
          cw.use_wq(a, sh, i);
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
    // x_out * xm = -q mean(dh w_pre q) / rms.  1 / rms^2 is held to what fp32 has: for a row of zeros and
    // an eps below 2^-127 it meets a sum of zero (the sum first, and no bound: 65536 x 2048 bf16
    // without a gate 412 us, 395 so)
    constexpr float kMost = 3.4028235e38f;
    const float xm = -fminf(rx * rx, kMost) * (rx * s[1] * a.inv_dim);
    float su2[2] = {0.f, 0.f}, su[1];
    float u[K::NC][K::C];
    if (live)
#pragma unroll
      for (int i = 0; i < K::NC; ++i) {
        float t[K::C];
        if (a.dx_out) lt.read(st, i, t);
        else
#pragma unroll
          for (int m = 0; m < K::C; ++m) t[m] = 0.f;
        if (a.dh) {
          float x[K::C], d[K::C];
          cw.use_wq(a, sh, i);
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
            float z[K::C], g[K::C];
            lg.read(st, i, z);
            v_sigmoid(z, g, rest);
            v_mul(t, t, g);
          } else {
            v_mul(t, t, g_row);
          }
          v_fma(col_t[i], t, y, col_t[i]);
          cw.use_rw(a, sh, i);
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
      const float um = -fminf(ry * ry, kMost) * su[0] * a.inv_dim;
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
  if (!a.cols) return;
  // the CTA's column sums: a warp's groups by shuffles, then the slices (warps, or groups of whole
  // warps) side by side in shared memory
  const int slices = tpr < 32 ? (int)blockDim.x / 32 : a.rpb;
  const int slice = tpr < 32 ? (int)threadIdx.x / 32 : grp.id;
  const bool writes = tpr >= 32 || (int)(threadIdx.x & 31) < tpr;
  float* cols = reinterpret_cast<float*>(ring);  // [slices][2][dim]
  __syncthreads();                               // the ring has been read
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
        cols[slice * 2 * a.dim + k] = p, cols[(slice * 2 + 1) * a.dim + k] = q;
      }
    }
  }
  __syncthreads();
  // where they go: the workspace, or the results, if there is one CTA
  float* out = a.part + (int64_t)blockIdx.x * 2 * a.dim;
  for (int k = threadIdx.x; k < a.dim; k += blockDim.x) {
    float p = cols[k], q = cols[a.dim + k];
    for (int r = 1; r < slices; ++r) p += cols[r * 2 * a.dim + k], q += cols[(r * 2 + 1) * a.dim + k];
    if (gridDim.x == 1) put_cols(a, k, p, q);
    else out[k] = p, out[a.dim + k] = q;
  }
}

// Sums the CTAs' parts (none: zeros): 32 columns a CTA, 32 threads a column over interleaved parts, then over
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

// CTAs: a row a group up to one CTA an SM, then at least four rows a group up to `cap`, so that the
// column parts stay small beside the rows.  (A cluster of 16 CTAs that added its parts itself, in
// one launch, gained little on few rows, 16 x 1024 6.3 us against 6.7, and lost on more, 96 x 1024
// 9.7 against 7.3.)
constexpr int kNormCtasPerSm = 2 * kNormBackward / 160;  // at most (a CTA has at least 160 threads)

static int64_t norm_bwd_grid(int64_t n, int rpb, int64_t cap) {
  const int64_t sms = device_sms(), all = (n + rpb - 1) / rpb, four = (n + 4 * rpb - 1) / (4 * rpb);
  const int64_t blocks = all <= sms ? all : four > sms ? four : sms;
  return blocks < 1 ? 1 : blocks < cap ? blocks : cap;
}

int64_t gated_norm_bwd_workspace(int64_t n, int dim) {
  NormArgs a{};
  a.dim = dim;
  norm_shape(a, 1, kNormBackward);
  return norm_bwd_grid(n, a.rpb, (int64_t)device_sms() * kNormCtasPerSm) * 2 * dim * (int64_t)sizeof(float);
}

template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
static cudaError_t norm_bwd_v(NormArgs& a, int* parts, cudaStream_t s) {
  const int threads = a.rpb * a.tpr, per = (V * EPU > 8 ? kNormWide : kAheadBackward<EPU, V> ? 2 * kNormThreads : 2 * kNormBackward) / threads;
  int smem = norm_ring(a, kAheadBackward<EPU, V> ? 0 : kRingBytes<XT, BT, EPU, V, 2, GATE ? 3 : 2>, per, V * EPU > 8 ? a.tpr * 128 : 0);
  const int slices = a.tpr < 32 ? threads / 32 : a.rpb;
  const int cols = slices * 2 * a.dim * (int)sizeof(float);
  if (smem < cols) smem = cols;
  constexpr auto kern = k_gated_norm_bwd<XT, BT, EPU, V, GATE, WARP>;
  const cudaError_t e = prepare_kernel<kern>();
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)norm_bwd_grid(a.n, a.rpb, (int64_t)device_sms() * norm_fit(per, smem));
  if (a.cols && grid > 1) *parts = (int)grid;
  return launch_early(kern, grid, threads, smem, s, a);
}

struct NormBackward {
  static constexpr int most(int epu) { return epu <= 2 ? kNormThreads : kNormBackward; }
  cudaStream_t s;
  int* parts;  // CTAs whose column sums are in the workspace (0: none to add)
  template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
  cudaError_t run(NormArgs& a) const { return norm_bwd_v<XT, BT, EPU, V, GATE, WARP>(a, parts, s); }
};

cudaError_t launch_gated_norm_bwd(const emb_norm& p, void* ws, cudaStream_t s) {
  NormArgs a = norm_args(p);
  a.part = static_cast<float*>(ws);
  a.cols = p.d_dw_post || p.d_dres_scale || p.d_dw_pre;
  int parts = 0;
  if (p.n > 0) {
    const cudaError_t e = norm_call(p, a, NormBackward{s, &parts});
    if (e != cudaSuccess || parts == 0) return e;
  } else if (!a.cols) {
    return cudaSuccess;
  } else {
    a.w_post = a.res_scale = nullptr;  // a sum over no rows is zero, whatever the vectors hold
  }
  return launch_early(k_gated_norm_cols, (p.dim + 31) / 32, 1024, 0, s, a, parts);
}

}  // namespace emb
