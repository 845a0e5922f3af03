// Gated norm, forward: the kernel and its launch (formulas and design: gated_norm.cuh).
#include "gated_norm.cuh"

namespace emb {

// GATE: a gate for each element.
template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
__global__ void __launch_bounds__(V * EPU > 8 ? kNormWide : kNormForward, V * EPU > 8 || kAheadForward<EPU, V> ? 1 : 2) k_gated_norm(NormArgs a) {
  let_next_start();
  wait_for_earlier();
  using K = Chunks<EPU, V>;
  using LX = Lane<XT, EPU, V, WARP, kAheadForward<EPU, V>>;
  using LB = Lane<BT, EPU, V, WARP, kAheadForward<EPU, V>>;
  extern __shared__ __align__(16) char ring[];
  __shared__ __align__(16) float red_all[8 * 2 * 16];
  for (int i = threadIdx.x; i < 8 * 2 * 16; i += blockDim.x) red_all[i] = 0.f;
  const RowGroup grp{a.tpr, (int)threadIdx.x / a.tpr, (int)threadIdx.x % a.tpr};
  float* red = red_all + (a.tpr > 32 ? grp.id : 0) * 2 * 16;
  const Share<V, WARP> sh(grp.sub, a.tpr);
  const int left = a.packs - sh.first, tpr = a.tpr;
  const uint32_t plx = blockDim.x * LX::S::kBytes, plb = blockDim.x * LB::S::kBytes;
  const uint32_t stage_bytes =
      kAheadForward<EPU, V> ? 0 : blockDim.x * kRingBytes<XT, BT, EPU, V, 1, GATE ? 2 : 1>;
  const uint32_t tx = smem_at(ring) + threadIdx.x * LX::S::kBytes;
  const uint32_t tb = smem_at(ring) + threadIdx.x * LB::S::kBytes + V * plx;
  LX lx(tx, plx);
  LB ly(tb, plb), lg(tb + V * plb, plb);
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
  RowGate<BT> row_gate;
  if (!GATE) row_gate.fetch(a, row);
  ColWeights<EPU, V, WARP> cw;
  cw.init(a, sh, reinterpret_cast<float*>(ring + a.stages * stage_bytes));
  for (int s = 0; s < a.stages; ++s) {
    lx.zero_tail(s * stage_bytes, left, sh);
    ly.zero_tail(s * stage_bytes, left, sh);
    if (GATE) lg.zero_tail(s * stage_bytes, left, sh);
  }
  __syncthreads();  // red_all is cleared, shared weights are there
  uint32_t st = 0;
  // every group runs as many rounds as the CTA's first: shuffles and barriers stay whole
  for (uint32_t r0 = blockIdx.x * a.rpb; r0 < a.n; r0 += step, row += step) {
    const bool live = row < a.n;
    if constexpr (kAheadForward<EPU, V>) lx.advance(), ly.advance(), lg.advance();
    fetch(row + (a.stages - 1) * step, st == 0 ? last : st - stage_bytes);
    float g_row = 1.f, rest;
    if (!GATE) row_gate.take(a, row + step, g_row, rest);
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
          cw.use_rw(a, sh, i);
          v_mul(f[i], f[i], ry);
          if (GATE) {
            float z[K::C], others[K::C];
            lg.read(st, i, z);
            v_sigmoid(z, g, others);
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
          cw.use_wq(a, sh, i);
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
static cudaError_t norm_fwd_v(NormArgs& a, cudaStream_t s) {
  const int threads = a.rpb * a.tpr, per = (V * EPU > 8 || kAheadForward<EPU, V> ? 1 : 2) * kNormForward / threads;
  const int smem = norm_ring(a, kAheadForward<EPU, V> ? 0 : kRingBytes<XT, BT, EPU, V, 1, GATE ? 2 : 1>, per, V * EPU > 8 ? a.tpr * 128 : 0);
  constexpr auto kern = k_gated_norm<XT, BT, EPU, V, GATE, WARP>;
  const int64_t blocks = ((int64_t)a.n + a.rpb - 1) / a.rpb, cap = (int64_t)device_sms() * norm_fit(per, smem);
  const cudaError_t e = prepare_kernel<kern>();
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)(blocks < cap ? blocks : cap), threads, smem, s, a);
}

struct NormForward {
  static constexpr int most(int) { return kNormForward; }
  cudaStream_t s;
  template <typename XT, typename BT, int EPU, int V, bool GATE, bool WARP>
  cudaError_t run(NormArgs& a) const { return norm_fwd_v<XT, BT, EPU, V, GATE, WARP>(a, s); }
};

cudaError_t launch_gated_norm(const emb_norm& p, cudaStream_t s) {
  if (p.n == 0) return cudaSuccess;
  NormArgs a = norm_args(p);
  return norm_call(p, a, NormForward{s});
}

}  // namespace emb
