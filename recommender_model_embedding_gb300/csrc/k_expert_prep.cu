// What the experts' products need beside the tensor cores' work: operands on 16-byte boundaries, fp32
// operands as three bf16 planes, and the gradient of a gated block's halves.
//
// fp32 -> three bf16: v0 = v rounded, v1 = (v - v0) rounded, v2 = (v - v0 - v1) rounded.  Both
// differences are exact in fp32 and each remainder has eight significant bits less, so v0 + v1 + v2 = v
// wherever the last one is not below bf16's range.  A value that would round beyond bf16's largest is cut
// instead, and infinities and NaN stand in v0 alone.
//
// Gated block: from h = act(g) u, dg = dh u act'(g) and du = dh act(g), side by side as the product's
// operand, rounded to bf16 as the tensor cores take them (fp32: three planes).  Both kernels are bound by
// HBM bandwidth.
#include <algorithm>

#include "expert_mm.cuh"

namespace emb {

namespace {

constexpr int kPrepThreads = 256;

// elements [0, EPU) of a row's piece; places from `valid` on are zero
template <typename T, int EPU>
__device__ __forceinline__ void load_piece(const T* p, int valid, bool vec, float (&v)[EPU]) {
  if constexpr (EPU == 8) {
    if (vec && valid >= 8) {
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
  }
#pragma unroll
  for (int i = 0; i < EPU; ++i) {
    v[i] = 0.f;
    if (i < valid) {
      Pack<T, 1> a;
      a.load(p + i);
      float x[1];
      a.get(x);
      v[i] = x[0];
    }
  }
}

template <int PLANES, int EPU>
__device__ __forceinline__ void store_piece(__nv_bfloat16* to, int64_t plane, const float (&v)[EPU]) {
  if constexpr (PLANES == 1) {
    Pack<__nv_bfloat16, EPU> o;
    o.set(v);
    o.store(to);
  } else {
    float a[EPU], b[EPU], c[EPU];
#pragma unroll
    for (int i = 0; i < EPU; ++i) split3(v[i], a[i], b[i], c[i]);
    Pack<__nv_bfloat16, EPU> o;
    o.set(a);
    o.store(to);
    o.set(b);
    o.store(to + plane);
    o.set(c);
    o.store(to + 2 * plane);
  }
}

template <typename T, int PLANES>
__global__ void __launch_bounds__(kPrepThreads)
    k_expert_pack(const T* src, int64_t ld, int64_t half_step, int64_t expert_step, int vec, const int32_t* last,
                  FastDiv rows, FastDiv halves, uint32_t all, int inner, int shift, __nv_bfloat16* to, int64_t to_ld,
                  int64_t to_half, int64_t to_expert, int64_t to_plane) {
  wait_for_earlier();
  let_next_start();
  const uint32_t per = kPrepThreads >> shift;
  const uint32_t most = last ? (uint32_t)min(max(*last, 0), (int)all) : all;
  const int units = (inner + 7) / 8, sub = threadIdx.x & ((1 << shift) - 1);
  for (uint32_t i = blockIdx.x * per + (threadIdx.x >> shift); i < most; i += gridDim.x * per) {
    const uint32_t m = rows.div(i), r = i - m * rows.d, e = halves.div(m), h = m - e * halves.d;
    const T* from = src + (int64_t)r * ld + (int64_t)h * half_step + (int64_t)e * expert_step;
    __nv_bfloat16* out = to + (int64_t)r * to_ld + (int64_t)h * to_half + (int64_t)e * to_expert;
    for (int u = sub; u < units; u += 1 << shift) {
      float v[8];
      load_piece<T, 8>(from + u * 8, inner - u * 8, vec, v);
      store_piece<PLANES, 8>(out + u * 8, to_plane, v);
    }
  }
}

template <typename T, int PLANES, int ACT, int EPU>
__global__ void __launch_bounds__(kPrepThreads)
    k_expert_gated_bwd(const T* dh, int64_t dh_ld, const T* gu, int64_t gu_ld, const int32_t* last, uint32_t S, int f,
                       int shift, __nv_bfloat16* to, int64_t to_ld, int64_t to_plane) {
  constexpr bool F32 = PLANES == 3;  // what is to be of fp32's exactness
  wait_for_earlier();
  let_next_start();
  const uint32_t per = kPrepThreads >> shift;
  const uint32_t most = last ? (uint32_t)min(max(*last, 0), (int)S) : S;
  const int units = f / EPU, sub = threadIdx.x & ((1 << shift) - 1);
  for (uint32_t r = blockIdx.x * per + (threadIdx.x >> shift); r < most; r += gridDim.x * per) {
    const T *d = dh + (int64_t)r * dh_ld, *g = gu + (int64_t)r * gu_ld;
    __nv_bfloat16* out = to + (int64_t)r * to_ld;
    for (int c = sub; c < units; c += 1 << shift) {
      float dv[EPU], gv[EPU], uv[EPU];
      load_piece<T, EPU>(d + c * EPU, EPU, true, dv);
      load_piece<T, EPU>(g + c * EPU, EPU, true, gv);
      load_piece<T, EPU>(g + f + c * EPU, EPU, true, uv);
#pragma unroll
      for (int i = 0; i < EPU; ++i) {
        float slope;
        const float a = activate<ACT, F32, true>(gv[i], slope);
        gv[i] = dv[i] * uv[i] * slope;
        uv[i] = dv[i] * a;
      }
      store_piece<PLANES, EPU>(out + c * EPU, to_plane, gv);
      store_piece<PLANES, EPU>(out + f + c * EPU, to_plane, uv);
    }
  }
}

// threads of a row: a power of two, as many as it has pieces, up to a CTA's
int row_shift(int64_t units) {
  int shift = 0;
  while (shift < 8 && (1 << shift) < units) ++shift;
  return shift;
}

unsigned row_grid(int64_t rows, int shift) {
  const int64_t per = kPrepThreads >> shift;
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, (int64_t)device_sms() * 16));
}

}  // namespace

cudaError_t launch_expert_pack(const PackArgs& a, cudaStream_t s) {
  const int64_t all = a.to.rows * a.to.halves * a.to.experts;
  if (all == 0) return cudaSuccess;
  const int shift = row_shift((a.to.inner + 7) / 8), elem = a.f32 ? 4 : 2;
  const int vec = rows_on(a.src, a.ld, elem, 16) && a.half_step * elem % 16 == 0 && a.expert_step * elem % 16 == 0;
  const auto run = [&](auto kern, auto* src) {
    return launch_early(kern, row_grid(all, shift), kPrepThreads, 0, s, src, a.ld, a.half_step, a.expert_step, vec, a.last,
                        FastDiv((uint32_t)a.to.rows), FastDiv((uint32_t)a.to.halves), (uint32_t)all, (int)a.to.inner, shift,
                        const_cast<__nv_bfloat16*>(a.to.p), a.to.ld, a.to.half_step, a.to.expert_step, a.to.plane_step);
  };
  return a.f32 ? run(k_expert_pack<float, 3>, static_cast<const float*>(a.src))
               : run(k_expert_pack<__nv_bfloat16, 1>, static_cast<const __nv_bfloat16*>(a.src));
}

cudaError_t launch_expert_gated_bwd(const emb_product& p, const MmOperand& to, cudaStream_t s) {
  if (p.rows == 0) return cudaSuccess;
  const int elem = p.dtype == EMB_BF16 ? 2 : 4;
  const bool vec = p.out % 8 == 0 && rows16(p.d_dout, p.dout_ld, elem) && rows16(p.d_gu, p.gu_ld, elem);
  const int shift = row_shift(vec ? p.out / 8 : p.out);
  const int32_t* last = p.d_offsets ? p.d_offsets + p.experts : nullptr;
  const auto run = [&](auto kern, auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    return launch_early(kern, row_grid(p.rows, shift), kPrepThreads, 0, s, static_cast<const T*>(p.d_dout), p.dout_ld,
                        static_cast<const T*>(p.d_gu), p.gu_ld, last, (uint32_t)p.rows, (int)p.out, shift,
                        const_cast<__nv_bfloat16*>(to.p), to.ld, to.plane_step);
  };
  const auto by_act = [&](auto act) {
    constexpr int A = decltype(act)::value;
    using H = __nv_bfloat16;
    H* h = nullptr;
    float* f = nullptr;
    if (p.dtype == EMB_F32) return vec ? run(k_expert_gated_bwd<float, 3, A, 8>, f) : run(k_expert_gated_bwd<float, 3, A, 1>, f);
    if (to.planes == 3) return vec ? run(k_expert_gated_bwd<H, 3, A, 8>, h) : run(k_expert_gated_bwd<H, 3, A, 1>, h);
    return vec ? run(k_expert_gated_bwd<H, 1, A, 8>, h) : run(k_expert_gated_bwd<H, 1, A, 1>, h);
  };
  switch (p.act) {
    case EMB_ACT_SILU: return by_act(std::integral_constant<int, EMB_ACT_SILU>());
    case EMB_ACT_GELU: return by_act(std::integral_constant<int, EMB_ACT_GELU>());
    case EMB_ACT_RELU: return by_act(std::integral_constant<int, EMB_ACT_RELU>());
    default: return by_act(std::integral_constant<int, EMB_ACT_SIGMOID>());
  }
}

}  // namespace emb
