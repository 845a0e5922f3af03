// What the experts' products need beside the tensor cores' work: operands on 16-byte boundaries, fp32
// operands as three bf16 planes, and the gradient of a gated block's halves.
//
// fp32 -> three bf16: v0 = v rounded, v1 = (v - v0) rounded, v2 = (v - v0 - v1) rounded.  Both
// differences are exact in fp32 and each remainder has eight significant bits less, so v0 + v1 + v2 = v
// wherever the last one is not below bf16's range.  A value that would round beyond bf16's largest is cut
// instead, and infinities and NaN stand in v0 alone.
//
// Gated block: from h = act(g) u, dg = dh u act'(g) and du = dh act(g), side by side as the product's
// operand, in planes too: rounded to bf16 they would put dx 1.7e-3 off in the 2-norm beside its own rounding, which
// is as much, and an fp32 dw 2.6e-3.  fp32 rows, and an fp32 dw of bf16 rows, take three planes, bf16 results two
// (2^-14 of each element is left out, their own rounding is up to 2^-8).  Both kernels are bound by HBM bandwidth:
// 524288 x 1024 in bf16 to three planes 9.7 GB in 1.50 ms (6.4 TB/s, 95% of the measured copy rate); the planes of
// 8198 x 479 rows and 12 x 1280 x 479 weights in fp32 113 MB in 24 us (4.7 TB/s, in L2 for the most part).
#include <algorithm>

#include "expert_mm.cuh"

namespace emb {

namespace {

constexpr int kPrepThreads = 256;

// Eight elements of a row, zero from `valid` on, of a matrix that lies in [lo, hi): in whole 16-byte words where the
// row is not on their boundary too (those that hold the elements, shifted into place), one by one at the matrix's
// ends.
template <typename T>
__device__ __forceinline__ void load_any8(const T* p, int valid, uintptr_t lo, uintptr_t hi, float (&v)[8]) {
  constexpr int N = 8 * sizeof(T) / 4, C = N / 4 + 1;  // words of the elements, 16-byte words that hold them
  const uintptr_t at = reinterpret_cast<uintptr_t>(p), from = at & ~(uintptr_t)15;
  const uint32_t s = (uint32_t)(at - from);
  uint32_t w[N];
  if (valid >= 8 && from >= lo && from + 16 * (s ? C : C - 1) <= hi) {
    uint32_t q[4 * C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (c < C - 1 || s) u = reinterpret_cast<const uint4*>(from)[c];
      q[4 * c] = u.x, q[4 * c + 1] = u.y, q[4 * c + 2] = u.z, q[4 * c + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < 4 * C - 1; ++i) q[i] = s & 4 ? q[i + 1] : q[i];
#pragma unroll
    for (int i = 0; i < 4 * C - 3; ++i) q[i] = s & 8 ? q[i + 2] : q[i];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = sizeof(T) == 2 ? __funnelshift_r(q[i], q[i + 1], (s & 2) * 8) : q[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = i < valid ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
      } else {
        const uint32_t a = 2 * i < valid ? reinterpret_cast<const uint16_t*>(p)[2 * i] : 0u;
        const uint32_t b = 2 * i + 1 < valid ? reinterpret_cast<const uint16_t*>(p)[2 * i + 1] : 0u;
        w[i] = a | b << 16;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = sizeof(T) == 4 ? __uint_as_float(w[i]) : __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

// EPU elements on their boundary
template <typename T, int EPU>
__device__ __forceinline__ void load_piece(const T* p, float (&v)[EPU]) {
  if constexpr (EPU == 8 && sizeof(T) == 4) {
    Pack<T, 4> a, b;
    a.load(p);
    b.load(p + 4);
    float x[4], y[4];
    a.get(x);
    b.get(y);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i], v[4 + i] = y[i];
  } else {
    Pack<T, EPU> a;
    a.load(p);
    a.get(v);
  }
}

// BELOW: parts of one sign, for products with a single plane
template <int PLANES, bool BELOW, int EPU>
__device__ __forceinline__ void store_piece(__nv_bfloat16* to, int64_t plane, const float (&v)[EPU]) {
  if constexpr (PLANES == 1) {
    Pack<__nv_bfloat16, EPU> o;
    o.set(v);
    o.store(to);
  } else {
    float a[EPU], b[EPU], c[EPU];
#pragma unroll
    for (int i = 0; i < EPU; ++i)
      if (BELOW) split3_below(v[i], a[i], b[i], c[i]);
      else split3(v[i], a[i], b[i], c[i]);
    Pack<__nv_bfloat16, EPU> o;
    o.set(a);
    o.store(to);
    o.set(b);
    o.store(to + plane);
    if (PLANES == 2) return;
    o.set(c);
    o.store(to + 2 * plane);
  }
}

// The matrices to copy, in one launch: blocks [first, next one's first) are a job's.
struct PackJob {
  const void* src;
  int64_t ld, half_step, expert_step;
  const int32_t* last;
  FastDiv rows{1}, halves{1};
  uint32_t all, first, blocks;
  int inner, shift;
  __nv_bfloat16* to;
  int64_t to_ld, to_half, to_expert, to_plane;
};
struct PackJobs {
  PackJob job[kMaxPacks];
  int count;
};

template <typename T, int PLANES>
__global__ void __launch_bounds__(kPrepThreads) k_expert_pack(const __grid_constant__ PackJobs jobs) {
  wait_for_earlier();
  let_next_start();
  int j = 0;
  while (j + 1 < jobs.count && blockIdx.x >= jobs.job[j + 1].first) ++j;
  const PackJob& a = jobs.job[j];
  const int shift = a.shift;
  const uint32_t per = kPrepThreads >> shift;
  const uint32_t most = a.last ? (uint32_t)min(max(*a.last, 0), (int)a.all) : a.all;
  const int units = (a.inner + 7) / 8, sub = threadIdx.x & ((1 << shift) - 1);
  const int64_t bytes = ((int64_t)(a.rows.d - 1) * a.ld + a.inner) * (int64_t)sizeof(T);
  for (uint32_t i = (blockIdx.x - a.first) * per + (threadIdx.x >> shift); i < most; i += a.blocks * per) {
    const uint32_t m = a.rows.div(i), r = i - m * a.rows.d, e = a.halves.div(m), h = m - e * a.halves.d;
    const T* from = static_cast<const T*>(a.src) + (int64_t)h * a.half_step + (int64_t)e * a.expert_step;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(from), hi = lo + bytes;
    from += (int64_t)r * a.ld;
    __nv_bfloat16* out = a.to + (int64_t)r * a.to_ld + (int64_t)h * a.to_half + (int64_t)e * a.to_expert;
    for (int u = sub; u < units; u += 1 << shift) {
      float v[8];
      load_any8<T>(from + u * 8, a.inner - u * 8, lo, hi, v);
      store_piece<PLANES, false, 8>(out + u * 8, a.to_plane, v);
    }
  }
}

// EPU columns of each half at a time: eight, or where rows or halves are not on 16-byte boundaries one (neighbouring
// lanes, neighbouring columns: pieces of eight of the shifted result cost more, 773 against some 390 us for 175347 x
// 471 gelu in bf16, for each column's activation comes twice).
template <typename T, int PLANES, int ACT, int EPU>
__global__ void __launch_bounds__(kPrepThreads)
    k_expert_gated_bwd(const T* dh, int64_t dh_ld, const T* gu, int64_t gu_ld, const int32_t* last, uint32_t S, int f,
                       int shift, __nv_bfloat16* to, int64_t to_ld, int64_t to_plane, int beside) {
  constexpr bool F32 = PLANES == 3, BELOW = sizeof(T) == 2;  // F32: what is to be of fp32's exactness
  if (!beside) wait_for_earlier();
  let_next_start();
  const uint32_t per = kPrepThreads >> shift;
  const uint32_t most = last ? (uint32_t)min(max(*last, 0), (int)S) : S;
  const int units = f / EPU, sub = threadIdx.x & ((1 << shift) - 1);
  for (uint32_t r = blockIdx.x * per + (threadIdx.x >> shift); r < most; r += gridDim.x * per) {
    const T *d = dh + (int64_t)r * dh_ld, *g = gu + (int64_t)r * gu_ld;
    __nv_bfloat16* out = to + (int64_t)r * to_ld;
    for (int c = sub; c < units; c += 1 << shift) {
      float dv[EPU], gv[EPU], uv[EPU];
      load_piece<T, EPU>(d + c * EPU, dv);
      load_piece<T, EPU>(g + c * EPU, gv);
      load_piece<T, EPU>(g + f + c * EPU, uv);
#pragma unroll
      for (int i = 0; i < EPU; ++i) {
        float slope;
        const float a = activate<ACT, F32, true>(gv[i], slope);
        gv[i] = dv[i] * uv[i] * slope;
        uv[i] = dv[i] * a;
      }
      store_piece<PLANES, BELOW, EPU>(out + c * EPU, to_plane, gv);
      store_piece<PLANES, BELOW, EPU>(out + f + c * EPU, to_plane, uv);
    }
  }
  if (beside) wait_for_earlier();
}

// threads of a row: a power of two, as many as it has pieces, up to a CTA's
int row_shift(int64_t units) {
  int shift = 0;
  while (shift < 8 && (1 << shift) < units) ++shift;
  return shift;
}

unsigned row_grid(int64_t rows, int shift) {
  const int64_t per = kPrepThreads >> shift;
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, (int64_t)device_sms() * 128));
}

}  // namespace

cudaError_t launch_expert_packs(const PackArgs* args, int count, cudaStream_t s) {
  PackJobs jobs{};
  unsigned blocks = 0;
  for (int i = 0; i < count; ++i) {
    const PackArgs& a = args[i];
    const int64_t all = a.to.rows * a.to.halves * a.to.experts;
    if (all == 0) continue;
    const int shift = row_shift((a.to.inner + 7) / 8);
    const unsigned mine = row_grid(all, shift);
    jobs.job[jobs.count++] = {a.src, a.ld, a.half_step, a.expert_step, a.last, FastDiv((uint32_t)a.to.rows), FastDiv((uint32_t)a.to.halves),
                              (uint32_t)all, blocks, mine, (int)a.to.inner, shift, const_cast<__nv_bfloat16*>(a.to.p), a.to.ld,
                              a.to.half_step, a.to.expert_step, a.to.plane_step};
    blocks += mine;
  }
  if (blocks == 0) return cudaSuccess;
  return args[0].f32 ? launch_early(k_expert_pack<float, 3>, blocks, kPrepThreads, 0, s, jobs)
                     : launch_early(k_expert_pack<__nv_bfloat16, 1>, blocks, kPrepThreads, 0, s, jobs);
}

cudaError_t launch_expert_gated_bwd(const emb_product& p, const MmOperand& to, bool beside, cudaStream_t s) {
  if (p.rows == 0) return cudaSuccess;
  const int elem = p.dtype == EMB_BF16 ? 2 : 4;
  const bool vec = p.out % 8 == 0 && rows16(p.d_dout, p.dout_ld, elem) && rows16(p.d_gu, p.gu_ld, elem);
  const int shift = row_shift(vec ? p.out / 8 : p.out);
  const int32_t* last = p.d_offsets ? p.d_offsets + p.experts : nullptr;
  const auto run = [&](auto kern, auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    return launch_early(kern, row_grid(p.rows, shift), kPrepThreads, 0, s, static_cast<const T*>(p.d_dout), p.dout_ld,
                        static_cast<const T*>(p.d_gu), p.gu_ld, last, (uint32_t)p.rows, (int)p.out, shift,
                        const_cast<__nv_bfloat16*>(to.p), to.ld, to.plane_step, (int)beside);
  };
  const auto by_act = [&](auto act) {
    constexpr int A = decltype(act)::value;
    using H = __nv_bfloat16;
    H* h = nullptr;
    float* f = nullptr;
    if (p.dtype == EMB_F32) return vec ? run(k_expert_gated_bwd<float, 3, A, 8>, f) : run(k_expert_gated_bwd<float, 3, A, 1>, f);
    if (to.planes == 3) return vec ? run(k_expert_gated_bwd<H, 3, A, 8>, h) : run(k_expert_gated_bwd<H, 3, A, 1>, h);
    return vec ? run(k_expert_gated_bwd<H, 2, A, 8>, h) : run(k_expert_gated_bwd<H, 2, A, 1>, h);
  };
  switch (p.act) {
    case EMB_ACT_SILU: return by_act(std::integral_constant<int, EMB_ACT_SILU>());
    case EMB_ACT_GELU: return by_act(std::integral_constant<int, EMB_ACT_GELU>());
    case EMB_ACT_RELU: return by_act(std::integral_constant<int, EMB_ACT_RELU>());
    default: return by_act(std::integral_constant<int, EMB_ACT_SIGMOID>());
  }
}

}  // namespace emb
