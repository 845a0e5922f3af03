// Shared by the experts' products: the rows of each expert, activations and their slopes, and the
// launchers' interfaces.
#pragma once

#include <cuda.h>

#include "rows_common.cuh"

namespace emb {

constexpr int kMaxExperts = EMB_EXPERT_MAX;

// The first row of each expert, cuts[0..E], by one warp: the offsets held to [0, S] and to an
// ascending order (so whatever they hold, the experts' rows lie inside the matrix and apart).
// Without offsets all rows are the one expert's.
__device__ __forceinline__ void expert_cuts(const int32_t* offsets, int E, int S, int32_t* cuts, int lane) {
  int32_t before = 0;
  for (int b = 0; b <= E; b += 32) {
    const int e = b + lane;
    int32_t c = S;
    if (offsets != nullptr && e <= E) c = min(max(offsets[e], 0), S);
    if (offsets == nullptr && e == 0) c = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c = max(c, v);
    }
    c = max(c, before);
    before = __shfl_sync(0xFFFFFFFFu, c, 31);
    if (e <= E) cuts[e] = c;
  }
  __syncwarp();
}

// prefix[0..E]: sums of count(rows of the expert) before each, by one warp.
template <typename F>
__device__ __forceinline__ void expert_prefix(const int32_t* cuts, int E, int32_t* prefix, int lane, F count) {
  int32_t total = 0;
  for (int b = 0; b < E; b += 32) {
    const int e = b + lane;
    int32_t c = e < E ? count(cuts[e + 1] - cuts[e]) : 0;
    const int32_t mine = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c += v;
    }
    if (e < E) prefix[e] = total + c - mine;
    total += __shfl_sync(0xFFFFFFFFu, c, 31);
  }
  if (lane == 0) prefix[E] = total;
  __syncwarp();
}

// v = a + b + c, each exact in bf16 once c is rounded there: the differences are exact in fp32 and each
// remainder has eight significant bits less.  A value that would round beyond bf16's largest is cut instead,
// and infinities and NaN stand in a alone.
__device__ __forceinline__ void split3(float v, float& a, float& b, float& c) {
  a = __bfloat162float(__float2bfloat16_rn(v));
  b = c = 0.f;
  if (!(fabsf(v) <= 3.4028235e38f)) return;
  if (fabsf(a) > 3.4e38f) a = __bfloat162float(__float2bfloat16_rz(v));
  const float r = v - a;
  b = __bfloat162float(__float2bfloat16_rn(r));
  c = r - b;  // (rounded where it is stored)
}

// ---- activations ----

// Exponential and quotient: CUDA's full ones for fp32 results, the fast ones for bf16 (their error,
// below 2^-17 where the result is not lost anyway, is far inside bf16's 2^-9).
template <bool FULL>
__device__ __forceinline__ float sigmoid_of(float v) {
  return FULL ? 1.f / (1.f + expf(-v)) : __fdividef(1.f, 1.f + fminf(__expf(-v), 1e37f));
}

// act(v), and in `slope` its derivative where wanted.  silu v s(v); gelu v P(v) with the normal
// distribution P(v) = erfc(-v / sqrt 2) / 2; relu; sigmoid s(v) = 1 / (1 + exp(-v)).  Far out, where
// v times zero or a lost sum would be NaN, the limits hold (NaN stays NaN).
template <int ACT, bool FULL, bool SLOPE>
__device__ __forceinline__ float activate(float v, float& slope) {
  if (ACT == EMB_ACT_RELU) {
    if (SLOPE) slope = v > 0.f ? 1.f : 0.f;
    return v < 0.f ? 0.f : v;
  }
  if (ACT == EMB_ACT_GELU) {
    const float p = 0.5f * erfcf(-0.70710678f * v);
    // (exp(-v v / 2) is zero beyond 14; there v may be infinite)
    if (SLOPE) slope = p + (fabsf(v) < 14.5f ? 0.39894228f * v * (FULL ? expf(-0.5f * v * v) : __expf(-0.5f * v * v)) : 0.f);
    return v < -14.5f ? 0.f : v * p;
  }
  const float s = sigmoid_of<FULL>(v);
  if (ACT == EMB_ACT_SIGMOID) {
    // 1 - s(v) = s(-v), which is not lost where s is near one
    if (SLOPE) slope = s * sigmoid_of<FULL>(-v);
    return s;
  }
  if (SLOPE) {
    const float rest = sigmoid_of<FULL>(-v);
    slope = fabsf(v) < 104.f || v != v ? s + v * s * rest : (v > 0.f ? 1.f : 0.f);
  }
  return v < -104.f ? 0.f : v * s;
}

// ---- operands and launchers ----

// A tensor-core operand in memory: bf16 matrices of `rows` rows of `inner` elements, 16-byte aligned,
// row, half, expert and plane steps in elements (multiples of 8).
struct MmOperand {
  const __nv_bfloat16* p = nullptr;
  int64_t inner = 0, rows = 0, ld = 0, half_step = 0, expert_step = 0, plane_step = 0;
  int halves = 1, experts = 1, planes = 1;
};

// Copy of matrices for the tensor cores: rows [0, rows) of each of `halves` x `experts` matrices.
struct PackArgs {
  const void* src = nullptr;
  int64_t ld = 0, half_step = 0, expert_step = 0;  // of src, in its elements
  int f32 = 0;
  const int32_t* last = nullptr;  // rows from *last on need no copy (NULL: all)
  MmOperand to;
};
cudaError_t launch_expert_pack(const PackArgs& a, cudaStream_t s);
// [dg, du] of a gated block's backward, to rows of 2 * p.out
cudaError_t launch_expert_gated_bwd(const emb_product& p, const MmOperand& to, cudaStream_t s);

struct MmArgs {
  MmOperand a, b;
  bool b_mn = false;             // rows product: b's rows run along the contraction
  const int32_t* offsets = nullptr;
  int E = 1;
  int S = 0;
  int M = 0, N = 0, K = 0;       // rows product: N columns, K; weight gradient: M x N
  int act = -1;                  // rows product: gated (N: columns of a half), or -1
  bool f32 = false;              // operands split in three planes
  void* out = nullptr;
  int64_t out_ld = 0, out_step = 0;
  bool out_bf16 = false;
  void* gu = nullptr;
  int64_t gu_ld = 0;
  int split = 0;                 // weight gradient: rows of a part (a multiple of 64), 0: no parts
  float* parts = nullptr;        // [parts][M][N]
};
cudaError_t launch_expert_mm_rows(const MmArgs& a, cudaStream_t s);
cudaError_t launch_expert_mm_wgrad(const MmArgs& a, cudaStream_t s);

}  // namespace emb
