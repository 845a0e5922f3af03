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

// What the products of the small parts add to that of the large ones, for fp32 operands.  An infinite or NaN element
// stands in its large part alone, and the large parts' product is then what the definition gives (a large part is zero
// only with its element); the small ones' is not, infinity times a part of zero is NaN: it is left out.
__device__ __forceinline__ float with_small(float large, float small) {
  return fabsf(large) <= 3.4028235e38f ? large + small : large;
}

// v = a + b + c once more, with parts of v's own sign of which none is zero unless v is: a is the bf16 below v in
// magnitude, b the one below v - a, c what is left (eight bits at most, or one).  So an infinite factor times the
// parts gives infinities of one sign, as it does times v.  Without c the parts are at most 2^-14 of v short of it.
__device__ __forceinline__ void split3_below(float v, float& a, float& b, float& c) {
  const auto below = [](float x) {
    const uint32_t u = __float_as_uint(x), m = u & 0x7FFFFFFFu;
    return __uint_as_float(m ? (u & 0x80000000u) | ((m - 1) & 0xFFFF0000u) : u);
  };
  a = b = c = v;
  if (!(fabsf(v) <= 3.4028235e38f)) return;
  a = below(v);
  const float r = v - a;
  b = below(r);
  c = r - b;
}

// ---- activations ----

// s(v) = 1 / (1 + exp(-v)): for fp32 results with CUDA's full exponential and quotient, for bf16 with the
// hardware's approximate power of two and reciprocal (their error, 2^-22 and |v| 2^-24 of the value, is far inside
// bf16's 2^-9 wherever the value is not zero to bf16 anyway).  Where exp(-v) overflows s is zero.
template <bool FULL>
__device__ __forceinline__ float sigmoid_of(float v) {
  if (FULL) return 1.f / (1.f + expf(-v));
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.44269504f * v));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// act(v), and in `slope` its derivative where wanted.  silu v s(v); gelu v P(v) with the normal
// distribution P(v) = erfc(-v / sqrt 2) / 2; relu; sigmoid s(v).  Finite v gives finite results; an infinite one
// NaN where the formula has infinity times zero.
template <int ACT, bool FULL, bool SLOPE>
__device__ __forceinline__ float activate(float v, float& slope) {
  if (ACT == EMB_ACT_RELU) {
    if (SLOPE) slope = v > 0.f ? 1.f : 0.f;
    return v < 0.f ? 0.f : v;
  }
  if (ACT == EMB_ACT_GELU) {
    const float p = 0.5f * erfcf(-0.70710678f * v);
    if (SLOPE) slope = fmaf(0.39894228f * v, FULL ? expf(-0.5f * v * v) : __expf(-0.5f * v * v), p);
    return v * p;
  }
  const float s = sigmoid_of<FULL>(v);
  // 1 - s(v) = s(-v), which is not lost where s is near one
  const float rest = SLOPE ? sigmoid_of<FULL>(-v) : 0.f;
  if (ACT == EMB_ACT_SIGMOID) {
    if (SLOPE) slope = s * rest;
    return s;
  }
  if (SLOPE) slope = fmaf(v * s, rest, s);
  return v * s;
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
constexpr int kMaxPacks = 3;
cudaError_t launch_expert_packs(const PackArgs* args, int count, cudaStream_t s);  // all fp32, or all bf16
// [dg, du] of a gated block's backward, to rows of 2 * p.out
// (planes: three, or two for bf16 rows and results)
cudaError_t launch_expert_gated_bwd(const emb_product& p, const MmOperand& to, bool beside, cudaStream_t s);

struct MmArgs {
  MmOperand a, b;
  bool b_mn = false;             // rows product: b's rows run along the contraction
  const int32_t* offsets = nullptr;
  int E = 1;
  int S = 0;
  int M = 0, N = 0, K = 0;       // rows product: N columns, K; weight gradient: M x N
  bool turned = false;           // weight gradient: out is N x M
  int act = -1;                  // rows product: gated (N: columns of a half), or -1
  bool f32 = false;
  void* out = nullptr;
  int64_t out_ld = 0, out_step = 0;
  bool out_bf16 = false;
  void* gu = nullptr;
  int64_t gu_ld = 0;
  int tile_n = 256;              // weight gradient: columns of a tile, 256 or 128
  int split = 0;                 // weight gradient: rows of a part (a multiple of 64), 0: no parts
  float* parts = nullptr;        // as out, one after the other
  // launched right after a kernel of the same call, one that lets the next start only when it has passed its own
  // wait, and needs nothing of it: the two run side by side
  bool beside = false;
};
// A rows product where experts have few rows, from the matrices as they lie.
struct FewArgs {
  const int32_t* offsets = nullptr;
  int E = 1, S = 0, in = 0, out = 0, act = -1;  // out: of a half where gated
  bool f32 = false, turned = false;             // turned: w's rows run along the outputs
  const void *x = nullptr, *w = nullptr;
  int64_t x_ld = 0, w_ld = 0, w_step = 0, half = 0;
  void *y = nullptr, *gu = nullptr;
  int64_t y_ld = 0, gu_ld = 0;
};
cudaError_t launch_expert_few(const FewArgs& a, cudaStream_t s);
int64_t mm_pairs();
cudaError_t launch_expert_mm_rows(const MmArgs& a, cudaStream_t s);
cudaError_t launch_expert_mm_wgrad(const MmArgs& a, cudaStream_t s);

}  // namespace emb
