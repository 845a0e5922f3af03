// The experts' products where an expert has few rows (serving): the linear layer's and the gated block's
// forward, without the tensor memory's tiles.
//
// Bound by reading the weights once, and for a single request by the chain of launch, offsets, loads, sum
// and store.  A tile of the large kernel takes 256 rows through a pipeline that is filled by a few CTAs;
// here a CTA takes 16 outputs (32 where the weights lie turned) of one expert and up to 8, 16 or 32 of its
// rows, so that a small call still spreads over the SMs.  Its eight warps share the contraction, 32 (16) of K a
// step with the loads of several steps ahead of their use, and add up through shared memory in a fixed order;
// where tiles are many, each warp takes one of its own.  The warp's matrix instruction (m16n8k16) takes the weights as
// A and the rows as B; the order of the contraction is free, so a lane's fragments are the eight elements along
// K that one load brings, of an output's weights and of a row alike.  Turned weights come four outputs for
// each of a lane's four k, paired along k by byte permutes.  fp32: three bf16 planes of each and six products, as in
// the large kernel.
//
// Measured, one row for each of two of eight experts, 2 x 1024 x 512 bf16 weights: 2.9 us a call (8.9 through the large
// kernel); 32 rows over eight experts of 512 x 1024: 3.7 us (11.0).  64 experts of 1024 x 512 with a row each, call
// after call: 12.4 us for 67 MB of weights, 5.4 TB/s, much of it from L2, which can hold them.
#include <algorithm>

#include "expert_few.cuh"

namespace emb {

namespace {

struct FewParams {
  const int32_t* offsets;
  int E, S, in, out;         // out: of a half
  const void *x, *w;
  int64_t x_ld, w_ld, w_step, half;
  int x_vec, w_vec;
  int act;
  void *y, *gu;
  int64_t y_ld, gu_ld;
};

// Fragments of a step: A of M tiles of 16 outputs, or B of one of 8 rows; planes, halves of the step, registers
template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;

// Products of a step's fragments; fp32: all planes with i + j <= 2, the small ones' sum apart from the large one, and
// both added in fp32 (the matrix instruction does not round to nearest: summed in it alone 1487 elements were 1.3e-6
// off).
template <int PLANES>
__device__ __forceinline__ void few_mma(float (&c)[4], const uint32_t (&a)[PLANES][4], const uint32_t (&b)[PLANES][2]) {
  if constexpr (PLANES == 3) {
    float d[4] = {}, large[4] = {};
    mma16816(d, a[2], b[0][0], b[0][1]);
    mma16816(d, a[1], b[1][0], b[1][1]);
    mma16816(d, a[0], b[2][0], b[2][1]);
    mma16816(d, a[1], b[0][0], b[0][1]);
    mma16816(d, a[0], b[1][0], b[1][1]);
    mma16816(large, a[0], b[0][0], b[0][1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] += with_small(large[i], d[i]);
  } else {
    mma16816(c, a[0], b[0][0], b[0][1]);
  }
}

template <typename T>
__device__ __forceinline__ void store_one(T* p, float v) {
  const float one[1] = {v};
  Pack<T, 1> o;
  o.set(one);
  o.store(p);
}

template <bool FULL>
__device__ __forceinline__ float act_by(int act, float v) {
  float none;
  switch (act) {
    case EMB_ACT_SILU: return activate<EMB_ACT_SILU, FULL, false>(v, none);
    case EMB_ACT_GELU: return activate<EMB_ACT_GELU, FULL, false>(v, none);
    case EMB_ACT_RELU: return activate<EMB_ACT_RELU, FULL, false>(v, none);
    default: return activate<EMB_ACT_SIGMOID, FULL, false>(v, none);
  }
}

// NT: eights of rows.  share: warps that share a tile's contraction.
template <typename T, bool GATED, int NT, bool TURNED, int share>
__global__ void __launch_bounds__(kFewThreads, 2) k_expert_few(FewParams p) {
  constexpr int H = GATED ? 2 : 1, PL = kPlanes<T>, RT = 8 * NT;
  constexpr int OUTS = TURNED ? 32 : 16, MT = OUTS / 16;  // outputs of a CTA (of each half), in tiles of 16
  constexpr int STEP = TURNED ? 16 : 32, U = PL == 3 ? (NT * H == 1 ? 2 : 1) : NT == 1 ? (TURNED ? 4 : 2) : NT == 2 ? 2 : 1;
  __shared__ float sums[kFewWarps][RT][H * OUTS + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  wait_for_earlier();
  let_next_start();
  int e, r0, rows;
  if (!few_tile(p.offsets, p.E, p.S, RT, blockIdx.y, lane, e, r0, rows)) return;
  constexpr int tiles = kFewWarps / share;  // tiles of outputs of the CTA
  const int o0 = (blockIdx.x * tiles + warp / share) * OUTS, steps = (p.in + STEP - 1) / STEP, first = warp % share;
  const T* w = static_cast<const T*>(p.w) + e * p.w_step;
  const T* x = static_cast<const T*>(p.x) + (int64_t)r0 * p.x_ld;
  float acc[H][MT][NT][4] = {};
  if constexpr (!TURNED) {
    // the lane's two outputs (held inside the matrix: what lies past its end is not stored)
    const T *wa = w + (int64_t)min(o0 + g, p.out - 1) * p.w_ld, *wb = w + (int64_t)min(o0 + g + 8, p.out - 1) * p.w_ld;
    for (int s0 = first; s0 < steps; s0 += share * U) {
      Raw<T, 8> ra[U][H][2], rx[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s0 + u * share) * STEP + t * 8, at = k < p.in ? k : 0;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          ra[u][h][0].load(wa + h * p.half + at, p.in - k, p.w_vec);
          ra[u][h][1].load(wb + h * p.half + at, p.in - k, p.w_vec);
        }
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          const int r = g + 8 * m;
          rx[u][m].load(x + (int64_t)(r < rows ? r : 0) * p.x_ld + at, r < rows ? p.in - k : 0, p.x_vec);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t a[H][2][PL][4], b[NT][2][PL][2];  // [..][half of the step][plane][register]
        if constexpr (PL == 1) {
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) a[h][q >> 1][0][(q & 1) * 2] = ra[u][h][0].w[q], a[h][q >> 1][0][(q & 1) * 2 + 1] = ra[u][h][1].w[q];
#pragma unroll
          for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int q = 0; q < 4; ++q) b[m][q >> 1][0][q & 1] = rx[u][m].w[q];
        } else {
          float v[3][8];
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              planes_of(ra[u][h][i].w, v);
#pragma unroll
              for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                for (int q = 0; q < 4; ++q) a[h][q >> 1][pl][(q & 1) * 2 + i] = pair_bf16(v[pl][2 * q], v[pl][2 * q + 1]);
            }
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            planes_of(rx[u][m].w, v);
#pragma unroll
            for (int pl = 0; pl < PL; ++pl)
#pragma unroll
              for (int q = 0; q < 4; ++q) b[m][q >> 1][pl][q & 1] = pair_bf16(v[pl][2 * q], v[pl][2 * q + 1]);
          }
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) few_mma<PL>(acc[h][0][m], a[h][i], b[m][i]);
      }
    }
  } else {
    // rows of the matrix run along the outputs: the lane's four, o0 + 4 g.., become rows g and g + 8 of two tiles
    const int o = o0 + 4 * g, ov = p.out - o;
    for (int s0 = first; s0 < steps; s0 += share * U) {
      Raw<T, 4> ra[U][H][4], rx[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s0 + u * share) * STEP + t * 4;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool there = k + i < p.in;
            ra[u][h][i].load(w + h * p.half + (int64_t)(there ? k + i : 0) * p.w_ld + (ov > 0 ? o : 0), there ? ov : 0, p.w_vec);
          }
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          const int r = g + 8 * m;
          rx[u][m].load(x + (int64_t)(r < rows ? r : 0) * p.x_ld + (k < p.in ? k : 0), r < rows ? p.in - k : 0, p.x_vec);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t a[H][MT][PL][4], b[NT][PL][2];
        if constexpr (PL == 1) {
#pragma unroll
          for (int h = 0; h < H; ++h)
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {  // k pairs; rows g and g + 8: outputs 2 j and 2 j + 1 of the four
                a[h][j][0][2 * i] = __byte_perm(ra[u][h][2 * i].w[j], ra[u][h][2 * i + 1].w[j], 0x5410);
                a[h][j][0][2 * i + 1] = __byte_perm(ra[u][h][2 * i].w[j], ra[u][h][2 * i + 1].w[j], 0x7632);
              }
#pragma unroll
          for (int m = 0; m < NT; ++m) b[m][0][0] = rx[u][m].w[0], b[m][0][1] = rx[u][m].w[1];
        } else {
          float v[4][3][4];
#pragma unroll
          for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) planes_of(ra[u][h][i].w, v[i]);
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
              for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  a[h][j][pl][q] = pair_bf16(v[(q >> 1) * 2][pl][2 * j + (q & 1)], v[(q >> 1) * 2 + 1][pl][2 * j + (q & 1)]);
          }
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            planes_of(rx[u][m].w, v[0]);
#pragma unroll
            for (int pl = 0; pl < PL; ++pl)
#pragma unroll
              for (int q = 0; q < 2; ++q) b[m][pl][q] = pair_bf16(v[0][pl][2 * q], v[0][pl][2 * q + 1]);
          }
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int m = 0; m < NT; ++m) few_mma<PL>(acc[h][j][m], a[h][j], b[m]);
      }
    }
  }
  // accumulator: outputs of rows g (registers 0, 1) and g + 8 (2, 3), rows 2 t and 2 t + 1 of x
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          sums[warp][8 * m + 2 * t + (q & 1)][h * OUTS + (TURNED ? 4 * g + 2 * j + (q >> 1) : g + 8 * (q >> 1))] = acc[h][j][m][q];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * tiles * OUTS; i += kFewThreads) {
    const int o = i % OUTS, q = i / OUTS % tiles, r = i / (OUTS * tiles), col = (blockIdx.x * tiles + q) * OUTS + o;
    if (col >= p.out) continue;
    float v[H] = {};
#pragma unroll
    for (int k = 0; k < share; ++k)
#pragma unroll
      for (int h = 0; h < H; ++h) v[h] += sums[q * share + k][r][h * OUTS + o];
    T* y = static_cast<T*>(p.y) + (int64_t)(r0 + r) * p.y_ld + col;
    if constexpr (GATED) {
      if (p.gu != nullptr) {
        T* gu = static_cast<T*>(p.gu) + (int64_t)(r0 + r) * p.gu_ld + col;
        store_one(gu, v[0]);
        store_one(gu + p.out, v[1]);
      }
      store_one(y, act_by<PL == 3>(p.act, v[0]) * v[1]);
    } else {
      store_one(y, v[0]);
    }
  }
}

template <typename T, bool GATED, int NT>
cudaError_t run_few(const FewParams& p, bool turned, cudaStream_t s) {
  // (a gated block's two halves are the sums and registers of twice the outputs: 32 rows of them in bf16 as the
  // weights usually lie, else 16)
  if constexpr (GATED && NT == 4)
    if (turned || sizeof(T) == 4) return run_few<T, GATED, 2>(p, turned, s);
  const int outs = turned ? 32 : 16, down = (int)few_tiles(p.S, p.E, 8 * NT), across = (p.out + outs - 1) / outs;
  const int share = few_share((int64_t)down * across), tiles = kFewWarps / share;
  const auto run = [&](auto kern) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((across + tiles - 1) / tiles), (unsigned)down);
    cfg.blockDim = dim3(kFewThreads), cfg.stream = s, cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
  };
  if constexpr (!(GATED && NT == 4))
    if (turned) return share == kFewWarps ? run(k_expert_few<T, GATED, NT, true, kFewWarps>) : run(k_expert_few<T, GATED, NT, true, kFewAlone>);
  if constexpr (!(GATED && NT == 4 && sizeof(T) == 4))
    return share == kFewWarps ? run(k_expert_few<T, GATED, NT, false, kFewWarps>) : run(k_expert_few<T, GATED, NT, false, kFewAlone>);
  return cudaErrorInvalidValue;
}

template <typename T, bool GATED>
cudaError_t few_rows(const FewParams& p, bool turned, cudaStream_t s) {
  const int each = (p.S + p.E - 1) / p.E;  // rows of an expert, on average
  return each <= 8 ? run_few<T, GATED, 1>(p, turned, s) : each <= 16 ? run_few<T, GATED, 2>(p, turned, s) : run_few<T, GATED, 4>(p, turned, s);
}

}  // namespace

cudaError_t launch_expert_few(const FewArgs& a, cudaStream_t s) {
  if (a.S == 0) return cudaSuccess;
  const int elem = a.f32 ? 4 : 2, each = a.turned ? 4 : 8;
  FewParams p{a.offsets, a.E, a.S, a.in, a.out, a.x, a.w, a.x_ld, a.w_ld, a.w_step, a.half, 0, 0, a.act, a.y, a.gu, a.y_ld, a.gu_ld};
  const int bytes = std::min(16, elem * each);
  p.x_vec = rows_on(a.x, a.x_ld, elem, bytes);
  p.w_vec = rows_on(a.w, a.w_ld, elem, bytes) && a.w_step * elem % bytes == 0 && a.half * elem % bytes == 0;
  using H = __nv_bfloat16;
  if (a.act >= 0) return a.f32 ? few_rows<float, true>(p, a.turned, s) : few_rows<H, true>(p, a.turned, s);
  return a.f32 ? few_rows<float, false>(p, a.turned, s) : few_rows<H, false>(p, a.turned, s);
}

}  // namespace emb
