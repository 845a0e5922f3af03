// Products of few rows with 4-bit weights, rows grouped by expert, and the packing of such weights.
//
//   out[r][o] = sum over groups G of columns: scale[e][o][G] * sum over i in G of (code[e][o][i] - 8) x[r][i]
//
// Bound by reading the codes (half a byte a weight) while an expert has few rows, and there by how many
// instructions a code costs: multiplied by ordinary fp32 arithmetic, a code of one row costs about
// three, over what the memory rate leaves time for.  So the products go through the warp's matrix
// instruction (m16n8k16, bf16 with fp32 sums): codes less eight are exact in bf16, a group's sum is
// formed with codes alone and multiplied by its scale in fp32.  A lane's A fragment is its own codes as
// they come (the order of the contraction is free, so the k of a fragment are what one load
// brings), 1.5 instructions a code; B is eight rows of x.  fp32 rows are three bf16 planes, v = v0 + v1 + v2,
// each with its product, so nothing is lost of them.
//
// A CTA takes 16 outputs of one expert and its (up to 8, 16 or 32) rows; its eight warps share the
// contraction and add up through shared memory in a fixed order.  Where outputs are many, each warp takes 64 (fp32 with
// 32 rows: 32) of its own, for which the rows are brought, and in fp32 split, once.
//
// Measured, groups of 64: one row for each of two of eight experts of 2048 x 1024 3.3 us a call; 64 experts of that
// with a row each 34 us in bf16 (33% of the copy rate), 65 in fp32; 25 experts of 4200 x 5064, whose rows lie on
// 4-byte boundaries only, 245 and 340.
// With 64 experts neither memory (DRAM busy 24% in bf16, 13% in fp32) nor issue (40% of the cycles) is full: the 13 warps
// an SM that 128 registers leave wait for loads of 4 and 8 bytes a lane.
#include <algorithm>

#include "expert_few.cuh"

namespace emb {

namespace {

// Codes k and k + 4 of a word of eight, less eight, as bf16: 128 + code is exact, and so is the difference.
__device__ __forceinline__ uint32_t codes_at(uint32_t word, int k) {
  const uint32_t v = ((word >> (4 * k)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Eight elements of a row of x as the fragments of two products: pairs (k, k + 4) of each plane.
template <typename T, int PLANES>
__device__ __forceinline__ void x_pairs(const Raw<T, 8>& x, uint32_t (&f)[PLANES][4]) {
  if constexpr (PLANES == 1) {
    f[0][0] = __byte_perm(x.w[0], x.w[2], 0x5410), f[0][1] = __byte_perm(x.w[0], x.w[2], 0x7632);
    f[0][2] = __byte_perm(x.w[1], x.w[3], 0x5410), f[0][3] = __byte_perm(x.w[1], x.w[3], 0x7632);
  } else {
    float p[3][8];
    planes_of(x.w, p);
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[q][i] = pair_bf16(p[q][i], p[q][i + 4]);
  }
}

// W words of eight codes, zero from byte `valid` on.  From any byte: the two aligned words that hold one, shifted, or
// byte by byte at the ends of the codes, [lo, hi).
template <int W>
__device__ __forceinline__ void load_codes(const uint8_t* q, int valid, bool vec, uintptr_t lo, uintptr_t hi, uint32_t (&w)[W]) {
  if (vec && valid >= 4 * W) {
    if constexpr (W == 1) w[0] = *reinterpret_cast<const uint32_t*>(q);
    if constexpr (W == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      w[0] = v.x, w[1] = v.y;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    w[j] = 0;
    const int left = valid - 4 * j;
    if (left <= 0) continue;
    const uintptr_t at = reinterpret_cast<uintptr_t>(q + 4 * j), from = at & ~(uintptr_t)3;
    const uint32_t s = (uint32_t)(at - from) * 8;
    if (from >= lo && from + 8 <= hi) {
      const uint32_t a = *reinterpret_cast<const uint32_t*>(from), b = reinterpret_cast<const uint32_t*>(from)[1];
      w[j] = __funnelshift_r(a, b, s);
      if (left < 4) w[j] &= (1u << (8 * left)) - 1;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) w[j] |= (uint32_t)q[4 * j + i] << (8 * i);
    }
  }
}

// W: words (of eight codes) that a lane takes of a step: 1, or 2 where groups of 64 and codes on
// eight-byte boundaries allow it: the four lanes of an output stay inside a group.  NT: eights of rows.  U: steps loaded ahead.  share: warps
// that share a tile's contraction; MT: tiles of 16 outputs of a warp, for which x is brought and split once.
template <typename T, int W, int NT, int U, int share, int MT>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_linear4(const T* x, int64_t x_ld, int x_vec, const int32_t* offsets, int E, int S, const uint8_t* q, const float* scale,
              int in, int out_dim, int q_vec, int per_group, int groups, T* out, int64_t out_ld, int tile0) {
  constexpr int PLANES = sizeof(T) == 4 ? 3 : 1, RT = 8 * NT, SPAN = 32 * W;  // SPAN: k of a step
  __shared__ float sums[kFewWarps][RT][16 * MT + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  wait_for_earlier();
  let_next_start();
  int e, r0, rows;
  if (!few_tile(offsets, E, S, RT, tile0 + (int)blockIdx.y, lane, e, r0, rows)) return;
  const int row_bytes = (in + 1) / 2, steps = (in + SPAN - 1) / SPAN;
  constexpr int tiles = kFewWarps / share, OUTS = 16 * MT;
  const int o0 = (blockIdx.x * tiles + warp / share) * OUTS;
  float acc[MT][NT][4] = {};
  // this lane's two outputs of each tile (held inside the matrix: what lies past its end is not stored)
  uint32_t oa[MT], ob[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) oa[i] = min(o0 + 16 * i + g, out_dim - 1), ob[i] = min(o0 + 16 * i + g + 8, out_dim - 1);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(q), hi = lo + (int64_t)E * out_dim * row_bytes;
  q += (int64_t)e * out_dim * row_bytes, scale += (int64_t)e * out_dim * groups;
  x += (int64_t)r0 * x_ld;
  for (int s0 = warp % share; s0 < steps; s0 += share * U) {
    uint32_t wa[U][MT][W], wb[U][MT][W];
    float fa[U][MT], fb[U][MT];
    Raw<T, 8> rx[U][W][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int st = s0 + u * share, k0 = st * SPAN + t * (8 * W), b0 = k0 / 2;
      const bool there = k0 < in;
      const int gi = per_group == 1 ? st : st / per_group;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        load_codes<W>(q + (int64_t)oa[i] * row_bytes + (there ? b0 : 0), there ? row_bytes - b0 : 0, q_vec, lo, hi, wa[u][i]);
        load_codes<W>(q + (int64_t)ob[i] * row_bytes + (there ? b0 : 0), there ? row_bytes - b0 : 0, q_vec, lo, hi, wb[u][i]);
        fa[u][i] = st < steps ? scale[(int64_t)oa[i] * groups + gi] : 0.f;
        fb[u][i] = st < steps ? scale[(int64_t)ob[i] * groups + gi] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          const int r = g + 8 * m, k = k0 + 8 * j;
          rx[u][j][m].load(x + (int64_t)(r < rows ? r : 0) * x_ld + (k < in ? k : 0), r < rows ? in - k : 0, x_vec);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t f[W][NT][PLANES][4];
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int m = 0; m < NT; ++m) x_pairs<T, PLANES>(rx[u][j][m], f[j][m]);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float part[NT][4] = {};
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {codes_at(wa[u][i][j], 2 * h), codes_at(wb[u][i][j], 2 * h), codes_at(wa[u][i][j], 2 * h + 1),
                                   codes_at(wb[u][i][j], 2 * h + 1)};
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
              for (int pl = PLANES - 1; pl >= 0; --pl) mma16816(part[m], a, f[j][m][pl][2 * h], f[j][m][pl][2 * h + 1]);
          }
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          acc[i][m][0] = fmaf(fa[u][i], part[m][0], acc[i][m][0]), acc[i][m][1] = fmaf(fa[u][i], part[m][1], acc[i][m][1]);
          acc[i][m][2] = fmaf(fb[u][i], part[m][2], acc[i][m][2]), acc[i][m][3] = fmaf(fb[u][i], part[m][3], acc[i][m][3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int m = 0; m < NT; ++m)
#pragma unroll
      for (int k = 0; k < 4; ++k) sums[warp][m * 8 + 2 * t + (k & 1)][16 * i + g + 8 * (k >> 1)] = acc[i][m][k];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * tiles * OUTS; i += kFewThreads) {
    const int o = i % OUTS, j = i / OUTS % tiles, r = i / (OUTS * tiles), col = (blockIdx.x * tiles + j) * OUTS + o;
    float v[1] = {0.f};
#pragma unroll
    for (int w = 0; w < share; ++w) v[0] += sums[j * share + w][r][o];
    if (col < out_dim) {
      Pack<T, 1> p;
      p.set(v);
      p.store(out + (int64_t)(r0 + r) * out_ld + col);
    }
  }
}

// One group of a row a warp pass: scale = max|w| / 7, code = w / scale rounded to the nearest integer
// (ties to even) + 8.
template <typename T>
__global__ void __launch_bounds__(256)
    k_quantize_rows4(const T* w, int64_t w_ld, int64_t n, int d, int group, uint8_t* q, float* scale) {
  wait_for_earlier();
  let_next_start();
  const int lane = threadIdx.x & 31, groups = (d + group - 1) / group, row_bytes = (d + 1) / 2;
  const int64_t all = n * groups;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5; i < all; i += (int64_t)gridDim.x * 8) {
    const int64_t r = i / groups;
    const int c0 = (int)(i - r * groups) * group, c1 = min(d, c0 + group);
    const T* row = w + r * w_ld;
    const auto at = [&](int c) {
      float v[1] = {0.f};
      if (c < c1) {
        Pack<T, 1> p;
        p.load(row + c);
        p.get(v);
      }
      return v[0];
    };
    float most = 0.f;
    for (int c = c0 + lane; c < c1; c += 32) most = fmaxf(most, fabsf(at(c)));
    for (int o = 16; o >= 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    const float s = __fdiv_rn(most, 7.f);
    const auto code = [&](int c) {
      const int v = s > 0.f ? __float2int_rn(__fdiv_rn(at(c), s)) : 0;
      return (uint32_t)(min(max(v, -7), 7) + 8);
    };
    for (int c = c0 + 2 * lane; c < c1; c += 64) q[r * row_bytes + c / 2] = (uint8_t)(code(c) | code(c + 1) << 4);
    if (lane == 0) scale[i] = s;
  }
}

template <typename T, int W, int NT>
cudaError_t run_linear4(const emb_product4& a, bool q_vec, cudaStream_t s) {
  constexpr bool F32 = sizeof(T) == 4;
  // Warps of their own for 64 outputs (fp32 with 32 rows: 32) where these fill the SMs, else eight warps for 16.
  constexpr int MT = F32 && NT == 4 ? 2 : 4;
  // Steps loaded ahead.  Shared tiles: two, and where a warp has more of them four in bf16 (with two steps a warp, four
  // take longer for the masks: 3.6 -> 4.3 us for a single request; in fp32 they leave room for one CTA an SM: 1 x
  // 7616 x 3664 29 -> 46 us).  Alone: what registers for two CTAs an SM hold.
  constexpr int U = NT == 4 ? 1 : 2, MORE = F32 || NT > 1 ? U : 4, ALONE = !F32 && W == 1 && NT <= 2 ? 2 : 1;
  const int groups = (a.in + a.group - 1) / a.group, x_vec = rows16(a.d_x, a.x_ld, sizeof(T));
  const int64_t across = (a.out + 15) / 16, all = few_tiles(a.rows, a.experts, 8 * NT);
  const bool alone = all * across >= (int64_t)device_sms() * 8 * MT, more = (a.in + 32 * W - 1) / (32 * W) > 2 * kFewWarps;
  const int wide = alone ? kFewWarps * MT : 1;  // tiles of a CTA
  const auto run = [&](auto kern, int64_t tile0, int64_t tiles) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((across + wide - 1) / wide), (unsigned)tiles);
    cfg.blockDim = dim3(kFewThreads), cfg.stream = s, cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(a.d_x), a.x_ld, x_vec, a.d_offsets, (int)a.experts, (int)a.rows,
                              (const uint8_t*)a.d_q, (const float*)a.d_scale, (int)a.in, (int)a.out, (int)q_vec, (int)a.group / (32 * W), groups,
                              static_cast<T*>(a.d_out), a.out_ld, (int)tile0);
  };
  // (a grid has 65535 rows at most)
  for (int64_t at = 0; at < all; at += 65535) {
    const int64_t n = std::min<int64_t>(65535, all - at);
    const cudaError_t e = alone  ? run(k_linear4<T, W, NT, ALONE, 1, MT>, at, n)
                          : more ? run(k_linear4<T, W, NT, MORE, kFewWarps, 1>, at, n)
                                 : run(k_linear4<T, W, NT, U, kFewWarps, 1>, at, n);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t linear4_of(const emb_product4& a, cudaStream_t s) {
  const int64_t each = (a.rows + a.experts - 1) / a.experts;  // rows of an expert, on average
  const uint64_t on = reinterpret_cast<uintptr_t>(a.d_q) | (uint64_t)((a.in + 1) / 2);
  if (each > 8) return each <= 16 ? run_linear4<T, 1, 2>(a, on % 4 == 0, s) : run_linear4<T, 1, 4>(a, on % 4 == 0, s);
  if constexpr (sizeof(T) == 2)
    if (a.group % 64 == 0 && on % 8 == 0) return run_linear4<T, 2, 1>(a, true, s);
  return run_linear4<T, 1, 1>(a, on % 4 == 0, s);
}

}  // namespace

cudaError_t launch_linear4(const emb_product4& a, cudaStream_t s) {
  if (a.rows == 0) return cudaSuccess;
  return a.dtype == EMB_BF16 ? linear4_of<__nv_bfloat16>(a, s) : linear4_of<float>(a, s);
}

cudaError_t launch_quantize_rows4(const void* w, int64_t w_ld, int64_t n, int d, int bf16, int group, uint8_t* q,
                                  float* scale, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int64_t groups = n * ((d + group - 1) / group);
  const unsigned grid = (unsigned)std::min<int64_t>((groups + 7) / 8, (int64_t)device_sms() * 32);
  return bf16 ? launch_early(k_quantize_rows4<__nv_bfloat16>, grid, 256, 0, s, static_cast<const __nv_bfloat16*>(w), w_ld, n, d, group, q, scale)
              : launch_early(k_quantize_rows4<float>, grid, 256, 0, s, static_cast<const float*>(w), w_ld, n, d, group, q, scale);
}

}  // namespace emb
