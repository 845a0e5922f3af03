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
// contraction and add up through shared memory in a fixed order.
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

// W words of eight codes, zero from byte `valid` on.
template <int W>
__device__ __forceinline__ void load_codes(const uint8_t* q, int valid, bool vec, uint32_t (&w)[W]) {
  if (vec && valid >= 4 * W) {
    if constexpr (W == 1) w[0] = *reinterpret_cast<const uint32_t*>(q);
    if constexpr (W == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(q);
      w[0] = v.x, w[1] = v.y;
    }
    if constexpr (W == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(q);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = 0;
  if (valid <= 0) return;
#pragma unroll
  for (int j = 0; j < W; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * j + i < valid) w[j] |= (uint32_t)q[4 * j + i] << (8 * i);
  }
}

// W: words (of eight codes) that a lane takes of a step: 1 for groups of 32, 2 of 64, 4 of 128 and more, so
// that the four lanes of an output stay inside a group.  NT: eights of rows.  U: steps loaded ahead.  share: warps
// that share a tile's contraction.
template <typename T, int W, int NT, int U, int share>
__global__ void __launch_bounds__(kFewThreads)
    k_linear4(const T* x, int64_t x_ld, int x_vec, const int32_t* offsets, int E, int S, const uint8_t* q, const float* scale,
              int in, int out_dim, int q_vec, int per_group, int groups, T* out, int64_t out_ld, int tile0) {
  constexpr int PLANES = sizeof(T) == 4 ? 3 : 1, RT = 8 * NT, SPAN = 32 * W;  // SPAN: k of a step
  __shared__ float sums[kFewWarps][RT][17];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  wait_for_earlier();
  let_next_start();
  int e, r0, rows;
  if (!few_tile(offsets, E, S, RT, tile0 + (int)blockIdx.y, lane, e, r0, rows)) return;
  const int row_bytes = (in + 1) / 2, steps = (in + SPAN - 1) / SPAN;
  constexpr int tiles = kFewWarps / share;
  const int o0 = (blockIdx.x * tiles + warp / share) * 16;
  float acc[NT][4] = {};
  // this lane's two outputs (held inside the matrix: what lies past its end is not stored)
  const int64_t oa = (int64_t)e * out_dim + min(o0 + g, out_dim - 1), ob = (int64_t)e * out_dim + min(o0 + g + 8, out_dim - 1);
  const uint8_t *qa = q + oa * row_bytes, *qb = q + ob * row_bytes;
  const float *sa = scale + oa * groups, *sb = scale + ob * groups;
  x += (int64_t)r0 * x_ld;
  for (int s0 = warp % share; s0 < steps; s0 += share * U) {
    uint32_t wa[U][W], wb[U][W];
    float fa[U], fb[U];
    Raw<T, 8> rx[U][W][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int st = s0 + u * share, k0 = st * SPAN + t * (8 * W), b0 = k0 / 2;
      const bool there = k0 < in;
      load_codes<W>(qa + (there ? b0 : 0), there ? row_bytes - b0 : 0, q_vec, wa[u]);
      load_codes<W>(qb + (there ? b0 : 0), there ? row_bytes - b0 : 0, q_vec, wb[u]);
      const int gi = per_group == 1 ? st : st / per_group;
      fa[u] = st < steps ? sa[gi] : 0.f, fb[u] = st < steps ? sb[gi] : 0.f;
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
      float part[NT][4] = {};
#pragma unroll
      for (int j = 0; j < W; ++j) {
        uint32_t f[NT][PLANES][4];
#pragma unroll
        for (int m = 0; m < NT; ++m) x_pairs<T, PLANES>(rx[u][j][m], f[m]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a[4] = {codes_at(wa[u][j], 2 * h), codes_at(wb[u][j], 2 * h), codes_at(wa[u][j], 2 * h + 1),
                                 codes_at(wb[u][j], 2 * h + 1)};
#pragma unroll
          for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int pl = PLANES - 1; pl >= 0; --pl) mma16816(part[m], a, f[m][pl][2 * h], f[m][pl][2 * h + 1]);
        }
      }
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        acc[m][0] = fmaf(fa[u], part[m][0], acc[m][0]), acc[m][1] = fmaf(fa[u], part[m][1], acc[m][1]);
        acc[m][2] = fmaf(fb[u], part[m][2], acc[m][2]), acc[m][3] = fmaf(fb[u], part[m][3], acc[m][3]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][m * 8 + 2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[m][i];
  __syncthreads();
  for (int i = threadIdx.x; i < rows * tiles * 16; i += kFewThreads) {
    const int o = i & 15, j = (i >> 4) % tiles, r = (i >> 4) / tiles, col = (blockIdx.x * tiles + j) * 16 + o;
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
cudaError_t run_linear4(const emb_product4& a, cudaStream_t s) {
  const int row_bytes = (a.in + 1) / 2, groups = (a.in + a.group - 1) / a.group;
  const bool vec_q = row_bytes % (4 * W) == 0 && reinterpret_cast<uintptr_t>(a.d_q) % (4 * W) == 0;
  const int x_vec = rows16(a.d_x, a.x_ld, sizeof(T));
  const int64_t across = (a.out + 15) / 16, all = few_tiles(a.rows, a.experts, 8 * NT);
  const int share = few_share(all * across), wide = kFewWarps / share;
  const auto run = [&](auto kern, int64_t tile0, int64_t tiles) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((across + wide - 1) / wide), (unsigned)tiles);
    cfg.blockDim = dim3(kFewThreads), cfg.stream = s, cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(a.d_x), a.x_ld, x_vec, a.d_offsets, (int)a.experts, (int)a.rows,
                              (const uint8_t*)a.d_q, (const float*)a.d_scale, (int)a.in, (int)a.out, (int)vec_q, (int)a.group / (32 * W), groups,
                              static_cast<T*>(a.d_out), a.out_ld, (int)tile0);
  };
  // (a grid has 65535 rows at most)
  // steps loaded ahead: two, and where a warp has more of them four in bf16 (with two steps a warp, four take longer for
  // the masks: 3.6 -> 4.3 us for a single request; in fp32 four leave room for one CTA an SM: 1 x 7616 x 3664 29 -> 46 us)
  constexpr int PLANES = sizeof(T) == 4 ? 3 : 1, U = W * NT * (PLANES == 3 ? 2 : 1) <= 4 ? 2 : 1, MORE = W * NT <= 2 && PLANES == 1 ? 4 : U;
  const bool more = (a.in + 32 * W - 1) / (32 * W) > 2 * share;
  for (int64_t at = 0; at < all; at += 65535) {
    const int64_t n = std::min<int64_t>(65535, all - at);
    const cudaError_t e = share != kFewWarps ? run(k_linear4<T, W, NT, MORE, kFewAlone>, at, n)
                          : more             ? run(k_linear4<T, W, NT, MORE, kFewWarps>, at, n)
                                             : run(k_linear4<T, W, NT, U, kFewWarps>, at, n);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int W>
cudaError_t linear4_rows(const emb_product4& a, cudaStream_t s) {
  const int64_t each = (a.rows + a.experts - 1) / a.experts;  // rows of an expert, on average
  return each <= 8 ? run_linear4<T, W, 1>(a, s) : each <= 16 ? run_linear4<T, W, 2>(a, s) : run_linear4<T, W, 4>(a, s);
}

template <typename T>
cudaError_t linear4_of(const emb_product4& a, cudaStream_t s) {
  return a.group % 128 == 0 ? linear4_rows<T, 4>(a, s) : a.group % 64 == 0 ? linear4_rows<T, 2>(a, s) : linear4_rows<T, 1>(a, s);
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
