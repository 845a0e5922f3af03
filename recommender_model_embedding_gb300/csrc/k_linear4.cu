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

#include "expert_mm.cuh"

namespace emb {

namespace {

constexpr int kL4Warps = 8, kL4Threads = 32 * kL4Warps;

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Codes k and k + 4 of a word of eight, less eight, as bf16: 128 + code is exact, and so is the difference.
__device__ __forceinline__ uint32_t codes_at(uint32_t word, int k) {
  const uint32_t v = ((word >> (4 * k)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ uint32_t pair_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight elements of a row of x from k on (zero from `valid` on) as the fragments of two products: pairs
// (k, k + 4) of each plane.
template <typename T, int PLANES>
__device__ __forceinline__ void x_pairs(const T* x, int valid, bool vec, uint32_t (&f)[PLANES][4]) {
  if constexpr (PLANES == 1) {
    uint32_t w[4];
    if (vec && valid >= 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(x);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < valid ? reinterpret_cast<const uint16_t*>(x)[2 * i] : 0u;
        const uint32_t hi = 2 * i + 1 < valid ? reinterpret_cast<const uint16_t*>(x)[2 * i + 1] : 0u;
        w[i] = lo | hi << 16;
      }
    }
    f[0][0] = __byte_perm(w[0], w[2], 0x5410), f[0][1] = __byte_perm(w[0], w[2], 0x7632);
    f[0][2] = __byte_perm(w[1], w[3], 0x5410), f[0][3] = __byte_perm(w[1], w[3], 0x7632);
  } else {
    float v[8];
    if (vec && valid >= 8) {
      const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < valid ? x[i] : 0.f;
    }
    float p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split3(v[i], p[0][i], p[1][i], p[2][i]);
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) f[q][i] = pair_bf16(p[q][i], p[q][i + 4]);
  }
}

// W: words (of eight codes) that a lane takes of a group's four lanes' share: 1 for groups of 32, 2 of
// 64, 4 of 128 and more.  NT: eights of rows.
template <typename T, int W, int NT, bool VEC_Q>
__global__ void __launch_bounds__(kL4Threads)
    k_linear4(const T* x, int64_t x_ld, int x_vec, const int32_t* offsets, int E, int S, const uint8_t* q, const float* scale,
              int in, int out_dim, int group, int col_tiles, T* out, int64_t out_ld) {
  constexpr int PLANES = sizeof(T) == 4 ? 3 : 1, RT = 8 * NT, SPAN = 32 * W;  // SPAN: k of a step
  __shared__ float sums[kL4Warps][RT][17];
  extern __shared__ int32_t tables[];
  int32_t *cuts = tables, *prefix = tables + E + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  wait_for_earlier();
  let_next_start();
  if (warp == 0) {
    expert_cuts(offsets, E, S, cuts, lane);
    expert_prefix(cuts, E, prefix, lane, [=](int rows) { return (rows + RT - 1) / RT; });
  }
  __syncthreads();
  const int row_bytes = (in + 1) / 2, groups = (in + group - 1) / group, steps = (in + SPAN - 1) / SPAN;
  const int per_group = group / SPAN;
  const int64_t tiles = (int64_t)prefix[E] * col_tiles;
  int e = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int rt = (int)(tile / col_tiles), o0 = (int)(tile - (int64_t)rt * col_tiles) * 16;
    while (rt >= prefix[e + 1]) ++e;
    const int r0 = cuts[e] + (rt - prefix[e]) * RT, rows = min(RT, cuts[e + 1] - r0);
    float acc[NT][4] = {};
    // this lane's two outputs (held inside the matrix: what lies past its end is not stored)
    const int oa = min(o0 + g, out_dim - 1), ob = min(o0 + g + 8, out_dim - 1);
    const int64_t base = (int64_t)e * out_dim;
    const uint8_t *qa = q + (base + oa) * row_bytes, *qb = q + (base + ob) * row_bytes;
    const float *sa = scale + (base + oa) * groups, *sb = scale + (base + ob) * groups;
    // warps take whole groups in turn
    for (int gi = warp; gi < groups; gi += kL4Warps) {
      float part[NT][4] = {};
      for (int st = gi * per_group; st < min(steps, (gi + 1) * per_group); ++st) {
        const int k0 = st * SPAN + t * (8 * W);
        uint32_t wa[W], wb[W];
        const int b0 = k0 / 2;
        if (VEC_Q && b0 + 4 * W <= row_bytes) {
          if constexpr (W == 1) wa[0] = *reinterpret_cast<const uint32_t*>(qa + b0), wb[0] = *reinterpret_cast<const uint32_t*>(qb + b0);
          if constexpr (W == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(qa + b0), v = *reinterpret_cast<const uint2*>(qb + b0);
            wa[0] = u.x, wa[1] = u.y, wb[0] = v.x, wb[1] = v.y;
          }
          if constexpr (W == 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(qa + b0), v = *reinterpret_cast<const uint4*>(qb + b0);
            wa[0] = u.x, wa[1] = u.y, wa[2] = u.z, wa[3] = u.w, wb[0] = v.x, wb[1] = v.y, wb[2] = v.z, wb[3] = v.w;
          }
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            wa[j] = wb[j] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (b0 + 4 * j + i < row_bytes) {
                wa[j] |= (uint32_t)qa[b0 + 4 * j + i] << (8 * i);
                wb[j] |= (uint32_t)qb[b0 + 4 * j + i] << (8 * i);
              }
          }
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const int k = k0 + 8 * j;
          uint32_t f[NT][PLANES][4];
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            const int r = g + 8 * m;
            x_pairs<T, PLANES>(x + (int64_t)(r0 + (r < rows ? r : 0)) * x_ld + (k < in ? k : 0), r < rows ? in - k : 0, x_vec, f[m]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {codes_at(wa[j], 2 * h), codes_at(wb[j], 2 * h), codes_at(wa[j], 2 * h + 1), codes_at(wb[j], 2 * h + 1)};
#pragma unroll
            for (int m = 0; m < NT; ++m)
#pragma unroll
              for (int pl = PLANES - 1; pl >= 0; --pl) mma16816(part[m], a, f[m][pl][2 * h], f[m][pl][2 * h + 1]);
          }
        }
      }
      const float fa = sa[gi], fb = sb[gi];
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        acc[m][0] = fmaf(fa, part[m][0], acc[m][0]), acc[m][1] = fmaf(fa, part[m][1], acc[m][1]);
        acc[m][2] = fmaf(fb, part[m][2], acc[m][2]), acc[m][3] = fmaf(fb, part[m][3], acc[m][3]);
      }
    }
#pragma unroll
    for (int m = 0; m < NT; ++m) {  // outputs g and g + 8, rows 2 t and 2 t + 1
      sums[warp][m * 8 + 2 * t][g] = acc[m][0], sums[warp][m * 8 + 2 * t + 1][g] = acc[m][1];
      sums[warp][m * 8 + 2 * t][g + 8] = acc[m][2], sums[warp][m * 8 + 2 * t + 1][g + 8] = acc[m][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < RT * 16; i += kL4Threads) {
      const int r = i >> 4, o = i & 15;
      float v[1] = {0.f};
#pragma unroll
      for (int w = 0; w < kL4Warps; ++w) v[0] += sums[w][r][o];
      if (r < rows && o0 + o < out_dim) {
        Pack<T, 1> p;
        p.set(v);
        p.store(out + (int64_t)(r0 + r) * out_ld + o0 + o);
      }
    }
    __syncthreads();
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
  const int row_bytes = (a.in + 1) / 2, col_tiles = (a.out + 15) / 16;
  const bool vec_q = row_bytes % (4 * W) == 0 && reinterpret_cast<uintptr_t>(a.d_q) % (4 * W) == 0;
  const int x_vec = rows16(a.d_x, a.x_ld, sizeof(T));
  const int64_t most = ((int64_t)a.rows / (8 * NT) + std::min<int64_t>(a.experts, a.rows)) * col_tiles;
  const unsigned grid = (unsigned)std::min<int64_t>(most, (int64_t)device_sms() * 16);
  const int smem = 2 * (a.experts + 1) * 4;
  const auto run = [&](auto kern) {
    return launch_early(kern, grid, kL4Threads, smem, s, static_cast<const T*>(a.d_x), a.x_ld, x_vec, a.d_offsets, (int)a.experts,
                        (int)a.rows, a.d_q, a.d_scale, (int)a.in, (int)a.out, (int)a.group, col_tiles, static_cast<T*>(a.d_out),
                        a.out_ld);
  };
  return vec_q ? run(k_linear4<T, W, NT, true>) : run(k_linear4<T, W, NT, false>);
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
