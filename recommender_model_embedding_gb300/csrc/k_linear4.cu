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
// contraction and add up through shared memory in a fixed order.  Where outputs are many, each warp takes tiles of its
// own and streams their codes through shared memory (k_linear4_stream; with fewer, in fp32, a CTA two tiles), or,
// where codes do not start on the boundaries that its copies need, loads them for 64 (with 32 rows: 32) outputs at a
// time.
//
// Measured, groups of 64: one row for each of two of eight experts of 2048 x 1024 3.3 us a call; 64 experts of that
// with a row each 30 us in bf16 (37% of the copy rate) and 38 in fp32 (34 and 65 with loads in place of the ring); 25
// experts of 4200 x 5064, whose rows lie on 4-byte boundaries only, 130 and 173 (245 and 340).
// An instruction is issued in 53 to 62% of the cycles there and DRAM busy for 23 to 32%: some 280 instructions for
// 128 codes of 16 outputs, 140 of them for taking the codes apart and multiplying, hold it up before memory does.
#include <algorithm>

#include "expert_few.cuh"
#include "interact_common.cuh"

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
// eight-byte boundaries allow it: the four lanes of an output stay inside a group.  NT: eights of rows.  U: steps
// loaded ahead.  share: warps that share a tile's contraction; MT: tiles of 16 outputs of a warp, for which x is
// brought and split once.
template <typename T, int W, int NT, int U, int share, int MT>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_linear4(const T* x, int64_t x_ld, int x_vec, const int32_t* offsets, int E, int S, const uint8_t* q, const float* scale,
              int in, int out_dim, int q_vec, int per_group, int groups, T* out, int64_t out_ld, int tile0) {
  constexpr int PLANES = sizeof(T) == 4 ? 3 : 1, RT = 8 * NT, SPAN = 32 * W;  // SPAN: k of a step
  __shared__ float sums[kFewWarps][RT][16 * MT + 1];
  static_assert(sizeof(sums) <= 48 * 1024, "shared memory of a fixed size");
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

// The same where outputs are many, codes start on a 16-byte boundary and their rows on 4-byte boundaries.  Each warp
// has tiles of 16 outputs of its own, up to MT at a time, and streams their codes and scales through a ring in shared
// memory, four stages (of 128 codes of 16 outputs) ahead of the one it multiplies; the CTA's rows of x lie beside
// them as the fragments they are taken as, up to KC columns at a time, so that they are brought, and in fp32 split,
// once for all warps.  Codes come in whole pieces of 16 bytes: four for an output's 64 bytes where rows start on such
// boundaries (WHOLE), else five.
constexpr int kRing4 = 5, kCodes4 = 128, kBytes4 = kCodes4 / 2;
constexpr int kPitch4 = kBytes4 + 16;                     // from one output's codes to the next: eight rows meet no bank twice
constexpr int kScales4 = 16 * kPitch4;                    // behind the codes, [step of 32 codes][output]
constexpr int kStage4 = kScales4 + kCodes4 / 32 * 16 * 4;
template <typename T, int NT>
struct Stream4 {
  static constexpr int PLANES = sizeof(T) == 4 ? 3 : 1, MT = PLANES == 3 && NT == 4 ? 2 : 4;
  static constexpr int KC = (PLANES == 3 ? 1024 : 2048) / NT, kX = KC / 32 * NT * PLANES * 512;
  static constexpr int kSmem = kX + kFewWarps * kRing4 * kStage4;
};

// `bytes` of N, zero behind them.
template <int N>
__device__ __forceinline__ void copy_ahead(uint32_t to, const void* from, int bytes) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

// SHARED: the CTA's tiles are all its warps', each of which takes every eighth stage of the columns; they add up at
// the end.
template <typename T, int NT, bool WHOLE, bool SHARED>
__global__ void __launch_bounds__(kFewThreads, 2)
    k_linear4_stream(const T* x, int64_t x_ld, int x_vec, const int32_t* offsets, int E, int S, const uint8_t* q, const float* scale,
                     int in, int out_dim, FastDiv per_group, int groups, T* out, int64_t out_ld, int tile0, int each) {
  using C = Stream4<T, NT>;
  constexpr int PLANES = C::PLANES, MT = C::MT, KC = C::KC, RT = 8 * NT;
  extern __shared__ __align__(16) unsigned char room4[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  wait_for_earlier();
  let_next_start();
  int e, r0, rows;
  if (!few_tile(offsets, E, S, RT, tile0 + (int)blockIdx.y, lane, e, r0, rows)) return;
  const int row_bytes = (in + 1) / 2, chunks = (in + KC - 1) / KC;
  constexpr int STEP = SHARED ? kFewWarps : 1;
  const int start = SHARED ? warp : 0;  // this warp's first stage of a chunk
  const int o0 = (SHARED ? blockIdx.x : blockIdx.x * kFewWarps + warp) * 16 * each;
  const int mine = min(max((out_dim - o0 + 15) / 16, 0), each);  // tiles of this warp
  const uint8_t* const end = q + (int64_t)E * out_dim * row_bytes;
  q += (int64_t)e * out_dim * row_bytes, scale += (int64_t)e * out_dim * groups;
  x += (int64_t)r0 * x_ld;
  uint4* const xs = reinterpret_cast<uint4*>(room4);
  unsigned char* const ring = room4 + C::kX + warp * (kRing4 * kStage4);
  const auto stages_of = [&](int c) { return (min(KC, in - c * KC) + kCodes4 - 1) / kCodes4; };
  // codes of output o of this warp's tile i (the last one's behind the matrix: what they give is not stored)
  const auto codes = [&](int i, int o) { return q + (int64_t)min(o0 + 16 * i + o, out_dim - 1) * row_bytes; };

  // The next stage to bring: its chunk, tile (nf + ni) and place; this lane's pieces of it, and its scales.
  constexpr int PIECES = WHOLE ? 4 : 5, COPIES = (16 * PIECES + 31) / 32;
  const uint8_t* from[COPIES];
  const float* from_scale = scale;
  int nf = 0, nc = 0, ni = 0, nq = start, k0 = start * kCodes4, nstages = stages_of(0);
  const auto place = [&] {
#pragma unroll
    for (int j = 0; j < COPIES; ++j) {
      const int i = j * 32 + lane;
      from[j] = codes(nf + ni, i / PIECES) + k0 / 2;
      from[j] -= reinterpret_cast<uintptr_t>(from[j]) & 15;
      from[j] += i % PIECES * 16;
    }
    from_scale = scale + (int64_t)min(o0 + 16 * (nf + ni) + (lane & 15), out_dim - 1) * groups;
  };
  if (start >= nstages) nf = mine;  // (a warp without a stage of the first chunk has none of the others)
  if (nf < mine) place();
  const auto bring = [&](int slot) {
    if (nf < mine) {
      const uint32_t at = smem_u32(ring + slot * kStage4);
      // whole stages, five pieces of which end inside the row
      const bool inside = k0 + (WHOLE ? 1 : 2) * kCodes4 <= in;
#pragma unroll
      for (int j = 0; j < COPIES; ++j) {
        const int i = j * 32 + lane, r = i / PIECES, piece = i % PIECES;
        if (16 * PIECES % 32 != 0 && i >= 16 * PIECES) break;
        int bytes = 16;
        const uint8_t* source = from[j];
        if (!inside) {  // none from behind the row's end, nor the matrices'
          if (WHOLE) {
            bytes = k0 / 2 + 16 * piece < row_bytes ? 16 : 0;
          } else {
            const int64_t left = codes(nf + ni, r) + row_bytes - from[j], all = end - from[j];
            bytes = left > 0 ? (int)(all < 16 ? all : 16) : 0;
          }
          if (bytes == 0) source = q - (reinterpret_cast<uintptr_t>(q) & 15);  // (a place to copy nothing from, on its boundary too)
        }
        copy_ahead<16>(at + r * kPitch4 + piece * 16, source, bytes);
        from[j] += STEP * kBytes4;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int u = j * 2 + (lane >> 4), k = k0 + 32 * u;
        const bool there = inside || k < in;
        copy_ahead<4>(at + kScales4 + (j * 32 + lane) * 4, from_scale + (there ? per_group.div((uint32_t)k / 32) : 0), there ? 4 : 0);
      }
      k0 += STEP * kCodes4, nq += STEP;
      if (nq >= nstages) {
        nq = start, k0 = nc * KC + start * kCodes4;
        if (++ni == min(MT, mine - nf)) {
          ni = 0;
          if (++nc == chunks) nc = 0, nf += MT;
          nstages = stages_of(nc), k0 = nc * KC + start * kCodes4;
          if (SHARED && start >= nstages) nf = mine;  // (the last chunk is shorter, and its tiles are the last)
          if (nf < mine) place();
        } else if (!SHARED && o0 + 16 * (nf + ni) + 16 <= out_dim) {  // 16 rows on, as far from a boundary
#pragma unroll
          for (int j = 0; j < COPIES; ++j) from[j] += 16 * (int64_t)row_bytes - nstages * kBytes4;
          from_scale += 16 * groups;
        } else {
          place();
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kRing4 - 1; ++s) bring(s);

  // where this lane's two outputs' codes start in a stage (in every tile as in the first)
  const uint32_t ga = g * kPitch4 + t * 4 + (WHOLE ? 0 : reinterpret_cast<uintptr_t>(codes(0, g)) & 15);
  const uint32_t gb = (g + 8) * kPitch4 + t * 4 + (WHOLE ? 0 : reinterpret_cast<uintptr_t>(codes(0, g + 8)) & 15);
  int slot = 0;
  for (int first = 0; first < each; first += MT) {
    float acc[MT][NT][4] = {};
    for (int c = 0; c < chunks; ++c) {
      const int stages = stages_of(c);
      if (first == 0) {  // (more than MT tiles are a warp's only where one piece holds all columns)
        if (c) __syncthreads();
        for (int i = warp; i < stages * (kCodes4 / 32) * NT; i += kFewWarps) {
          const int r = g + 8 * (i % NT), k = c * KC + i / NT * 32 + t * 8;
          Raw<T, 8> v;
          v.load(x + (int64_t)(r < rows ? r : 0) * x_ld + (k < in ? k : 0), r < rows ? in - k : 0, x_vec);
          uint32_t f[PLANES][4];
          x_pairs<T, PLANES>(v, f);
#pragma unroll
          for (int pl = 0; pl < PLANES; ++pl) xs[(i * PLANES + pl) * 32 + lane] = make_uint4(f[pl][0], f[pl][1], f[pl][2], f[pl][3]);
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (first + i >= mine) break;
        for (int st = start; st < stages; st += STEP) {
          // this stage has come, and all lanes are done with the one whose place is filled again
          asm volatile("cp.async.wait_group %0;" ::"n"(kRing4 - 2) : "memory");
          __syncwarp();
          bring(slot == 0 ? kRing4 - 1 : slot - 1);
          const unsigned char* at = ring + slot * kStage4;
          slot = slot + 1 == kRing4 ? 0 : slot + 1;
#pragma unroll
          for (int u = 0; u < kCodes4 / 32; ++u) {
            const uint32_t wa = *reinterpret_cast<const uint32_t*>(at + ga + u * 16);
            const uint32_t wb = *reinterpret_cast<const uint32_t*>(at + gb + u * 16);
            const float* s = reinterpret_cast<const float*>(at + kScales4) + u * 16 + g;
            const float fa = s[0], fb = s[8];
            uint32_t a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              a[h][0] = codes_at(wa, 2 * h), a[h][1] = codes_at(wb, 2 * h), a[h][2] = codes_at(wa, 2 * h + 1), a[h][3] = codes_at(wb, 2 * h + 1);
#pragma unroll
            for (int m = 0; m < NT; ++m) {
              float part[4] = {};
#pragma unroll
              for (int pl = PLANES - 1; pl >= 0; --pl) {
                const uint4 f = xs[(((st * (kCodes4 / 32) + u) * NT + m) * PLANES + pl) * 32 + lane];
                mma16816(part, a[0], f.x, f.y), mma16816(part, a[1], f.z, f.w);
              }
              acc[i][m][0] = fmaf(fa, part[0], acc[i][m][0]), acc[i][m][1] = fmaf(fa, part[1], acc[i][m][1]);
              acc[i][m][2] = fmaf(fb, part[2], acc[i][m][2]), acc[i][m][3] = fmaf(fb, part[3], acc[i][m][3]);
            }
          }
        }
      }
    }
    if constexpr (SHARED) {
      float* const sums = reinterpret_cast<float*>(room4);  // [warp][row][output]
      const int wide = 16 * each;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MT; ++i)
        if (i < each)
#pragma unroll
          for (int m = 0; m < NT; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sums[(warp * RT + m * 8 + 2 * t + (k & 1)) * wide + 16 * i + g + 8 * (k >> 1)] = acc[i][m][k];
      __syncthreads();
      for (int i = threadIdx.x; i < rows * wide; i += kFewThreads) {
        const int r = i / wide, o = i - r * wide;
        float v[1] = {0.f};
#pragma unroll
        for (int w = 0; w < kFewWarps; ++w) v[0] += sums[(w * RT + r) * wide + o];
        if (o0 + o < out_dim) {
          Pack<T, 1> p;
          p.set(v);
          p.store(out + (int64_t)(r0 + r) * out_ld + o0 + o);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (first + i >= mine) break;  // (what follows is the next warp's)
#pragma unroll
        for (int m = 0; m < NT; ++m)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r = m * 8 + 2 * t + (k & 1), o = o0 + 16 * (first + i) + g + 8 * (k >> 1);
            if (r < rows && o < out_dim) {
              const float v[1] = {acc[i][m][k]};
              Pack<T, 1> p;
              p.set(v);
              p.store(out + (int64_t)(r0 + r) * out_ld + o);
            }
          }
      }
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
  // Tiles of a warp at a time where these fill the SMs, else eight warps share one.  (Four of 32 rows would be 66,560
  // bytes of sums, above the 48 KB that shared memory of a fixed size may take.)
  constexpr int MT = NT == 4 ? 2 : 4;
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
  using C = Stream4<T, NT>;
  // Tiles of a warp: such that the SM with most CTAs has least to do where rows spread evenly, a CTA's start taking
  // about the time of six stages, and fewer than two CTAs an SM as long as two.  Where one piece holds all columns, a
  // warp's tiles can be more than MT (242 experts of 7824 x 352 in bf16: 141 us, with at most four 180).
  const int64_t full = std::min<int64_t>(a.experts, a.rows), likely = full * (((a.rows + full - 1) / full + 8 * NT - 1) / (8 * NT));
  const int64_t stages = (a.in + kCodes4 - 1) / kCodes4;
  const auto cost = [&](int n) {
    const int64_t ctas = likely * ((across + kFewWarps * n - 1) / (kFewWarps * n));
    return std::max<int64_t>((ctas + device_sms() - 1) / device_sms(), 2) * (n * stages + 6);
  };
  int each = C::MT;
  for (const int n : {1, 2, 3, 6, 8, 12, 16})
    if ((n <= C::MT || a.in <= C::KC) && cost(n) < cost(each)) each = n;
  const int row_bytes = (a.in + 1) / 2;
  const bool ring = reinterpret_cast<uintptr_t>(a.d_q) % 16 == 0 && row_bytes % 4 == 0;
  // From six tiles an SM on.  At 3.4 (one expert of 8192 x 4096, groups of 32) the shared sum takes 17 us and the
  // ring 21; at 6.7 (eight of 2048 x 1024) 11.3 and 8.7, with groups of 64 and eight rows each 9.3 and 10.4; at 13
  // (16 of 2048 x 512) 14.5 and 6.2.  In fp32 34 and 33, 20 and 12, 21 and 8.
  const bool streams = ring && likely * across >= (int64_t)device_sms() * 6;
  // Below that the ring's CTAs share their tiles, two at a time, where splitting rows of fp32 anew for each costs
  // most: from two tiles an SM on (one expert of 8192 x 4096 37 us with the shared sum of single tiles and 26 with
  // this, two of 2600 x 2600 25 and 18; at 1.7, 4096 x 479, 4.1 and 4.5).  With 32 rows, and in bf16, it gains
  // nothing (101 and 116, 12.7 and 14.6).
  constexpr bool kPairs = F32 && NT <= 2;
  const bool shared = kPairs && ring && !streams && likely * across >= (int64_t)device_sms() * 2;
  if (shared) each = 2;
  const int wide4 = shared ? each : kFewWarps * each;
  const auto stream = [&](auto kern, int64_t tile0, int64_t tiles) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((across + wide4 - 1) / wide4), (unsigned)tiles);
    cfg.blockDim = dim3(kFewThreads), cfg.dynamicSmemBytes = C::kSmem, cfg.stream = s, cfg.attrs = &attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const T*>(a.d_x), a.x_ld, x_vec, a.d_offsets, (int)a.experts, (int)a.rows,
                              (const uint8_t*)a.d_q, (const float*)a.d_scale, (int)a.in, (int)a.out, FastDiv(a.group / 32), groups,
                              static_cast<T*>(a.d_out), a.out_ld, (int)tile0, each);
  };
  // (a grid has 65535 rows at most)
  for (int64_t at = 0; at < all; at += 65535) {
    const int64_t n = std::min<int64_t>(65535, all - at);
    if constexpr (kPairs)
      if (shared) {
        const cudaError_t e = row_bytes % 16 == 0 ? stream(k_linear4_stream<T, NT, true, true>, at, n)
                                                  : stream(k_linear4_stream<T, NT, false, true>, at, n);
        if (e != cudaSuccess) return e;
        continue;
      }
    if (streams) {
      const cudaError_t e = row_bytes % 16 == 0 ? stream(k_linear4_stream<T, NT, true, false>, at, n) : stream(k_linear4_stream<T, NT, false, false>, at, n);
      if (e != cudaSuccess) return e;
      continue;
    }
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
