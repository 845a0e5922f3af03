// Shared by the products of few rows: which expert and rows a CTA has, the warp's matrix instruction, and
// the sum over a CTA's warps.
#pragma once

#include "expert_mm.cuh"

namespace emb {

constexpr int kFewWarps = 8, kFewThreads = 32 * kFewWarps;

// Tile j of the experts' rows, `most` to a tile, counted through the experts in order (every lane gets it);
// false behind the last.  Each warp looks for itself: no barrier stands before its first loads.
__device__ __forceinline__ bool few_tile(const int32_t* offsets, int E, int S, int most, int j, int lane, int& e, int& r0, int& rows) {
  if (offsets == nullptr) {
    e = 0, r0 = j * most, rows = min(most, S - r0);
    return rows > 0;
  }
  int before = 0;
  for (int b = 0; b < E; b += 32) {
    const int i = b + lane;
    const int lo = i < E ? min(max(offsets[i], 0), S) : S, hi = i < E ? max(min(max(offsets[i + 1], 0), S), lo) : S;
    const int n = (hi - lo + most - 1) / most;
    int c = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c += v;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + c > j);
    if (past) {
      const int at = __ffs(past) - 1;
      e = b + at;
      r0 = __shfl_sync(0xFFFFFFFFu, lo + (j - before - (c - n)) * most, at);
      rows = min(most, __shfl_sync(0xFFFFFFFFu, hi, at) - r0);
      return true;
    }
    before += __shfl_sync(0xFFFFFFFFu, c, 31);
  }
  return false;
}

// Tiles of S rows in E experts, at most.
inline int64_t few_tiles(int64_t S, int E, int most) { return S / most + (E < S ? E : S); }

// Warps that share a tile's contraction: all of a CTA's, or one alone where the tiles are so many that their warps fill
// the SMs (a CTA of eight warps for each of 8313 tiles with 352 inputs took 83 us, most of it in starting CTAs;
// two warps a tile 66, one 51).
constexpr int kFewAlone = 1;
inline int few_share(int64_t tiles) { return tiles >= (int64_t)device_sms() * 16 ? kFewAlone : kFewWarps; }

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pair_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive elements as loaded, zero from `valid` on: words of two bf16, or fp32.
template <typename T, int N>
struct Raw {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p, int valid, bool vec) {
    if (vec && valid >= N) {
      if constexpr (kWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 q = reinterpret_cast<const uint4*>(p)[i];
          w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x, w[1] = q.y;
      }
      return;
    }
    if (valid <= 0) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0u;
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = i < valid ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
      } else {
        const uint32_t lo = 2 * i < valid ? reinterpret_cast<const uint16_t*>(p)[2 * i] : 0u;
        const uint32_t hi = 2 * i + 1 < valid ? reinterpret_cast<const uint16_t*>(p)[2 * i + 1] : 0u;
        w[i] = lo | hi << 16;
      }
    }
  }
};

// fp32 values as three bf16 planes, and pairs of them as words
template <int N>
__device__ __forceinline__ void planes_of(const uint32_t (&v)[N], float (&p)[3][N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) split3(__uint_as_float(v[i]), p[0][i], p[1][i], p[2][i]);
}

}  // namespace emb
