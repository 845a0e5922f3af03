// The experts' matrix products on the 5th-generation tensor cores, rows grouped by expert.
//
//   rows product      C[r] = A[r] B_e^T, r in expert e's rows  (out = x W^T, dx = dout W; gated: the
//                     gate's and the up half's columns side by side, h = act(g) u in the epilogue)
//   weight gradient   C_e = sum over e's rows r of A[r]^T B[r]   (dW = dout^T x)
//
// Both are one kernel: a pair of CTAs (a cluster on two SMs) computes tiles of 256 x 256, each CTA
// holding 128 rows of the accumulator in its tensor memory, with tcgen05.mma.cta_group::2 (M = 256,
// N = 256, K = 16) issued by one thread of the pair's first CTA.  Per 64 of K each CTA brings 128 x
// 64 of A and of B by TMA (16 KB each, 128-byte swizzle) into a ring of five stages; the pair reads
// B from both.  A tile alone in one CTA (128 x 256) would write 48 KB and read 48 KB of shared memory
// for the same arithmetic as 32 KB and 32 KB here, over what an SM's shared memory moves in
// that time.  Operands may run along either axis (the descriptors take K-major and
// MN-major tiles), so neither direction of the pass and neither layout of the weights moves data.
//
// The grid stays resident and walks the tiles of all experts in turn (columns fastest, so tiles that
// run together share rows of A and the expert's weights in L2); which tiles there are is worked out
// from the experts' offsets on the device, so the host never waits for them.  Accumulators
// alternate between the two halves of tensor memory: eight warps write one tile out while the next
// is computed.  Rows of a tile behind its expert's last are computed and not stored.  Where the
// contraction runs over rows (weight gradient), a stage's rows behind the expert's last are set to
// zero in both operands before the tensor core reads them (they may hold anything, NaN too).
//
// fp32: each operand is split into three bf16 planes, v = v0 + v1 + v2 (eight significant bits each),
// and the six products a_i b_j with i + j <= 2 are added, small ones first; what is left
// out is below 2^-24 of the product.  The tensor core adds in fp32 but does not round to nearest, so an
// error would grow with the length of the sum: fp32 results are therefore summed over parts of K in
// registers.  bf16 results take the accumulator as it is (its error, below 2^-12 at K = 65536, is inside
// bf16's rounding).
#include <algorithm>
#include <atomic>

#include "expert_mm.cuh"
#include "interact_common.cuh"
#include "tc_common.cuh"

namespace emb {

constexpr int kMmEpi = 8;                          // warps that write tiles out
constexpr int kMmWarpTma = kMmEpi, kMmWarpMma = kMmEpi + 1, kMmWarpRelay = kMmEpi + 2;
constexpr int kMmThreads = 32 * (kMmEpi + 3);
constexpr int kMmStages = 5;
constexpr int kMmOperand = 128 * 128;              // bytes of an operand's stage: 128 x 64 bf16
constexpr int kMmStage = 2 * kMmOperand;
constexpr int kMmStaging = 32 * 128;               // bytes of a writing warp: 32 rows of 128
constexpr int kMmOffStaging = kMmStages * kMmStage;
constexpr int kMmOffBars = kMmOffStaging + kMmEpi * kMmStaging;
constexpr int kMmNumBars = 3 * kMmStages + 4;
constexpr int kMmOffTmem = kMmOffBars + 8 * kMmNumBars;
constexpr int kMmOffTables = kMmOffTmem + 16;
constexpr int kMmCols = 512;

struct MmParams {
  const int32_t* offsets;
  int E, S, N, K, nt, mt;
  int planes_terms;     // 1 or 6
  int chunk;            // blocks of 64 along K between sums in registers
  int split;
  uint32_t idesc;
  int b_mn;
  void* out;
  int64_t out_ld, out_step;
  int out_vec;
  void* gu;
  int64_t gu_ld;
  int gu_vec;
  int M;
  float* parts;
};

// ---- cluster-wide barriers, TMA, MMA of a pair ----

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t addr_in(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) {
  for (int n = 0; n < kWaitLimit; ++n) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred P;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n"
        " selp.u32 %0, 1, 0, P;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One box of a 5-d map (inner, rows, half, expert, plane) to shared memory; `bar` may lie in the
// pair's other CTA.
__device__ __forceinline__ void tma_box(const CUtensorMap* map, uint32_t dst, uint32_t bar, int x, int y,
                                        int half, int expert, int plane) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(half), "r"(expert), "r"(plane)
      : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Descriptor of a stage's operand (128-byte swizzle).  K-major: rows of 64 K, eight-row groups 1024
// bytes apart.  MN-major: rows of 64 M (or N), one for each K; eight K 1024 bytes apart, the next 64 M
// 8192 bytes on.
__device__ __forceinline__ uint64_t mm_desc(uint32_t saddr, bool mn) {
  const uint64_t d = umma_desc_sw128(saddr, 1024);
  return mn ? (d & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(8192 >> 4) << 16) : d;
}

// The tiles of the experts, walked in ascending order.
struct Walk {
  const int32_t *cuts, *prefix;
  int e = 0;
  __device__ __forceinline__ int local(int tile) {
    while (tile >= prefix[e + 1]) ++e;
    return tile - prefix[e];
  }
};

// ---- writing out ----

// 32 rows of 32 values, one row a lane, through the warp's staging to `rows` rows of `cols` valid
// columns: 16 bytes a lane where the output allows it.
template <typename T>
__device__ __forceinline__ void write32(const float (&v)[32], unsigned char* staging, int lane, T* out, int64_t ld,
                                        int rows, int cols, bool vec) {
  constexpr int kChunks = 32 * sizeof(T) / 16;  // of a row: 8 or 4
  constexpr int kEach = 16 / sizeof(T);
  // chunk c of row r at a place where neither writes (lanes: rows) nor reads (lanes: chunks) collide
  const auto place = [](int r, int c) {
    return kChunks == 8 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  };
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    float part[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) part[i] = v[c * kEach + i];
    Pack<T, kEach> p;
    p.set(part);
    p.store(reinterpret_cast<T*>(staging + place(lane, c)));
  }
  __syncwarp();
  if (vec && cols >= 32) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int r = (i * 32 + lane) / kChunks, c = lane % kChunks;
      Pack<T, kEach> p;
      p.load(reinterpret_cast<const T*>(staging + place(r, c)));
      if (r < rows) p.store(out + (int64_t)r * ld + c * kEach);
    }
  } else if (lane < cols) {
    const int c = lane / kEach, i = lane % kEach;
    for (int r = 0; r < min(rows, 32); ++r)
      out[(int64_t)r * ld + lane] = *reinterpret_cast<const T*>(staging + place(r, c) + i * sizeof(T));
  }
  __syncwarp();
}

// WGRAD: the contraction runs over rows.  ACT: gated, or -1.  SUM: parts of K are summed in registers.
template <bool WGRAD, int ACT, bool SUM, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
    k_expert_mm(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, MmParams p) {
  constexpr bool GATED = ACT >= 0;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // (the same in both CTAs)
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kMmOffBars);
  uint64_t* full = bars;                     // first CTA: stage filled in both
  uint64_t* empty = full + kMmStages;        // stage read (commit, to both)
  uint64_t* landed = empty + kMmStages;      // weight gradient: this CTA's copies have landed
  uint64_t* dfull = landed + kMmStages;      // [2] accumulator written (commit, to both)
  uint64_t* dempty = dfull + 2;              // [2] first CTA: accumulator read by both
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMmOffTmem);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int32_t* cuts = reinterpret_cast<int32_t*>(smem + kMmOffTables);
  int32_t* prefix = cuts + p.E + 1;

  if (tid == 0) {
    for (int i = 0; i < kMmStages; ++i) {
      mbar_init(full + i, WGRAD ? 2 : 1);
      mbar_init(empty + i, 1);
      mbar_init(landed + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(dfull + i, 1);
      mbar_init(dempty + i, 2 * kMmEpi);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmWarpMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "n"(kMmCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (warp == kMmWarpTma && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&amap) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&bmap) : "memory");
  }
  wait_for_earlier();
  if (warp == 0) {
    expert_cuts(p.offsets, p.E, p.S, cuts, lane);
    const int nt = p.nt, mt = p.mt, split = p.split;
    expert_prefix(cuts, p.E, prefix, lane, [=](int rows) {
      if (!WGRAD) return (rows + 255) / 256 * nt;
      return split ? (rows + split - 1) / split * mt * nt : mt * nt;
    });
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  let_next_start();
  const uint32_t tmem = *tmem_slot;
  const int tiles = prefix[p.E];
  const int terms = p.planes_terms;
  Walk walk{cuts, prefix};

  // blocks of 64 along a tile's contraction; WGRAD: and its rows [r0, r1)
  const auto k_blocks = [&](int local, int& r0, int& r1) {
    if (!WGRAD) return (p.K + 63) / 64;
    r0 = cuts[walk.e], r1 = cuts[walk.e + 1];
    if (p.split) {
      r0 += local / (p.mt * p.nt) * p.split;
      r1 = min(r1, r0 + p.split);
    }
    return (r1 - r0 + 63) / 64;
  };

  if (warp == kMmWarpTma) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 1;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        const int local = walk.local(tile), e = walk.e;
        const int n = local % p.nt, m = WGRAD ? local / p.nt % p.mt : local / p.nt;
        int r0 = 0, r1 = 0;
        const int blocks = k_blocks(local, r0, r1);
        const int m0 = (WGRAD ? 0 : cuts[e]) + m * 256 + (int)rank * 128;
        const int n0 = GATED ? n * 128 : n * 256 + (int)rank * 128;
        for (int c0 = 0; ok && c0 < blocks; c0 += p.chunk) {
          const int c1 = min(blocks, c0 + p.chunk);
          for (int t = 0; ok && t < terms; ++t) {
            // planes of the six products, small ones first: (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
            const int pa = terms == 1 ? 0 : (0x001012 >> (4 * t)) & 15, pb = terms == 1 ? 0 : (0x010210 >> (4 * t)) & 15;
            for (int kb = c0; kb < c1; ++kb) {
              if (!(ok = mbar_wait_bounded(empty + stage, phase) && !*abort_flag)) break;
              uint64_t* mine = (WGRAD ? landed : full) + stage;
              const uint32_t bar = WGRAD ? smem_u32(mine) : addr_in(smem_u32(mine), 0);
              if (WGRAD || rank == 0) mbar_arrive_expect_tx(mine, WGRAD ? kMmStage : 2 * kMmStage);
              const uint32_t a = sbase + stage * kMmStage, b = a + kMmOperand;
              if (WGRAD) {
                const int k = r0 + kb * 64;
                tma_box(&amap, a, bar, m0, k, 0, 0, pa);
                tma_box(&amap, a + 8192, bar, m0 + 64, k, 0, 0, pa);
                tma_box(&bmap, b, bar, n0, k, 0, 0, pb);
                tma_box(&bmap, b + 8192, bar, n0 + 64, k, 0, 0, pb);
              } else {
                const int half = GATED ? (int)rank : 0;
                tma_box(&amap, a, bar, kb * 64, m0, 0, 0, pa);
                if (p.b_mn) {
                  tma_box(&bmap, b, bar, n0, kb * 64, half, e, pb);
                  tma_box(&bmap, b + 8192, bar, n0 + 64, kb * 64, half, e, pb);
                } else {
                  tma_box(&bmap, b, bar, kb * 64, n0, half, e, pb);
                }
              }
              if (++stage == kMmStages) stage = 0, phase ^= 1;
            }
          }
        }
      }
      if (!ok) *abort_flag = 1;
      // the last copies are read before the CTA leaves: every stage handed back
      for (int i = 0; ok && i < kMmStages; ++i) {
        ok = mbar_wait_bounded(empty + stage, phase);
        if (++stage == kMmStages) stage = 0, phase ^= 1;
      }
    }
  } else if (warp == kMmWarpMma) {
    if (rank == 0 && lane == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, dphase = 1;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        const int local = walk.local(tile);
        int r0 = 0, r1 = p.K;
        const int blocks = k_blocks(local, r0, r1);
        for (int c0 = 0; ok && c0 < blocks; c0 += p.chunk) {
          const int c1 = min(blocks, c0 + p.chunk);
          if (!(ok = wait_cluster(dempty + buf, dphase))) break;
          tc_fence_after();
          uint32_t accumulate = 0;
          for (int t = 0; ok && t < terms; ++t)
            for (int kb = c0; kb < c1; ++kb) {
              if (!(ok = wait_cluster(full + stage, phase) && !*abort_flag)) break;
              tc_fence_after();
              const uint32_t a = sbase + stage * kMmStage;
              uint64_t da = mm_desc(a, WGRAD), db = mm_desc(a + kMmOperand, WGRAD || p.b_mn);
              const int left = r1 - r0 - kb * 64;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k * 16 < left) {
                  mma_pair(tmem + buf * 256, da, db, p.idesc, accumulate);
                  accumulate = 1;
                }
                da += WGRAD ? 2048 >> 4 : 32 >> 4;
                db += WGRAD || p.b_mn ? 2048 >> 4 : 32 >> 4;
              }
              commit_pair(empty + stage);
              if (++stage == kMmStages) stage = 0, phase ^= 1;
            }
          if (ok) commit_pair(dfull + buf);
          if (++buf == 2) buf = 0, dphase ^= 1;
        }
      }
      if (!ok) *abort_flag = 1;
    }
  } else if (warp == kMmWarpRelay) {
    if (WGRAD) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        const int local = walk.local(tile);
        int r0 = 0, r1 = 0;
        const int blocks = k_blocks(local, r0, r1);
        for (int c0 = 0; ok && c0 < blocks; c0 += p.chunk) {
          const int c1 = min(blocks, c0 + p.chunk);
          for (int t = 0; ok && t < terms; ++t)
            for (int kb = c0; kb < c1; ++kb) {
              if (!(ok = mbar_wait_bounded(landed + stage, phase) && !*abort_flag)) break;
              const int left = r1 - r0 - kb * 64;
              if (left < 64) {  // rows of 128 bytes, one for each K, in four boxes of 64
                unsigned char* at = smem + stage * kMmStage;
                for (int i = lane; i < (64 - left) * 32; i += 32)
                  *reinterpret_cast<uint4*>(at + (i >> 3 & 3) * 8192 + (left + (i >> 5)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async();
              }
              __syncwarp();
              if (lane == 0) arrive_cluster(addr_in(smem_u32(full + stage), 0));
              if (++stage == kMmStages) stage = 0, phase ^= 1;
            }
        }
      }
      if (!ok && lane == 0) *abort_flag = 1;
    }
  } else {
    const int quarter = warp & 3, side = warp >> 2;  // lanes 32 * quarter.., half of the columns
    unsigned char* staging = smem + kMmOffStaging + warp * kMmStaging;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    int buf = 0;
    uint32_t dphase = 0;
    bool ok = true;
    const auto release = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(addr_in(smem_u32(dempty + b), 0));
    };
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int local = walk.local(tile), e = walk.e;
      const int n = local % p.nt, m = WGRAD ? local / p.nt % p.mt : local / p.nt;
      int r0 = 0, r1 = 0;
      const int blocks = k_blocks(local, r0, r1);
      // this warp's rows, and how many of them are there
      const int row = (WGRAD ? 0 : cuts[e]) + m * 256 + (int)rank * 128 + quarter * 32;
      const int rows = (WGRAD ? p.M : cuts[e + 1]) - row;
      constexpr int kCols = GATED ? 64 : 128;  // of the output
      const int col = n * (2 * kCols) + side * kCols;
      // accumulator columns of part i of 32: gated, the gate's first and then the up half's
      const auto column = [&](int i) { return GATED ? (i >> 1) * 128 + side * 64 + (i & 1) * 32 : side * 128 + i * 32; };
      float acc[4][32];
      if (SUM) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[i][j] = 0.f;
        for (int c0 = 0; c0 < blocks; c0 += p.chunk) {
          ok = ok && mbar_wait_bounded(dfull + buf, dphase) && !*abort_flag;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v[32];
            __syncwarp();
            tmem_ld32(lanes + buf * 256 + column(i), v);
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[i][j] += ok ? v[j] : __int_as_float(0x7FC00000);
          }
          release(buf);
          if (++buf == 2) buf = 0, dphase ^= 1;
        }
      } else {
        ok = ok && mbar_wait_bounded(dfull + buf, dphase) && !*abort_flag;
        tc_fence_after();
      }
      // a wait that ran out shows as NaN
      const auto get = [&](int i, float (&v)[32]) {
        if (SUM) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = acc[i][j];
        } else {
          __syncwarp();
          tmem_ld32(lanes + buf * 256 + column(i), v);
          if (!ok)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __int_as_float(0x7FC00000);
        }
      };
      if (GATED) {
        T* out = static_cast<T*>(p.out) + (int64_t)row * p.out_ld + col;
        T* gu = static_cast<T*>(p.gu) + (int64_t)row * p.gu_ld + col;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float g[32], u[32];
          const int cols = p.N - col - i * 32;
          get(i, g);
          get(2 + i, u);
          if (!SUM && i == 1) release(buf);
          if (rows <= 0 || cols <= 0) continue;
          if (p.gu != nullptr) {
            write32<T>(g, staging, lane, gu + i * 32, p.gu_ld, rows, cols, p.gu_vec);
            write32<T>(u, staging, lane, gu + p.N + i * 32, p.gu_ld, rows, cols, p.gu_vec);
          }
          float none;
#pragma unroll
          for (int j = 0; j < 32; ++j) u[j] *= activate<ACT, SUM, false>(g[j], none);
          write32<T>(u, staging, lane, out + i * 32, p.out_ld, rows, cols, p.out_vec);
        }
      } else {
        T* out = static_cast<T*>(p.out) + (int64_t)row * p.out_ld + col;
        if (WGRAD) out += e * p.out_step;
        float* part = nullptr;
        if (WGRAD && p.split) part = p.parts + (int64_t)(tile / (p.mt * p.nt)) * p.M * p.N + (int64_t)row * p.N + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[32];
          get(i, v);
          if (!SUM && i == 3) release(buf);
          const int cols = p.N - col - i * 32;
          if (rows <= 0 || cols <= 0) continue;
          if (WGRAD && p.split)
            write32<float>(v, staging, lane, part + i * 32, p.N, rows, cols, p.N % 4 == 0);
          else
            write32<T>(v, staging, lane, out + i * 32, p.out_ld, rows, cols, p.out_vec);
        }
      }
      if (!SUM && ++buf == 2) buf = 0, dphase ^= 1;
    }
    if (!ok && lane == 0) *abort_flag = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kMmWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kMmCols) : "memory");
}

// Sums the parts of each expert's weight gradient, in order.
template <typename T>
__global__ void __launch_bounds__(256)
    k_expert_parts(const float* parts, const int32_t* offsets, int E, int S, int split, int M, int N, T* out, int64_t ld,
                   int64_t step) {
  __shared__ int32_t cuts[kMaxExperts + 1], prefix[kMaxExperts + 1];
  wait_for_earlier();
  if (threadIdx.x < 32) {
    expert_cuts(offsets, E, S, cuts, threadIdx.x);
    expert_prefix(cuts, E, prefix, threadIdx.x, [=](int rows) { return (rows + split - 1) / split; });
  }
  __syncthreads();
  let_next_start();
  const int64_t each = (int64_t)M * N;
  for (int e = blockIdx.y; e < E; e += gridDim.y) {
    const int a = prefix[e], b = prefix[e + 1];
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < each; i += (int64_t)gridDim.x * 256) {
      float v = 0.f;
      for (int k = a; k < b; ++k) v += parts[k * each + i];
      const int64_t r = i / N;
      Pack<T, 1> o;
      const float one[1] = {v};
      o.set(one);
      o.store(out + e * step + r * ld + (i - r * N));
    }
  }
}

// ---- host ----

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<void*> known{nullptr};
  void* f = known.load(std::memory_order_acquire);
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    known.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// Boxes of 64 elements by `box_rows` rows of an operand.  Every base and step is on a 16-byte boundary,
// and the kernel starts boxes at multiples of 64 elements.
bool make_map(CUtensorMap* map, const MmOperand& o, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return false;
  const cuuint64_t dims[5] = {(cuuint64_t)o.inner, (cuuint64_t)o.rows, (cuuint64_t)o.halves, (cuuint64_t)o.experts,
                              (cuuint64_t)o.planes};
  // (the step of an axis of one is never used, but has to be a step)
  const auto step = [](int64_t elements, bool used) { return (cuuint64_t)(used ? elements * 2 : 16); };
  const cuuint64_t steps[4] = {step(o.ld, o.rows > 1), step(o.half_step, o.halves > 1), step(o.expert_step, o.experts > 1),
                               step(o.plane_step, o.planes > 1)};
  const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, 1, 1, 1}, ones[5] = {1, 1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<__nv_bfloat16*>(o.p), dims, steps, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr uint32_t mm_idesc(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10)  // D fp32, A and B bf16
         | (a_mn ? 1u << 15 : 0) | (b_mn ? 1u << 16 : 0) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
}

template <bool WGRAD, int ACT, bool SUM, typename T>
cudaError_t launch_mm(const MmArgs& a, MmParams p, int64_t tiles_most, cudaStream_t s) {
  constexpr auto kern = k_expert_mm<WGRAD, ACT, SUM, T>;
  cudaError_t e = prepare_kernel<kern>();
  if (e != cudaSuccess) return e;
  CUtensorMap amap, bmap;
  if (!make_map(&amap, a.a, WGRAD ? 64 : 128) || !make_map(&bmap, a.b, WGRAD || a.b_mn ? 64 : 128))
    return cudaErrorInvalidValue;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(device_sms() / 2, tiles_most));
  const int smem = kMmOffTables + 2 * (p.E + 1) * 4 + 1024;
  return launch_early(kern, (unsigned)(2 * pairs), kMmThreads, smem, s, amap, bmap, p);
}

MmParams params_of(const MmArgs& a) {
  MmParams p{};
  const int elem = a.out_bf16 ? 2 : 4;
  p.offsets = a.offsets, p.E = a.E, p.S = a.S, p.N = a.N, p.K = a.K, p.M = a.M;
  p.planes_terms = a.f32 ? 6 : 1;
  p.out = a.out, p.out_ld = a.out_ld, p.out_step = a.out_step;
  p.out_vec = rows_on(a.out, a.out_ld, elem, 16) && a.out_step * elem % 16 == 0;
  p.gu = a.gu, p.gu_ld = a.gu_ld;
  p.gu_vec = rows_on(a.gu, a.gu_ld, elem, 16) && (int64_t)a.N * elem % 16 == 0;
  p.split = a.split, p.parts = a.parts;
  return p;
}

}  // namespace

cudaError_t launch_expert_mm_rows(const MmArgs& a, cudaStream_t s) {
  if (a.S == 0) return cudaSuccess;
  MmParams p = params_of(a);
  const bool gated = a.act >= 0;
  p.nt = (a.N + (gated ? 127 : 255)) / (gated ? 128 : 256), p.mt = 1;
  p.b_mn = a.b_mn;
  p.idesc = mm_idesc(false, a.b_mn);
  p.chunk = a.f32 ? 4 : 1 << 20;
  const int64_t most = ((int64_t)a.S / 256 + std::min(a.E, a.S)) * p.nt;
  using H = __nv_bfloat16;
  if (a.f32) switch (a.act) {
      case EMB_ACT_SILU: return launch_mm<false, EMB_ACT_SILU, true, float>(a, p, most, s);
      case EMB_ACT_GELU: return launch_mm<false, EMB_ACT_GELU, true, float>(a, p, most, s);
      case EMB_ACT_RELU: return launch_mm<false, EMB_ACT_RELU, true, float>(a, p, most, s);
      case EMB_ACT_SIGMOID: return launch_mm<false, EMB_ACT_SIGMOID, true, float>(a, p, most, s);
      default: return launch_mm<false, -1, true, float>(a, p, most, s);
    }
  switch (a.act) {
    case EMB_ACT_SILU: return launch_mm<false, EMB_ACT_SILU, false, H>(a, p, most, s);
    case EMB_ACT_GELU: return launch_mm<false, EMB_ACT_GELU, false, H>(a, p, most, s);
    case EMB_ACT_RELU: return launch_mm<false, EMB_ACT_RELU, false, H>(a, p, most, s);
    case EMB_ACT_SIGMOID: return launch_mm<false, EMB_ACT_SIGMOID, false, H>(a, p, most, s);
    default: return launch_mm<false, -1, false, H>(a, p, most, s);
  }
}

cudaError_t launch_expert_mm_wgrad(const MmArgs& a, cudaStream_t s) {
  MmParams p = params_of(a);
  p.nt = (a.N + 255) / 256, p.mt = (a.M + 255) / 256;
  p.idesc = mm_idesc(true, true);
  p.chunk = a.f32 ? 4 : 8;
  if (a.S > 0) {
    const int64_t parts = a.split ? (int64_t)a.S / a.split + std::min(a.E, a.S) : a.E;
    const cudaError_t e = a.out_bf16 ? launch_mm<true, -1, true, __nv_bfloat16>(a, p, parts * p.mt * p.nt, s)
                                     : launch_mm<true, -1, true, float>(a, p, parts * p.mt * p.nt, s);
    if (e != cudaSuccess || !a.split) return e;
  }
  // (no rows: no parts, and zeros)
  const int split = a.split ? a.split : 64;
  const int64_t each = (int64_t)a.M * a.N;
  const unsigned gx = (unsigned)std::min<int64_t>((each + 255) / 256, std::max(1, device_sms() * 8 / a.E));
  const auto sum = [&](auto* out) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(gx, (unsigned)a.E), cfg.blockDim = dim3(256), cfg.stream = s, cfg.attrs = &attr, cfg.numAttrs = 1;
    using T = std::remove_pointer_t<decltype(out)>;
    return cudaLaunchKernelEx(&cfg, k_expert_parts<T>, (const float*)a.parts, a.offsets, a.E, a.S, split, a.M, a.N, out,
                              a.out_ld, a.out_step);
  };
  return a.out_bf16 ? sum(static_cast<__nv_bfloat16*>(a.out)) : sum(static_cast<float*>(a.out));
}

}  // namespace emb
