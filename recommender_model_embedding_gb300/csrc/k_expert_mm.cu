// The experts' matrix products on the 5th-generation tensor cores, rows grouped by expert.
//
//   rows product      C[r] = A[r] B_e^T, r in expert e's rows  (out = x W^T, dx = dout W; gated: the
//                     gate's and the up half's columns side by side, h = act(g) u in the epilogue)
//   weight gradient   C_e = sum over e's rows r of A[r]^T B[r]   (dW = dout^T x)
//
// Both are one kernel: a pair of CTAs (a cluster on two SMs) computes tiles of 256 x 256, each CTA
// holding 128 rows of the accumulator in its tensor memory, with tcgen05.mma.cta_group::2 (M = 256,
// N = 256, K = 16) issued by one lane of the pair's first CTA.  Per 64 of K each CTA brings 128 x
// 64 of A and of B by TMA (16 KB each, 128-byte swizzle) into a ring of six stages (five beyond some 200
// experts, for their tables; with four 524288 x 512 x 2048 took 741 us, with five 706, with six 665); the pair
// reads B from both.  A tile alone in one CTA (128 x 256) would write 48 KB and read 48 KB of shared memory
// for the same arithmetic as 32 KB and 32 KB here, over what an SM's shared memory moves in
// that time.  Operands may run along either axis (the descriptors take K-major and
// MN-major tiles), so neither direction of the pass and neither layout of the weights moves data.
//
// The grid stays resident and walks the tiles of all experts in turn (columns fastest, so tiles that
// run together share rows of A and the expert's weights in L2); which tiles there are is worked out
// from the experts' offsets on the device, so the host never waits for them.  Accumulators
// alternate between the two halves of tensor memory: sixteen warps write one tile out while the next
// is computed.  Rows of a tile behind its expert's last are computed and not stored.  Where the
// contraction runs over rows (weight gradient), a stage's rows behind the expert's last are set to
// zero in both operands before the tensor core reads them (they may hold anything, NaN too).
//
// fp32: each operand is split into three bf16 planes, v = v0 + v1 + v2 (eight significant bits each),
// and the six products a_i b_j with i + j <= 2 are added; what is left out is below 2^-24 of the product.
// The three planes of 64 K lie in the ring side by side, so each is brought once for its six products (with three
// products, for an fp32 gradient of bf16 weights, such threes hold the copies up: 2.2 ms for 524288 x 2048 x 512
// instead of 1.9, so there, and with two, each product has a stage).  The tensor core adds in fp32 but does not round
// to nearest, so an error would grow with the length of the sum: fp32 results are therefore summed over parts of K in
// registers, the small products' apart from the large one's (8192 rows of bf16: 9.1e-6 off in the 2-norm in one sum,
// 4.8e-7 in parts of 512).  bf16 results take the accumulator as it is (its error, below 2^-12 at K = 65536, is
// inside bf16's rounding).
//
// Measured on bf16 rows of 64 experts: 524288 x 512 through 512 -> 2048 outputs gated, h alone 0.60 ms (1.8 PFLOP/s,
// the products alone, nothing stored, 0.57), with g and u too 0.81 ms; 1024 -> 512 0.34 ms; a linear layer's dx 2048
// -> 512 0.69 ms; dW 2048 x 512 0.69 ms (1.6 PFLOP/s).  Those are a cool chip's: after seconds of such work the power
// limit takes the clock from 2.07 to 1.5 GHz, and gated takes 0.67 and 0.95 ms, 1024 -> 512 0.38.  fp32, 65536 x 512
// through 1024 outputs: 0.29 ms.  With all operands in shared memory a stage takes the tensor core 512 cycles and the
// loop 520; what is over that is waiting for copies while stores share the way to memory.
#include <algorithm>
#include <atomic>

#include "expert_mm.cuh"
#include "interact_common.cuh"
#include "tc_common.cuh"

namespace emb {

constexpr int kMmEpi = 16;                         // warps that write tiles out
constexpr int kMmWarpTma = kMmEpi, kMmWarpMma = kMmEpi + 1, kMmWarpRelay = kMmEpi + 2;
constexpr int kMmThreads = 32 * (kMmEpi + 3);
constexpr int kMmMaxStages = 8;
constexpr int kMmOperand = 128 * 128;              // bytes of an operand's stage: 128 x 64 bf16
// bytes of a stage: both operands', B's as wide as the tile
__host__ __device__ constexpr int mm_stage(int tile_n) { return kMmOperand + tile_n * 64; }
constexpr int kMmPart = 32 * 64;                   // bytes that a warp writes at once: 32 rows of 64
// shared memory: the warps' parts, barriers, the tensor memory's address, tables of E + 1 rows and tiles, stages
constexpr int kMmNumBars = 3 * kMmMaxStages + 4;
constexpr int kMmOffBars = kMmEpi * kMmPart;
constexpr int kMmOffTmem = kMmOffBars + 8 * kMmNumBars;
constexpr int kMmOffTables = kMmOffTmem + 16;
constexpr int kMmMost = 232448;                    // bytes that a CTA can have
__host__ __device__ constexpr int mm_off_stages(int E) { return (kMmOffTables + 8 * (E + 1) + 1023) / 1024 * 1024; }
constexpr int mm_smem(int E, int stages, int tile_n) { return mm_off_stages(E) + stages * mm_stage(tile_n) + 1024; }  // (+ to align it)
constexpr int kMmCols = 512;

struct MmParams {
  const int32_t* offsets;
  int E, S, N, K, nt, mt;
  int terms;            // products of planes: 1, 2, 3 or 6
  uint32_t terms_a, terms_b;  // planes of each, four bits
  int tile_n;           // columns of a tile: 256 or 128
  int stages;
  int chunk;            // blocks of 64 along K between sums in registers
  int split;
  int turned;           // weight gradient: out (and parts) hold rows of M, one for each column
  int beside;           // starts beside the launch before it, and waits for that at its own end
  uint32_t idesc;
  int b_mn;
  int b_each;           // rows product: every expert has a matrix of its own
  void* out;
  int64_t out_ld, out_step;
  void* gu;
  int64_t gu_ld;
  int out_map, gu_map;  // whether the kernel has maps of them
  int M;
  float* parts;
};

// ---- cluster-wide barriers, TMA, MMA of a pair ----
//
// Every wait has a limit.  A role whose wait runs out does no more work, so the others' run out too, each once, and
// all meet at the kernel's end; the tiles concerned are written as NaN.

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One lane of the warp.  The warps that issue copies and products run their loops whole, and this lane the
// instruction: so their operands stay in the warp's uniform registers, which the instructions take (with a
// single lane in the loop they were moved there one by one, 587 cycles for a stage's products instead of 512).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ uint32_t addr_in(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// The same without release: for accumulators read (their loads have returned), where a release would hold the warp
// until its stores of the last tile have reached memory.
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
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

__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %6, 0;\n mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
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

// A warp's output: parts of 32 rows of 64 bytes (one row a lane: 32 bf16 or 16 fp32 values), staged in
// its buffer.  Full parts of an output on 16-byte boundaries leave as one TMA copy each, which takes the
// store out of the warp's hands (and out of the load-store pipe, which the tensor core's operands
// share); parts at an expert's end go row by row, those at the last columns element by element.  Chunk c of row r
// lies at c ^ (r / 2 % 4), the 64-byte swizzle, so that neither the lanes' writes nor reads collide.
struct Writer {
  unsigned char* staging;
  int lane;
  __device__ __forceinline__ static int place(int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); }

  // map: of `out`'s matrices, or NULL; x, y, z: the part's place in it
  template <typename T>
  __device__ __forceinline__ void part(const float* v, T* out, int64_t ld, int rows, int cols, const CUtensorMap* map, int x,
                                       int y, int z) {
    constexpr int kEach = 16 / sizeof(T), kCols = 4 * kEach;
    unsigned char* at = staging;
    // the last copy has read the buffer
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float e[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) e[i] = v[c * kEach + i];
      Pack<T, kEach> p;
      p.set(e);
      p.store(reinterpret_cast<T*>(at + place(lane, c)));
    }
    const bool whole = map != nullptr && rows >= 32 && cols >= kCols;
    if (whole) fence_proxy_async();
    __syncwarp();
    if (whole) {
      if (lane == 0)
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n"
                     "cp.async.bulk.commit_group;" ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(at))
                     : "memory");
      return;
    }
    if (map != nullptr && cols >= kCols) {
      const int c = lane & 3;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        Pack<T, kEach> p;
        p.load(reinterpret_cast<const T*>(at + place(r, c)));
        if (r < rows) p.store(out + (int64_t)r * ld + c * kEach);
      }
      return;
    }
    const int col = lane % kCols, c = col / kEach, i = col % kEach;
    if (col < cols)
      for (int r = lane / kCols; r < min(rows, 32); r += 32 / kCols)
        out[(int64_t)r * ld + col] = *reinterpret_cast<const T*>(at + place(r, c) + i * sizeof(T));
  }

  // 32 values a row
  template <typename T>
  __device__ __forceinline__ void write(const float (&v)[32], T* out, int64_t ld, int rows, int cols, const CUtensorMap* map,
                                        int x, int y, int z) {
    part<T>(v, out, ld, rows, cols, map, x, y, z);
    if constexpr (sizeof(T) == 4)
      if (cols > 16) part<T>(v + 16, out + 16, ld, rows, cols - 16, map, x + 16, y, z);
  }

  __device__ __forceinline__ void finish() {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// WGRAD: the contraction runs over rows.  ACT: gated, or -1.  SUM: parts of K are summed in registers.  SIX: fp32
// operands, six products of their planes.
template <bool WGRAD, int ACT, bool SUM, bool SIX, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMmThreads, 1)
    k_expert_mm(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap gmap, MmParams p) {
  constexpr bool GATED = ACT >= 0;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);  // (the same in both CTAs)
  const uint32_t sbase = smem_u32(smem) + mm_off_stages(p.E);  // the stages'
  const int stages = p.stages;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kMmOffBars);
  uint64_t* full = bars;                     // first CTA: stage filled in both
  uint64_t* empty = full + kMmMaxStages;        // stage read (commit, to both)
  uint64_t* landed = empty + kMmMaxStages;      // weight gradient: this CTA's copies have landed
  uint64_t* dfull = landed + kMmMaxStages;      // [2] accumulator written (commit, to both)
  uint64_t* dempty = dfull + 2;              // [2] first CTA: accumulator read by both
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMmOffTmem);
  int32_t* cuts = reinterpret_cast<int32_t*>(smem + kMmOffTables);
  int32_t* prefix = cuts + p.E + 1;

  if (tid == 0) {
    for (int i = 0; i < kMmMaxStages; ++i) {
      mbar_init(full + i, WGRAD ? 2 : 1);
      mbar_init(empty + i, 1);
      mbar_init(landed + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(dfull + i, 1);
      mbar_init(dempty + i, 2 * kMmEpi);
    }
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
  // (every CTA of the launch before it has passed its own wait: what came before that is done)
  if (!p.beside) wait_for_earlier();
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
  const int terms = SIX ? 6 : p.terms, tile_n = p.tile_n, slots = terms == 6 ? 3 : terms, stage_bytes = mm_stage(tile_n);  // slots: stages of 64 K
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
    {
      const bool one = elect_one();
      const uint32_t full0 = addr_in(smem_u32(full), 0);  // of the pair's first CTA
      int stage = 0;
      uint32_t phase = 1;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        const int local = walk.local(tile), e = walk.e;
        const int n = local % p.nt, m = WGRAD ? local / p.nt % p.mt : local / p.nt;
        int r0 = 0, r1 = 0;
        const int blocks = k_blocks(local, r0, r1);
        const int m0 = (WGRAD ? 0 : cuts[e]) + m * 256 + (int)rank * 128;
        const int n0 = GATED ? n * (tile_n / 2) : n * tile_n + (int)rank * (tile_n / 2);
        for (int c0 = 0; ok && c0 < blocks; c0 += p.chunk) {
          const int c1 = min(blocks, c0 + p.chunk);
          // six products: the planes of each 64 K side by side; two or three: a part's first products, then its
          // second ..
          const int outer = terms == 6 ? c1 - c0 : slots, inner = terms == 6 ? slots : c1 - c0;
          for (int u = 0; ok && u < outer; ++u)
            for (int v = 0; v < inner; ++v) {
              const int i = terms == 6 ? v : u, kb = c0 + (terms == 6 ? u : v);
              if (!(ok = mbar_wait_bounded(empty + stage, phase))) break;
              const int pa = terms == 6 ? 2 - i : p.terms_a >> (4 * i) & 15, pb = terms == 6 ? 2 - i : p.terms_b >> (4 * i) & 15;
              uint32_t bar;
              if (WGRAD && r1 - r0 - kb * 64 < 64) {  // by way of the warp that clears rows
                bar = smem_u32(landed + stage);
                if (one) mbar_arrive_expect_tx(landed + stage, stage_bytes);
              } else {
                bar = full0 + stage * 8;
                if (rank == 0 && one) {
                  mbar_arrive_expect_tx(full + stage, 2 * stage_bytes);
                  if (WGRAD) mbar_arrive(full + stage);
                }
              }
              const uint32_t a = sbase + stage * stage_bytes, b = a + kMmOperand;
              if (!one) {
              } else if (WGRAD) {
                const int k = r0 + kb * 64;
                tma_box(&amap, a, bar, m0, k, 0, 0, pa);
                tma_box(&amap, a + 8192, bar, m0 + 64, k, 0, 0, pa);
                tma_box(&bmap, b, bar, n0, k, 0, 0, pb);
                if (tile_n > 128) tma_box(&bmap, b + 8192, bar, n0 + 64, k, 0, 0, pb);
              } else {
                const int half = GATED ? (int)rank : 0, of = p.b_each ? e : 0;
                tma_box(&amap, a, bar, kb * 64, m0, 0, 0, pa);
                if (p.b_mn) {
                  tma_box(&bmap, b, bar, n0, kb * 64, half, of, pb);
                  if (tile_n > 128) tma_box(&bmap, b + 8192, bar, n0 + 64, kb * 64, half, of, pb);
                } else {
                  tma_box(&bmap, b, bar, kb * 64, n0, half, of, pb);
                }
              }
              if (++stage == stages) stage = 0, phase ^= 1;
            }
        }
      }
      // the last copies are read before the CTA leaves: every stage handed back
      for (int i = 0; ok && i < stages; ++i) {
        ok = mbar_wait_bounded(empty + stage, phase);
        if (++stage == stages) stage = 0, phase ^= 1;
      }
    }
  } else if (warp == kMmWarpMma) {
    if (rank == 0) {
      // One lane feeds the tensor core, which takes 512 cycles for a stage: the loop keeps to what has to be in it
      // (addresses of descriptors and barriers are steps from the first stage's).
      const uint64_t desc_a = mm_desc(sbase, WGRAD), desc_b = mm_desc(sbase + kMmOperand, WGRAD || p.b_mn);
      const uint32_t step_a = WGRAD ? 2048 >> 4 : 32 >> 4, step_b = WGRAD || p.b_mn ? 2048 >> 4 : 32 >> 4;
      const uint32_t hi_a = (uint32_t)(desc_a >> 32), hi_b = (uint32_t)(desc_b >> 32), idesc = p.idesc;
      const uint32_t stages = p.stages, stage_step = stage_bytes >> 4, terms_a = p.terms_a, terms_b = p.terms_b;
      const uint32_t empty0 = smem_u32(empty);
      const bool one = elect_one();
      const int chunk = p.chunk, K = p.K;
      int buf = 0;
      uint32_t stage = 0, phase = 0, dphase = 1;
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        int length = K;  // of the contraction
        if (WGRAD) {
          int r0 = 0, r1 = 0;
          k_blocks(walk.local(tile), r0, r1);
          length = r1 - r0;
        }
        for (int done = 0; ok && done < length; done += chunk * 64) {
          const int part = min(length - done, chunk * 64);
          if (!(ok = mbar_wait_bounded(dempty + buf, dphase))) break;
          tc_fence_after();
          const auto products = [&](int left, uint32_t sa, uint32_t sb, uint32_t d, uint32_t accumulate) {
            const uint32_t lo_a = (uint32_t)desc_a + sa * stage_step, lo_b = (uint32_t)desc_b + sb * stage_step;
            if (one) {
              mma_pair(d, lo_a, hi_a, lo_b, hi_b, idesc, accumulate);
              if (left > 48) {
#pragma unroll
                for (int k = 1; k < 4; ++k) mma_pair(d, lo_a + k * step_a, hi_a, lo_b + k * step_b, hi_b, idesc, 1);
              } else {
                for (int k = 1; k * 16 < left; ++k) mma_pair(d, lo_a + k * step_a, hi_a, lo_b + k * step_b, hi_b, idesc, 1);
              }
            }
          };
          // (rows cleared by the other CTA's threads want an acquire of the cluster's scope; copies do not)
          const auto come = [&](int left, uint32_t at, uint32_t parity) {
            return WGRAD && left < 64 ? wait_cluster(full + at, parity) : mbar_wait_bounded(full + at, parity);
          };
          const auto done_with_stage = [&] {
            if (one) commit_pair(empty0 + stage * 8);
            if (++stage == stages) stage = 0, phase ^= 1;
          };
          if constexpr (!SIX) {  // a stage for each product
            uint32_t accumulate = 0;
            for (int i = 0; ok && i < slots; ++i)
              for (int left = part; left > 0; left -= 64) {
                if (!(ok = come(left, stage, phase))) break;
                tc_fence_after();
                products(left, stage, stage, tmem + buf * 256, accumulate);
                accumulate = 1;
                done_with_stage();
              }
            if (ok && one) commit_pair(smem_u32(dfull + buf));
            buf ^= 1;
            dphase ^= buf ^ 1;
          } else {
            // A stage for each of both operands' planes, 2, 1, 0 in turn, and six products of them: the five small ones
            // into one half of the tensor memory, the large one into the other.
            const auto three = [&](int left, uint32_t at, uint32_t parity) {
              bool all = true;
              for (int i = 0; all && i < 3; ++i) {
                all = come(left, at, parity);
                if (++at == stages) at = 0, parity ^= 1;
              }
              return all;
            };
            bool ready = false;
            for (int left = part; ok && left > 0; left -= 64) {
              if (!ready && !(ok = three(left, stage, phase))) break;
              tc_fence_after();
              ready = false;
              const uint32_t first = stage;
              for (int t = 0; ok && t < 6; ++t) {
                uint32_t sa = first + 2 - (terms_a >> (4 * t) & 15), sb = first + 2 - (terms_b >> (4 * t) & 15);
                if (sa >= stages) sa -= stages;
                if (sb >= stages) sb -= stages;
                if (t == 5) {
                  // (the large sum's half, which is read first of a part)
                  if (left == part && !(ok = mbar_wait_bounded(dempty + 1, dphase))) break;
                  if (left > 64 && stages >= 6) {
                    // the next copies, waited for while the tensor core still has work (their stages are others)
                    uint32_t next = stage + 1, parity = phase;
                    if (next >= stages) next -= stages, parity ^= 1;
                    if (!(ok = ready = three(left - 64, next, parity))) break;
                  }
                  tc_fence_after();
                }
                products(left, sa, sb, t < 5 ? tmem + 256 : tmem, left < part || (t > 0 && t < 5));
                if (t == 2 || t >= 4) done_with_stage();  // (planes 2 are done with first, then 1)
              }
            }
            if (ok && one) commit_pair(smem_u32(dfull));
            dphase ^= 1;
          }
        }
      }
    }
  } else if (warp == kMmWarpRelay) {
    if (WGRAD) {
      int stage = 0;
      uint32_t phases = 0;  // of `landed`, a bit a stage
      bool ok = true;
      for (int tile = pair; ok && tile < tiles; tile += pairs) {
        const int local = walk.local(tile);
        int r0 = 0, r1 = 0;
        const int blocks = k_blocks(local, r0, r1);
        const int left = r1 - r0 - (blocks - 1) * 64;  // rows of the last block
        for (int c0 = 0; ok && c0 < blocks; c0 += p.chunk) {
          const int c1 = min(blocks, c0 + p.chunk);
          const bool clear = c1 == blocks && left < 64;
          if (terms == 6) stage = (stage + (c1 - c0 - 1) * slots) % stages;
          for (int i = 0; ok && i < slots; ++i) {
            if (terms != 6) stage = (stage + c1 - c0 - 1) % stages;  // the part's last block
            if (!clear) {
              stage = stage + 1 == stages ? 0 : stage + 1;
              continue;
            }
            if (!(ok = mbar_wait_bounded(landed + stage, phases >> stage & 1))) break;
            phases ^= 1u << stage;
            // rows of 128 bytes, one for each K, in boxes of 64: two of A, one or two of B
            unsigned char* at = smem + mm_off_stages(p.E) + stage * stage_bytes;
            const int boxes = tile_n > 128 ? 4 : 3;
            for (int q = lane; q < (64 - left) * 32; q += 32)
              if ((q >> 3 & 3) < boxes)
                *reinterpret_cast<uint4*>(at + (q >> 3 & 3) * 8192 + (left + (q >> 5)) * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) arrive_cluster(addr_in(smem_u32(full + stage), 0));
            stage = stage + 1 == stages ? 0 : stage + 1;
          }
        }
      }
    }
  } else {
    const int quarter = warp & 3, side = warp >> 2;  // lanes 32 * quarter.., parts `side` and `side` + 4 of 32 columns
    Writer to{smem + warp * kMmPart, lane};
    const CUtensorMap *om = p.out_map ? &omap : nullptr, *gm = p.gu_map ? &gmap : nullptr;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    // accumulator columns of the two parts: gated, the gate's and the up half's of the same outputs
    const uint32_t at0 = side * 32, at1 = GATED ? tile_n / 2 + side * 32 : 128 + side * 32;
    const bool has0 = !GATED || side * 32 < tile_n / 2, has1 = GATED ? has0 : tile_n > 128;
    int buf = 0;
    uint32_t dphase = 0;
    bool ok = true;
    const auto release = [&](int b) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster_relaxed(addr_in(smem_u32(dempty + b), 0));
    };
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int local = walk.local(tile), e = walk.e;
      const int n = local % p.nt, m = WGRAD ? local / p.nt % p.mt : local / p.nt;
      int r0 = 0, r1 = 0;
      const int blocks = k_blocks(local, r0, r1);
      // this warp's rows, and how many of them are there
      const int row = (WGRAD ? 0 : cuts[e]) + m * 256 + (int)rank * 128 + quarter * 32;
      const int rows = (WGRAD ? p.M : cuts[e + 1]) - row;
      const int col = n * (GATED ? tile_n / 2 : tile_n) + side * 32, cols = p.N - col;
      float v0[32], v1[32];
      if (SUM) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v0[j] = v1[j] = 0.f;
        for (int c0 = 0; c0 < blocks; c0 += p.chunk) {
          ok = ok && mbar_wait_bounded(dfull + buf, dphase);
          tc_fence_after();
          __syncwarp();
          // six products: the large one's sum from the lower half, then the small ones' from the upper
#pragma unroll
          for (int half = 0; half <= (int)SIX; ++half) {
            const uint32_t from = lanes + (SIX ? half : buf) * 256;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (!(i < 2 ? has0 : has1)) continue;
              float v[16];
              tmem_ld16(from + (i < 2 ? at0 : at1) + (i & 1) * 16, v);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float& sum = (i < 2 ? v0 : v1)[(i & 1) * 16 + j];
                sum = half ? with_small(sum, v[j]) : sum + v[j];
              }
            }
            release(SIX ? 1 - half : buf);
          }
          if (SIX) dphase ^= 1;
          else if (++buf == 2) buf = 0, dphase ^= 1;
        }
      } else {
        ok = ok && mbar_wait_bounded(dfull + buf, dphase);
        tc_fence_after();
        __syncwarp();
        if (has0) tmem_ld32(lanes + buf * 256 + at0, v0);
        if (has1) tmem_ld32(lanes + buf * 256 + at1, v1);
        release(buf);
        if (++buf == 2) buf = 0, dphase ^= 1;
      }
      if (!ok)  // a wait that ran out shows as NaN
#pragma unroll
        for (int j = 0; j < 32; ++j) v0[j] = v1[j] = __int_as_float(0x7FC00000);
      if (rows <= 0 || cols <= 0) continue;
      if (GATED) {
        if (!has0) continue;
        if (p.gu != nullptr) {
          T* gu = static_cast<T*>(p.gu) + (int64_t)row * p.gu_ld + col;
          to.write<T>(v0, gu, p.gu_ld, rows, cols, gm, col, row, 0);
          to.write<T>(v1, gu + p.N, p.gu_ld, rows, cols, gm, p.N + col, row, 0);
        }
        float none;
#pragma unroll
        for (int j = 0; j < 32; ++j) v1[j] *= activate<ACT, SUM, false>(v0[j], none);
        to.write<T>(v1, static_cast<T*>(p.out) + (int64_t)row * p.out_ld + col, p.out_ld, rows, cols, om, col, row, 0);
      } else if (WGRAD && p.turned) {
        // lanes are rows, so a column's 32 values are adjacent: stored as they are
        float* part = p.split ? p.parts + ((int64_t)(tile / (p.mt * p.nt)) * p.N + col) * p.M + row + lane : nullptr;
        T* out = static_cast<T*>(p.out) + e * p.out_step + (int64_t)col * p.out_ld + row + lane;
        if (lane < rows)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (i == 0 || has1)
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const int c = i * 128 + j;
                if (c >= cols) continue;
                const float v[1] = {(i ? v1 : v0)[j]};
                if (p.split) {
                  part[(int64_t)c * p.M] = v[0];
                } else {
                  Pack<T, 1> o;
                  o.set(v);
                  o.store(out + (int64_t)c * p.out_ld);
                }
              }
      } else if (WGRAD && p.split) {
        const int z = tile / (p.mt * p.nt);
        float* part = p.parts + ((int64_t)z * p.M + row) * p.N + col;
        to.write<float>(v0, part, p.N, rows, cols, om, col, row, z);
        if (has1 && cols > 128) to.write<float>(v1, part + 128, p.N, rows, cols - 128, om, col + 128, row, z);
      } else {
        T* out = static_cast<T*>(p.out) + (WGRAD ? e * p.out_step : 0) + (int64_t)row * p.out_ld + col;
        const int z = WGRAD ? e : 0;
        to.write<T>(v0, out, p.out_ld, rows, cols, om, col, row, z);
        if (has1 && cols > 128) to.write<T>(v1, out + 128, p.out_ld, rows, cols - 128, om, col + 128, row, z);
      }
    }
    to.finish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kMmWarpMma)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kMmCols) : "memory");
  if (p.beside) wait_for_earlier();
}

// Sums the parts of each expert's weight gradient, in a fixed order: a thread for EPU elements, or where parts are many
// eight, of which each takes an eighth of them, added up in shared memory.
template <typename T, int EPU, int SHARES>
__global__ void __launch_bounds__(256)
    k_expert_parts(const float* parts, const int32_t* offsets, int E, int S, int split, int64_t each, FastDiv pieces, T* out,
                   int64_t ld, int64_t step) {
  __shared__ int32_t cuts[kMaxExperts + 1], prefix[kMaxExperts + 1];
  constexpr int SLOTS = 256 / SHARES;
  __shared__ float sums[SHARES][SHARES > 1 ? SLOTS : 1][EPU + 1];
  wait_for_earlier();
  let_next_start();
  if (threadIdx.x < 32) {
    expert_cuts(offsets, E, S, cuts, threadIdx.x);
    expert_prefix(cuts, E, prefix, threadIdx.x, [=](int rows) { return (rows + split - 1) / split; });
  }
  __syncthreads();
  const int e = blockIdx.y, a = prefix[e], n = prefix[e + 1] - a, slot = threadIdx.x % SLOTS, share = threadIdx.x / SLOTS;
  const int k0 = (int)((int64_t)n * share / SHARES), k1 = (int)((int64_t)n * (share + 1) / SHARES);
  const uint32_t i = blockIdx.x * SLOTS + slot;  // of the matrix's pieces of EPU elements
  const bool there = (int64_t)i * EPU < each;
  float v[EPU] = {};
  if (there) {
    const float* from = parts + (a + k0) * each + (int64_t)i * EPU;
#pragma unroll 4
    for (int k = k0; k < k1; ++k, from += each) {
      Pack<float, EPU> q;
      float x[EPU];
      q.load(from);
      q.get(x);
#pragma unroll
      for (int j = 0; j < EPU; ++j) v[j] += x[j];
    }
  }
  if constexpr (SHARES > 1) {
#pragma unroll
    for (int j = 0; j < EPU; ++j) sums[share][slot][j] = v[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < EPU; ++j) {
      v[j] = 0.f;
#pragma unroll
      for (int k = 0; k < SHARES; ++k) v[j] += sums[k][slot][j];
    }
  }
  if (share || !there) return;
  const uint32_t r = pieces.div(i), c = i - r * pieces.d;
  Pack<T, EPU> o;
  o.set(v);
  o.store(out + e * step + (int64_t)r * ld + c * EPU);
}

// ---- host ----

// Pairs of CTAs that run at once.
int64_t mm_pairs() { return std::max(1, device_sms() / 2); }

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

uint32_t mm_idesc(bool a_mn, bool b_mn, int tile_n) {
  return (1u << 4) | (1u << 7) | (1u << 10)  // D fp32, A and B bf16
         | (a_mn ? 1u << 15 : 0) | (b_mn ? 1u << 16 : 0) | ((uint32_t)(tile_n >> 3) << 17) | ((256u >> 4) << 24);
}

// Parts (32 rows of 64 bytes) of `count` output matrices, where they lie on 16-byte boundaries.
bool make_out_map(CUtensorMap* map, void* p, int64_t rows, int64_t cols, int64_t ld, int64_t count, int64_t step, bool bf16) {
  const EncodeTiled encode = encode_tiled();
  const int elem = bf16 ? 2 : 4;
  if (encode == nullptr || p == nullptr || reinterpret_cast<uintptr_t>(p) % 16 || (rows > 1 && ld * elem % 16) ||
      (count > 1 && step * elem % 16))
    return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  const cuuint64_t steps[2] = {(cuuint64_t)(rows > 1 ? ld * elem : 16), (cuuint64_t)(count > 1 ? step * elem : 16)};
  const cuuint32_t box[3] = {64u / (cuuint32_t)elem, 32, 1}, ones[3] = {1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, steps, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool WGRAD, int ACT, bool SUM, bool SIX, typename T>
cudaError_t launch_mm(const MmArgs& a, MmParams p, int64_t tiles_most, cudaStream_t s) {
  constexpr auto kern = k_expert_mm<WGRAD, ACT, SUM, SIX, T>;
  cudaError_t e = prepare_kernel<kern>();
  if (e != cudaSuccess) return e;
  CUtensorMap amap, bmap, omap, gmap;
  if (!make_map(&amap, a.a, WGRAD ? 64 : 128) || !make_map(&bmap, a.b, WGRAD || a.b_mn ? 64 : p.tile_n / 2))
    return cudaErrorInvalidValue;
  if (WGRAD && a.turned)
    p.out_map = 0;
  else if (WGRAD && a.split)
    p.out_map = make_out_map(&omap, a.parts, a.M, a.N, a.N, tiles_most / (p.mt * p.nt), (int64_t)a.M * a.N, false);
  else
    p.out_map = make_out_map(&omap, a.out, WGRAD ? a.M : a.S, a.N, a.out_ld, WGRAD ? a.E : 1, a.out_step, a.out_bf16);
  // (the up half's parts start at column N)
  p.gu_map = ACT >= 0 && a.N * (a.out_bf16 ? 2 : 4) % 16 == 0 && make_out_map(&gmap, a.gu, a.S, 2 * (int64_t)a.N, a.gu_ld, 1, 0, a.out_bf16);
  if (!p.out_map) omap = amap;
  if (!p.gu_map) gmap = amap;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(mm_pairs(), tiles_most));
  p.stages = kMmMaxStages;
  while (mm_smem(p.E, p.stages, p.tile_n) > kMmMost) --p.stages;
  const int smem = mm_smem(p.E, p.stages, p.tile_n);
  return launch_early(kern, (unsigned)(2 * pairs), kMmThreads, smem, s, amap, bmap, omap, gmap, p);
}

MmParams params_of(const MmArgs& a) {
  MmParams p{};
  p.offsets = a.offsets, p.E = a.E, p.S = a.S, p.N = a.N, p.K = a.K, p.M = a.M;
  p.terms = 1;
  // products of the operands' planes (a, b), small ones first
  if (a.a.planes > 1 && a.b.planes > 1) {  // (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
    p.terms = 6, p.terms_a = 0x001012, p.terms_b = 0x010210;
  } else if (a.a.planes > 1) {             // (2,0) (1,0) (0,0), or without the first
    p.terms = a.a.planes, p.terms_a = p.terms == 3 ? 0x012 : 0x01;
  } else if (a.b.planes > 1) {
    p.terms = a.b.planes, p.terms_b = p.terms == 3 ? 0x012 : 0x01;
  }
  p.out = a.out, p.out_ld = a.out_ld, p.out_step = a.out_step;
  p.gu = a.gu, p.gu_ld = a.gu_ld;
  p.split = a.split, p.parts = a.parts, p.beside = a.beside, p.turned = a.turned;
  return p;
}

}  // namespace

static_assert(mm_smem(kMaxExperts, 5, 256) <= kMmMost && mm_smem(128, 6, 256) <= kMmMost && mm_smem(128, 8, 128) <= kMmMost, "shared memory of the products");

cudaError_t launch_expert_mm_rows(const MmArgs& a, cudaStream_t s) {
  if (a.S == 0) return cudaSuccess;
  MmParams p = params_of(a);
  const bool gated = a.act >= 0;
  const int64_t N = gated ? 2 * (int64_t)a.N : a.N, down = (int64_t)a.S / 256 + std::min(a.E, a.S);
  // rows of tiles: at most `down`, and about as many as there are experts, or half a one for each beyond their rows
  const int64_t about = std::max<int64_t>(std::min(a.E, a.S), (a.S + 255) / 256 + (a.E > 1 ? a.E / 2 : 0));
  // columns of a tile by the rounds of tiles that the pairs of SMs go through; one of 128 columns takes about 0.6 of
  // the time of one of 256
  const auto rounds = [&](int n) { return (about * ((N + n - 1) / n) + mm_pairs() - 1) / mm_pairs(); };
  p.tile_n = 5 * rounds(256) > 3 * rounds(128) ? 128 : 256;
  p.nt = (int)((N + p.tile_n - 1) / p.tile_n), p.mt = 1;
  if (gated) p.nt = (a.N + p.tile_n / 2 - 1) / (p.tile_n / 2);
  p.b_mn = a.b_mn, p.b_each = a.b.experts > 1;
  p.idesc = mm_idesc(false, a.b_mn, p.tile_n);
  p.chunk = a.f32 ? 8 : 1 << 20;
  const int64_t most = down * p.nt;
  using H = __nv_bfloat16;
  if (a.f32) switch (a.act) {
      case EMB_ACT_SILU: return launch_mm<false, EMB_ACT_SILU, true, true, float>(a, p, most, s);
      case EMB_ACT_GELU: return launch_mm<false, EMB_ACT_GELU, true, true, float>(a, p, most, s);
      case EMB_ACT_RELU: return launch_mm<false, EMB_ACT_RELU, true, true, float>(a, p, most, s);
      case EMB_ACT_SIGMOID: return launch_mm<false, EMB_ACT_SIGMOID, true, true, float>(a, p, most, s);
      default: return launch_mm<false, -1, true, true, float>(a, p, most, s);
    }
  switch (a.act) {
    case EMB_ACT_SILU: return launch_mm<false, EMB_ACT_SILU, false, false, H>(a, p, most, s);
    case EMB_ACT_GELU: return launch_mm<false, EMB_ACT_GELU, false, false, H>(a, p, most, s);
    case EMB_ACT_RELU: return launch_mm<false, EMB_ACT_RELU, false, false, H>(a, p, most, s);
    case EMB_ACT_SIGMOID: return launch_mm<false, EMB_ACT_SIGMOID, false, false, H>(a, p, most, s);
    default: return launch_mm<false, -1, false, false, H>(a, p, most, s);
  }
}

cudaError_t launch_expert_mm_wgrad(const MmArgs& a, cudaStream_t s) {
  MmParams p = params_of(a);
  p.tile_n = a.tile_n;
  p.nt = (a.N + p.tile_n - 1) / p.tile_n, p.mt = (a.M + 255) / 256;
  p.idesc = mm_idesc(true, true, p.tile_n);
  p.chunk = p.terms == 3 ? 4 : 8;
  if (a.S > 0) {
    const int64_t parts = a.split ? (int64_t)a.S / a.split + std::min(a.E, a.S) : a.E;
    const cudaError_t e = a.f32        ? launch_mm<true, -1, true, true, float>(a, p, parts * p.mt * p.nt, s)
                          : a.out_bf16 ? launch_mm<true, -1, true, false, __nv_bfloat16>(a, p, parts * p.mt * p.nt, s)
                                       : launch_mm<true, -1, true, false, float>(a, p, parts * p.mt * p.nt, s);
    if (e != cudaSuccess || !a.split) return e;
  }
  // (no rows: no parts, and zeros)
  const int split = a.split ? a.split : 64;
  const int oe = a.out_bf16 ? 2 : 4, rows = a.turned ? a.N : a.M, cols = a.turned ? a.M : a.N;  // of out
  const bool vec = cols % 4 == 0 && rows_on(a.out, a.out_ld, oe, 4 * oe) && a.out_step % 4 == 0;
  // (parts come of matrices of a few dozen tiles, and zeros alone where there are no rows)
  const bool many = a.split && a.S / a.split >= 16 * a.E;
  const auto sum = [&](auto kern, auto* out) {
    const int epu = vec ? 4 : 1, slots = many ? 32 : 256;
    cudaError_t e = cudaSuccess;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    // a launch takes rows with below 2^31 pieces
    const int64_t most = std::max<int64_t>(1, INT32_MAX / (cols / epu) - 64);
    for (int64_t r = 0; r < rows && e == cudaSuccess; r += most) {
      const int64_t here = std::min<int64_t>(most, rows - r);
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3((unsigned)((here * cols / epu + slots - 1) / slots), (unsigned)a.E);
      cfg.blockDim = dim3(256), cfg.stream = s, cfg.attrs = &attr, cfg.numAttrs = 1;
      e = cudaLaunchKernelEx(&cfg, kern, (const float*)a.parts, a.offsets, a.E, a.S, split, here * cols, FastDiv((uint32_t)(cols / epu)),
                             out + r * a.out_ld, a.out_ld, a.out_step);
    }
    return e;
  };
  const auto of = [&](auto* out) {
    using T = std::remove_pointer_t<decltype(out)>;
    if (many) return vec ? sum(k_expert_parts<T, 4, 8>, out) : sum(k_expert_parts<T, 1, 8>, out);
    return vec ? sum(k_expert_parts<T, 4, 1>, out) : sum(k_expert_parts<T, 1, 1>, out);
  };
  return a.out_bf16 ? of(static_cast<__nv_bfloat16*>(a.out)) : of(static_cast<float*>(a.out));
}

}  // namespace emb
