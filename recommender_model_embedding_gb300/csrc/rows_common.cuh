// Row access shared by the expert and gated-norm kernels: packs of EPU consecutive elements
// of an fp32 or bf16 row (up to 16 bytes, where everything is aligned for it; else one
// element), held as loaded and widened to fp32 where they are used.
#pragma once

#include <atomic>
#include <type_traits>
#include <utility>

#include "emb_internal.cuh"

namespace emb {

template <typename T, int EPU>
struct Pack;  // raw register image of EPU elements

template <>
struct Pack<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = *p; }
  __device__ __forceinline__ void zero() { r = 0.f; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = r; }
  __device__ __forceinline__ void set(const float (&v)[1]) { r = v[0]; }
  __device__ __forceinline__ void store(float* p) const { *p = r; }
};

template <>
struct Pack<__nv_bfloat16, 1> {
  __nv_bfloat16 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *p; }
  __device__ __forceinline__ void zero() { r = __float2bfloat16_rn(0.f); }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __bfloat162float(r); }
  __device__ __forceinline__ void set(const float (&v)[1]) { r = __float2bfloat16_rn(v[0]); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = r; }
};

template <>
struct Pack<float, 2> {
  float2 r;
  __device__ __forceinline__ void set(const float (&v)[2]) { r = make_float2(v[0], v[1]); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float2*>(p) = r; }
};

template <>
struct Pack<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
  }
  __device__ __forceinline__ void set(const float (&v)[4]) {
    r = make_float4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = r; }
};

template <>
struct Pack<__nv_bfloat16, 2> {
  uint32_t r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint32_t*>(p);
  }
  __device__ __forceinline__ void zero() { r = 0u; }
  __device__ __forceinline__ void get(float (&v)[2]) const {
    v[0] = __uint_as_float(r << 16);
    v[1] = __uint_as_float(r & 0xFFFF0000u);
  }
  __device__ __forceinline__ void set(const float (&v)[2]) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
    r = *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint32_t*>(p) = r; }
};

template <>
struct Pack<__nv_bfloat16, 4> {
  uint2 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void zero() { r = make_uint2(0u, 0u); }
  __device__ __forceinline__ void set(const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    r = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint2*>(p) = r;
  }
};

template <>
struct Pack<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // widening a bf16 is a 16-bit shift
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = r;
  }
};

// Quotient by a divisor fixed at launch: for i < 2^31, i / d = (i * mul) >> sh with
// sh = 31 + ceil(log2 d) and mul = ceil(2^sh / d) (mul * d - 2^sh < d <= 2^(sh - 31), so the
// excess i * (mul * d - 2^sh) / 2^sh stays below 1 and the floor is exact).
struct FastDiv {
  uint32_t d, mul;
  int sh;
  explicit FastDiv(uint32_t d_ = 1) : d(d_) {
    int l = 0;
    while ((1ull << l) < d) ++l;
    sh = 31 + l;
    mul = (uint32_t)(((1ull << sh) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t div(uint32_t i) const {
    return (uint32_t)(((uint64_t)i * mul) >> sh);
  }
};

// Sum over the `tpr` lanes (a power of two <= 32) that share a row.
__device__ __forceinline__ float lanes_sum(float v, int tpr) {
  for (int o = tpr >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The tower's kernels run for microseconds, so they are launched early: the next kernel of the
// stream may be set up and its CTAs placed while the last one still runs.  Every kernel
// therefore passes wait_for_earlier() before it touches anything that earlier work writes or
// reads (it holds until that work has finished and its writes are visible; since every kernel
// passes it, that covers all earlier work, not the last kernel's alone), and says
// let_next_start() once its own CTAs may be joined.  Work of other kinds before or after such a
// kernel (copies, kernels launched in the ordinary way) is ordered as always.
__device__ __forceinline__ void wait_for_earlier() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), unsigned grid, int threads, int smem, cudaStream_t s,
                         A&&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem, cfg.stream = s, cfg.attrs = &attr, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

// Multiprocessors of the current device (context-free calls; the count is read once a device).
inline int device_sms() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    if (dev < kDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && sms > 0) {
      if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
      return sms;
    }
  }
  cudaGetLastError();
  return 1;
}

// Lets a kernel take as much dynamic shared memory as a CTA can have (asked for once per kernel and
// device: the request costs a call's host time).
template <auto KERN>
cudaError_t prepare_kernel() {
  static std::atomic<uint64_t> done{0};
  int dev = 0, most = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes fa{};
  e = cudaFuncGetAttributes(&fa, KERN);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)fa.sharedSizeBytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Whether a matrix of rows allows accesses of `bytes` (a power of two): base and row step on
// such boundaries.
inline bool rows_on(const void* p, int64_t ld, int elem, int bytes) {
  return p == nullptr ||
         (((reinterpret_cast<uintptr_t>(p) | (uint64_t)(ld * elem)) & (uint64_t)(bytes - 1)) == 0);
}
inline bool rows16(const void* p, int64_t ld, int elem) { return rows_on(p, ld, elem, 16); }

}  // namespace emb
