// lm_common.cuh -- element access and reductions shared by the kernels of the
// language-model operators.  Arithmetic is fp32 throughout; a bf16 value is
// widened exactly on load and rounded once, to nearest even, on store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "launch.cuh"

namespace rcc {
namespace lm {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// Two fp32 operations in one instruction, each rounded as usual.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight consecutive elements on a boundary of eight: one access, so that the
// threads of a warp fill whole 32-byte sectors (two 16-byte accesses would
// leave every sector half written, twice).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                 "=f"(v[6]), "=f"(v[7])
               : "l"(p) : "memory");
}
__device__ __forceinline__ void widen2(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  widen2(a.x, v[0], v[1]);
  widen2(a.y, v[2], v[3]);
  widen2(a.z, v[4], v[5]);
  widen2(a.w, v[6], v[7]);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]),
                                            pack2(v[4], v[5]), pack2(v[6], v[7]));
}
// Eight columns of a row of `dim`, for thread t of the G that share a slab of
// 8 G columns beginning at `base`: eight neighbours (VEC: aligned rows of whole
// vectors), or, for any alignment and length, every G-th column, so that a
// warp's accesses stay side by side.  Columns past the row read as zero and are
// not written.
template <bool VEC, int G>
__device__ __forceinline__ bool slab_live(size_t base, int t, size_t dim) {
  return base + (VEC ? t * 8 : t) < dim;
}
template <bool VEC, int G, typename T>
__device__ __forceinline__ void load_slab(const T* row, size_t base, int t, size_t dim,
                                          float (&v)[8]) {
  if constexpr (VEC) {
    load8(row + base + t * 8, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = base + e * G + t < dim ? to_f32(row[base + e * G + t]) : 0.f;
  }
}
template <bool VEC, int G, typename T>
__device__ __forceinline__ void store_slab(T* row, size_t base, int t, size_t dim,
                                           const float (&v)[8]) {
  if constexpr (VEC) {
    store8(row + base + t * 8, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (base + e * G + t < dim) from_f32(v[e], row[base + e * G + t]);
  }
}

// `n` (4, 8 or 16) bytes of global memory into shared memory, asynchronously
template <int N>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(N)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the newest N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A token id or label; one outside [0, vocab) comes back as -1 (padding).
__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, size_t t, size_t vocab) {
  const int64_t id = ids64 ? static_cast<const int64_t*>(ids)[t]
                           : static_cast<const int32_t*>(ids)[t];
  return id >= 0 && id < static_cast<int64_t>(vocab) ? id : -1;
}

// Barriers in shared memory, by their shared address
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Waits for a phase, at most about two seconds; false when that ran out.
constexpr long long kWaitCycles = 4000000000ll;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  if (bar_try(bar, parity)) return true;
  const long long t0 = clock64();
  do {
    if (bar_try(bar, parity)) return true;
  } while (clock64() - t0 < kWaitCycles);
  return false;
}

// launch_kernel for a grid of clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                           int cluster, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

constexpr int kMaxDevices = 64;  // whose properties are remembered

inline int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
  return dev;
}

// SMs of the current device (152 on GB300), asked for once a device.
inline int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  const int dev = current_device();
  int n = dev < kMaxDevices ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 152;
  }
  if (dev < kMaxDevices) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Lets `kernel` have `bytes` of dynamic shared memory on the current device;
// `done`, one bit a device, says where that has been asked for already.
template <typename K>
inline cudaError_t allow_shared(K kernel, int bytes, std::atomic<uint64_t>& done) {
  const int dev = current_device();
  const uint64_t bit = dev < kMaxDevices ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace lm
}  // namespace rcc
