// dtypes.cuh -- the element types of the dense-table operators (spmv_dtype)
// and their conversions from and to fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "internal.h"

namespace spmv {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Calls f(T{}) with T = the C++ type of a (checked) spmv_dtype.
template <class F>
cudaError_t with_dtype(int type, F&& f) {
  switch (type) {
    case SPMV_F16: return f(__half{});
    case SPMV_BF16: return f(__nv_bfloat16{});
    default: return f(float{});
  }
}

inline bool dtype_ok(int type) { return type >= SPMV_F32 && type <= SPMV_BF16; }
inline int dtype_bytes(int type) { return type == SPMV_F32 ? 4 : 2; }

// Host-side argument checks: the bytes from the first element of n rows of
// `width` elements to past the last one, whether two such ranges share a
// byte, whether a pointer is not a multiple of an element's size.
inline long long extent(long long n, long long width, long long ld, int bytes) {
  return n > 0 && width > 0 ? ((n - 1) * ld + width) * bytes : 0;
}
inline bool overlap(const void* a, long long na, const void* b, long long nb) {
  const char* pa = static_cast<const char*>(a);
  const char* pb = static_cast<const char*>(b);
  return na > 0 && nb > 0 && pa < pb + nb && pb < pa + na;
}
inline bool misaligned(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}

// The most dynamic shared memory a kernel may ask for, allowed once per device
// (not during a stream capture: one call outside it comes first).
struct KernelOnce {
  std::atomic<unsigned long long> devices{0};
  cudaError_t allow(const void* kernel, int smem) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// Launches a kernel that may start before the one ahead of it in the stream has
// ended (it waits for that by itself, grid_dependency_wait, before it touches
// memory), which hides most of the gap between two short kernels.
// Such a kernel is under way while its inputs may still be written, so it reads
// them by ordinary loads: the read-only path (__ldg, const __restrict__) is for
// data that nothing writes during the kernel's life.
template <class... P, class... A>
cudaError_t launch_dependent_smem(void (*kernel)(P...), dim3 grid, int threads, size_t smem,
                                  cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  note_launches(1);
  return e;
}

template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s,
                             A&&... args) {
  return launch_dependent_smem(kernel, grid, threads, 0, s, static_cast<A&&>(args)...);
}

// E consecutive elements as one aligned access of E * sizeof(T) bytes (a
// power of two, at most 32: two 16-byte accesses).
template <class T, int E>
struct __align__(sizeof(T) * E < 16 ? sizeof(T) * E : 16) Pack {
  T v[E];
};

}  // namespace spmv
