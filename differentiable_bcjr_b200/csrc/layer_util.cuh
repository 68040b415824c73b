// layer_util.cuh -- element types and small helpers of the calls in bcjr_layer.h.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bcjr_layer.h"

namespace bcjr {

inline bool ptr_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool dtype_ok(int d) { return d == BCJR_F32 || d == BCJR_F16 || d == BCJR_BF16; }
inline size_t dtype_size(int d) { return d == BCJR_F32 ? 4 : 2; }
inline bcjr_status launched() { return cudaGetLastError() == cudaSuccess ? BCJR_OK : BCJR_ERR_CUDA; }
inline cudaStream_t as_stream(bcjr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// What is asked of each device once.  Several host threads may call at the same
// time: they would store the same answer, and nothing is stored of a call that failed.
constexpr int kDevices = 64;
using PerDevice = std::atomic<int>[kDevices];

inline int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kDevices ? dev : -1;
}

inline int device_attribute(cudaDeviceAttr attr, PerDevice& known, int dev) {
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, attr, dev) != cudaSuccess) return 0;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Multiprocessors of the current device.
inline int sm_count() {
  static PerDevice known;
  const int dev = current_device();
  return dev < 0 ? 0 : device_attribute(cudaDevAttrMultiProcessorCount, known, dev);
}

// Lets a kernel (one `done` a kernel) use as much dynamic shared memory on the
// current device as a CTA can have.  The limit is the kernel's, for all host
// threads, so it is never set to what one launch needs: a thread with a small
// launch would lower it between another one's setting and its launch.
inline bool allow_shared(const void* kernel, PerDevice& done) {
  static PerDevice most;
  const int dev = current_device();
  if (dev < 0) return false;
  if (done[dev].load(std::memory_order_acquire)) return true;
  const int bytes = device_attribute(cudaDevAttrMaxSharedMemoryPerBlockOptin, most, dev);
  if (bytes <= 0) return false;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done[dev].store(1, std::memory_order_release);
  return true;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Element i of an array whose type is only known at run time (a uniform branch).
__device__ __forceinline__ float load_as_f32(const void* p, int dtype, size_t i) {
  if (dtype == BCJR_F32) return static_cast<const float*>(p)[i];
  if (dtype == BCJR_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Elements i .. i + 3, which are aligned together.
__device__ __forceinline__ float4 load4_as_f32(const void* p, int dtype, size_t i) {
  if (dtype == BCJR_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
  if (dtype == BCJR_F16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
    return make_float4(a.x, a.y, b.x, b.y);
  }
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

__device__ __forceinline__ void store_from_f32(void* p, int dtype, size_t i, float v) {
  if (dtype == BCJR_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == BCJR_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

}  // namespace bcjr
