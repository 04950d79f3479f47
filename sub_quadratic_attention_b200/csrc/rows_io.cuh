// rows_io.cuh -- element conversions and small helpers shared by the row operators
// (gated_scan.cu, residual_norm.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "spectre_mix.h"

namespace rows_io {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline int status_of(cudaError_t e) {
    if (e == cudaSuccess) return SPECTRE_OK;
    cudaGetLastError();
    return e == cudaErrorMemoryAllocation ? SPECTRE_ERR_NOMEM : SPECTRE_ERR_CUDA;
}

inline bool current_device_is(int dev) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return cur == dev;
}

// The current device and its SM count, or SPECTRE_ERR_DEVICE where it is no sm_100 device.
inline int usable_device(int *dev, int *nsm) {
    int major = 0;
    if (cudaGetDevice(dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(nsm, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
        cudaGetLastError();
        return SPECTRE_ERR_DEVICE;
    }
    return major == 10 ? SPECTRE_OK : SPECTRE_ERR_DEVICE;
}

}  // namespace rows_io
