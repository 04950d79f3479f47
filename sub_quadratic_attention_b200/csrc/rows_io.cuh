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

// Two fp32 operations an instruction, on neighbouring values of a thread.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
template <int N> __device__ __forceinline__ void fma_all(float (&r)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2) {
        const float2 x = fma2({a[j], a[j + 1]}, {b[j], b[j + 1]}, {c[j], c[j + 1]});
        r[j] = x.x, r[j + 1] = x.y;
    }
    if constexpr (N % 2) r[N - 1] = fmaf(a[N - 1], b[N - 1], c[N - 1]);
}
template <int N> __device__ __forceinline__ void mul_all(float (&r)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2) {
        const float2 x = mul2({a[j], a[j + 1]}, {b[j], b[j + 1]});
        r[j] = x.x, r[j + 1] = x.y;
    }
    if constexpr (N % 2) r[N - 1] = a[N - 1] * b[N - 1];
}
template <int N> __device__ __forceinline__ void add_all(float (&r)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2) {
        const float2 x = add2({a[j], a[j + 1]}, {b[j], b[j + 1]});
        r[j] = x.x, r[j + 1] = x.y;
    }
    if constexpr (N % 2) r[N - 1] = a[N - 1] + b[N - 1];
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
