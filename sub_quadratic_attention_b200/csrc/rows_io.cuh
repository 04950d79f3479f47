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

// N neighbouring fp32 values of a thread, in pairs on which one instruction does two operations
// (N even), or one value.  The pairs stay 64-bit registers from operation to operation.
__device__ __forceinline__ unsigned long long pair_of(float x, float y) {
    unsigned long long p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
template <int N> struct Vec {
    static_assert(N % 2 == 0, "");
    unsigned long long p[N / 2];
    __device__ __forceinline__ Vec() {}
    __device__ __forceinline__ explicit Vec(float f) {
#pragma unroll
        for (int i = 0; i < N / 2; i++) p[i] = pair_of(f, f);
    }
    __device__ __forceinline__ float operator[](int j) const {
        float x, y;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p[j / 2]));
        return j % 2 ? y : x;
    }
    __device__ __forceinline__ void set(int j, float f) { p[j / 2] = j % 2 ? pair_of((*this)[j - 1], f) : pair_of(f, (*this)[j + 1]); }
};
template <> struct Vec<1> {
    float p;
    __device__ __forceinline__ Vec() {}
    __device__ __forceinline__ explicit Vec(float f) : p(f) {}
    __device__ __forceinline__ float operator[](int) const { return p; }
    __device__ __forceinline__ void set(int, float f) { p = f; }
};
template <int N> __device__ __forceinline__ Vec<N> operator+(const Vec<N> &a, const Vec<N> &b) {
    Vec<N> r;
    if constexpr (N == 1) r.p = a.p + b.p;
    else
#pragma unroll
        for (int i = 0; i < N / 2; i++) asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.p[i]) : "l"(a.p[i]), "l"(b.p[i]));
    return r;
}
template <int N> __device__ __forceinline__ Vec<N> operator*(const Vec<N> &a, const Vec<N> &b) {
    Vec<N> r;
    if constexpr (N == 1) r.p = a.p * b.p;
    else
#pragma unroll
        for (int i = 0; i < N / 2; i++) asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.p[i]) : "l"(a.p[i]), "l"(b.p[i]));
    return r;
}
template <int N> __device__ __forceinline__ Vec<N> fma(const Vec<N> &a, const Vec<N> &b, const Vec<N> &c) {
    Vec<N> r;
    if constexpr (N == 1) r.p = fmaf(a.p, b.p, c.p);
    else
#pragma unroll
        for (int i = 0; i < N / 2; i++) asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.p[i]) : "l"(a.p[i]), "l"(b.p[i]), "l"(c.p[i]));
    return r;
}
template <int N> __device__ __forceinline__ float sum_of(Vec<N> v) {
    if constexpr (N == 1) {
        return v.p;
    } else if constexpr (N == 2) {
        return v[0] + v[1];
    } else {
        Vec<N / 2> a, b;
#pragma unroll
        for (int i = 0; i < N / 4; i++) a.p[i] = v.p[i], b.p[i] = v.p[i + N / 4];
        return sum_of(a + b);
    }
}

// N values as they stand in memory, aligned to all of them.
template <typename T, int N> struct alignas(sizeof(T) * N) Pack {
    T v[N];
};
template <int N> __device__ __forceinline__ Vec<N> floats(const Pack<float, N> &x) {
    Vec<N> r;
    if constexpr (N == 1) r.p = x.v[0];
    else
#pragma unroll
        for (int i = 0; i < N / 2; i++) r.p[i] = pair_of(x.v[2 * i], x.v[2 * i + 1]);
    return r;
}
template <int N> __device__ __forceinline__ Vec<N> floats(const Pack<__nv_bfloat16, N> &x) {
    Vec<N> r;
    if constexpr (N == 1) r.p = __bfloat162float(x.v[0]);
    else
#pragma unroll
        for (int i = 0; i < N / 2; i++) {
            const unsigned u = reinterpret_cast<const unsigned *>(x.v)[i];   // a bf16 is a float's upper half
            r.p[i] = pair_of(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
    return r;
}
template <typename T, int N> __device__ __forceinline__ Pack<T, N> packed(const Vec<N> &f) {
    Pack<T, N> r;
    if constexpr (N > 1 && sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < N / 2; i++) {
            unsigned u;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
            reinterpret_cast<unsigned *>(r.v)[i] = u;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) r.v[j] = from_f<T>(f[j]);
    }
    return r;
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
