// Device pieces shared by the norm/rotation, cache and cache-attention kernels.
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"
#include "kv.h"

namespace q4 {

enum : unsigned {
    kFaultBadSlot = 32u,       // a cache slot at or past num_pages * page_size
    kFaultBadPage = 64u,       // a page id outside [0, num_pages)
    kFaultBadLength = 128u,    // a sequence length outside [0, max_pages * page_size]
    kFaultBadPosition = 256u,  // a position outside [0, max_pos)
};

__device__ __forceinline__ float qnan() { return __int_as_float(0x7fc00000); }

// 16 bytes of activations: four fp32 or eight 16-bit values.
template <typename T>
struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
};

template <typename T, int N>
__device__ __forceinline__ void load_floats(const T* p, float (&x)[N]);

template <>
__device__ __forceinline__ void load_floats<float, 4>(const float* p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
template <>
__device__ __forceinline__ void load_floats<float, 8>(const float* p, float (&x)[8]) {
    const float4 v = reinterpret_cast<const float4*>(p)[0], w = reinterpret_cast<const float4*>(p)[1];
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ void load_halves8(const T* p, float (&x)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(w[i], T());
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void load_floats<__half, 8>(const __half* p, float (&x)[8]) {
    load_halves8(p, x);
}
template <>
__device__ __forceinline__ void load_floats<__nv_bfloat16, 8>(const __nv_bfloat16* p, float (&x)[8]) {
    load_halves8(p, x);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
// Values leave in the activation type with one rounding to nearest even, the only one after the fp32 arithmetic.
template <typename T, int N>
__device__ __forceinline__ void store_floats(T* p, const float (&x)[N]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] =
                make_uint4(pack2(x[8 * i], x[8 * i + 1], T()), pack2(x[8 * i + 2], x[8 * i + 3], T()),
                           pack2(x[8 * i + 4], x[8 * i + 5], T()), pack2(x[8 * i + 6], x[8 * i + 7], T()));
    }
}

// Calls fn with a value of the activation type of `dtype` (validated by the ABI).
template <typename F>
cudaError_t with_dtype(int dtype, F fn) {
    if (dtype == Q4_F16) return fn(__half());
    if (dtype == Q4_BF16) return fn(__nv_bfloat16());
    return fn(float());
}

// Row of the cache's planar Q4 matrices (qs [rows][D/2], d [rows][D/32]) of head h at page `page`, offset `off`.
__device__ __forceinline__ long long cache_row(const kv4_cache& c, int page, int h, int off) {
    return ((long long)page * c.num_kv_heads + h) * c.page_size + off;
}

}  // namespace q4
