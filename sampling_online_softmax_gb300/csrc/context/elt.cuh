// elt.cuh -- the element types of queries, keys and values, and e4m3 with a power of two a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace spec {
namespace context {

template <typename T>
struct Elt;

template <>
struct Elt<__nv_bfloat16> {
    static constexpr int kLeastExp = -110;  // of a row's power of two: 2^e and q 2^e stay normal
    static constexpr int kTopExp = 120;     // where a row's largest q 2^e could be 2^128, past bf16's range
    static constexpr uint32_t kInfinity = 0x7f80;
    static __device__ __forceinline__ float2 to_float2(uint32_t x) {
        return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t from_float2(float a, float b) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

template <>
struct Elt<__half> {
    static constexpr int kLeastExp = -24;  // fp16 holds multiples of 2^-24 alone
    static constexpr int kTopExp = 8;      // where a row's largest q 2^e could be 2^16, past fp16's range
    static constexpr uint32_t kInfinity = 0x7c00;
    static __device__ __forceinline__ float2 to_float2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }
    static __device__ __forceinline__ uint32_t from_float2(float a, float b) {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &x, float *v) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = Elt<T>::to_float2(w[k]);
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float *v) {
    return make_uint4(Elt<T>::from_float2(v[0], v[1]), Elt<T>::from_float2(v[2], v[3]), Elt<T>::from_float2(v[4], v[5]), Elt<T>::from_float2(v[6], v[7]));
}

// Two e4m3 values from the low 16 bits (exact).
__device__ __forceinline__ float2 e4m3x2(uint32_t x) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}
// The power of two that a scale byte stands for; NaN for 255, so that its row is.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return byte == 255 ? __int_as_float(0x7fffffff) : __uint_as_float(max(byte, 1u) << 23);
}

}  // namespace context
}  // namespace spec
