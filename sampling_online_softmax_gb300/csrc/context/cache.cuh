// cache.cuh -- writing keys and values into the paged cache, in 8 bits or as they are, and reading
// them back.
//
// A row is the D values of one token and key head.  8 bits: the row's power of two 2^e is the least
// with max |x| <= 448 2^e, so that every value fits e4m3 (largest 448 = 1.75 * 2^8); a power of two
// costs a floating format no precision and makes x / 2^e and q 2^e exact, so one rounding, to e4m3,
// is all there is.
//
// A row is held by D / 8 lanes, 16 bytes of it each, so a warp's loads and stores are whole 128-byte
// lines; the row's maximum takes log2(D / 8) shuffles.  Both kernels move bytes and are bound by HBM
// where there are many rows, by launch and two dependent trips (table entry, then row) where there
// are few.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "context.h"
#include "elt.cuh"

namespace spec {
namespace context {

constexpr int kCacheThreads = 256;

struct CacheRowsArgs {
    CacheView cache;
    const unsigned char *src[2];  // append: k, v
    unsigned char *dst[2];        // read: k, v
    long long batch_stride[2], token_stride[2];  // append, in elements
    const int32_t *select, *start, *count;
    int B, N, S;
    uint32_t *status;
};

// Where row (b, i) lies: page * page_size + slot, or -1 where there is nothing to do.
__device__ __forceinline__ long long cache_place(const CacheRowsArgs &a, int b, int i) {
    const int start = __ldg(a.start + b);
    if (start < 0 || (a.count && i >= __ldg(a.count + b))) return -1;
    const long long pos = static_cast<long long>(start) + i;
    const int column = static_cast<int>(pos >> a.cache.page_bits);
    if (column >= a.cache.table_width) {
        atomicOr(a.status, SPEC_DEV_BAD_LENGTH);
        return -1;
    }
    const int page = __ldg(a.cache.table + static_cast<size_t>(b) * a.cache.table_width + column);
    if (page < 0 || page >= a.cache.pages) {
        atomicOr(a.status, SPEC_DEV_BAD_PAGE);
        return -1;
    }
    return (static_cast<long long>(page) << a.cache.page_bits) + (pos & ((1 << a.cache.page_bits) - 1));
}

// The index of head g's row at `place` in [pages, kv_heads, page_size].
__device__ __forceinline__ size_t cache_row(const CacheView &c, long long place, int g) {
    const long long page = place >> c.page_bits, slot = place & ((1 << c.page_bits) - 1);
    return (static_cast<size_t>(page * c.kv_heads + g) << c.page_bits) + static_cast<size_t>(slot);
}

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kCacheThreads) cache_append_kernel(const CacheRowsArgs a) {
    constexpr int kLanes = D / 8;
    const int part = threadIdx.x % kLanes;
    const long long rows = 2ll * a.B * a.S * a.cache.kv_heads;  // k and v next to each other: (b, i, k/v, head)
    const long long step = static_cast<long long>(gridDim.x) * (kCacheThreads / kLanes);
    const long long first = static_cast<long long>(blockIdx.x) * (kCacheThreads / kLanes) + threadIdx.x / kLanes;
    // (every lane of a warp goes round together: the shuffles below take all of them)
    for (long long at = first; at - first % (32 / kLanes) < rows; at += step) {
        const int g = static_cast<int>(at % a.cache.kv_heads);
        const int which = static_cast<int>(at / a.cache.kv_heads & 1);
        const long long token = at / (2 * a.cache.kv_heads);
        const int b = static_cast<int>(token / a.S), i = static_cast<int>(token % a.S);
        long long place = -1;
        int from = i;
        if (at < rows) {
            if (a.select) from = __ldg(a.select + token);
            if (from >= a.N) atomicOr(a.status, SPEC_DEV_BAD_LENGTH);
            else if (from >= 0) place = cache_place(a, b, i);
        }
        uint4 x = make_uint4(0, 0, 0, 0);
        if (place >= 0) {
            const T *row = reinterpret_cast<const T *>(a.src[which]) + b * a.batch_stride[which] + from * a.token_stride[which] + static_cast<size_t>(g) * D;
            x = __ldg(reinterpret_cast<const uint4 *>(row) + part);
        }
        const size_t row = place >= 0 ? cache_row(a.cache, place, g) : 0;
        if (!Q8) {
            if (place >= 0) *reinterpret_cast<uint4 *>(a.cache.data[which] + (row * D + part * 8) * 2) = x;
            continue;
        }
        float v[8], most = 0.0f;
        unpack8<T>(x, v);
        bool odd = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            most = fmaxf(most, fabsf(v[k]));
            odd |= !isfinite(v[k]);
        }
#pragma unroll
        for (int m = 1; m < kLanes; m *= 2) {
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, m));
            odd |= __shfl_xor_sync(0xffffffffu, static_cast<int>(odd), m) != 0;
        }
        // max = c 2^(E - 127), 1 <= c < 2 (a subnormal maximum has E = 0 and is far below the least e)
        const uint32_t bits = __float_as_uint(most);
        const int e = max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), Elt<T>::kLeastExp);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float top = e >= Elt<T>::kTopExp ? 240.0f : 448.0f;  // 256 2^e would not come back
        uint32_t q[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const float2 pair = make_float2(fminf(fmaxf(v[k] * inv, -top), top), fminf(fmaxf(v[k + 1] * inv, -top), top));
            q[k / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(pair, __NV_SATFINITE, __NV_E4M3)) << (k % 4 * 8);
        }
        if (place >= 0) {
            *reinterpret_cast<uint2 *>(a.cache.data[which] + row * D + part * 8) = make_uint2(q[0], q[1]);
            if (part == 0) a.cache.scale[which][row] = odd ? 255 : static_cast<uint8_t>(e + 127);
        }
    }
}

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheRowsArgs a) {
    constexpr int kLanes = D / 8;
    const int part = threadIdx.x % kLanes;
    const long long rows = 2ll * a.B * a.S * a.cache.kv_heads;
    const long long step = static_cast<long long>(gridDim.x) * (kCacheThreads / kLanes);
    for (long long at = static_cast<long long>(blockIdx.x) * (kCacheThreads / kLanes) + threadIdx.x / kLanes; at < rows; at += step) {
        const int g = static_cast<int>(at % a.cache.kv_heads);
        const int which = static_cast<int>(at / a.cache.kv_heads & 1);
        const long long token = at / (2 * a.cache.kv_heads);
        const long long place = cache_place(a, static_cast<int>(token / a.S), static_cast<int>(token % a.S));
        if (place < 0) continue;
        const size_t row = cache_row(a.cache, place, g);
        uint4 x;
        if (!Q8) {
            x = *reinterpret_cast<const uint4 *>(a.cache.data[which] + (row * D + part * 8) * 2);
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(a.cache.data[which] + row * D + part * 8);
            const float s = scale_of(a.cache.scale[which][row]);
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const float2 f = e4m3x2((k < 4 ? q.x : q.y) >> (k % 4 * 8));
                v[k] = f.x * s;
                v[k + 1] = f.y * s;
            }
            x = pack8<T>(v);
        }
        reinterpret_cast<uint4 *>(a.dst[which])[(static_cast<size_t>(token) * a.cache.kv_heads + g) * kLanes + part] = x;
    }
}

}  // namespace context
}  // namespace spec
