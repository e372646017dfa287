// cache.cuh -- writing keys and values into the paged cache, in 8 bits or as they are, and reading
// them back.
//
// A row is the D values of one token and key head.  8 bits: the row's power of two 2^e is the least
// with max |x| <= 448 2^e, so that every value fits e4m3 (largest 448 = 1.75 * 2^8); a power of two
// costs a floating format no precision and makes x / 2^e and q 2^e exact, so one rounding, to e4m3,
// is all there is.
//
// A row is held by lanes with 16 bytes of it each (16 of its 8-bit values, where it is read back), so a
// warp's loads are whole lines; the row's maximum takes log2 of the lanes' number shuffles.  A CTA's
// threads take the rows of one token, or of a few, and two tokens at a time are under way: where a token
// goes is worked out once for its keys and values.  Where there are many tokens (39950 of 8 heads of 128, from bf16 to
// 8 bits and back: 72 us at the copy rate) writing takes 61 us and reading 53, 4 - 4.7 TB/s: the first is bound by its
// arithmetic (issue slots 63 % busy: maxima, scaling, conversions), the second by loads under way.  Where there are few, by
// launch and three dependent trips (start, page, row): 384 accepted tokens of 64 sequences, both ways, 6.3 us.
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

// Where row (b, i), token `from` of `tokens`, lies: page * page_size + slot, or -1 where there is nothing to do.
__device__ __forceinline__ long long cache_place(const CacheRowsArgs &a, int b, int i, int from, int tokens) {
    const int start = __ldg(a.start + b);
    if (start < 0 || from < 0 || (a.count && i >= __ldg(a.count + b))) return -1;
    if (from >= tokens) {
        atomicOr(a.status, SPEC_DEV_BAD_LENGTH);
        return -1;
    }
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

// A thread's share of the rows of a token, `items` lanes of them in all: the same of its keys and its values.
struct CacheShare {
    int items, tokens, sub, rounds;  // tokens that the CTA takes at once, this thread's of them; rounds over a token's lanes
    __device__ CacheShare(int kv_heads, int lanes) {
        items = kv_heads * lanes;
        tokens = max(1, kCacheThreads / items);
        sub = items <= kCacheThreads ? threadIdx.x / items : 0;
        rounds = (items + kCacheThreads - 1) / kCacheThreads;
    }
    __device__ int item(int round) const { return items <= kCacheThreads ? threadIdx.x % items : threadIdx.x + round * kCacheThreads; }
};

// kCacheTokens: under way at once; 2, or 1 where the tokens are few and a CTA each is there for them.
template <typename T, int D, bool Q8, int kCacheTokens>
__global__ void __launch_bounds__(kCacheThreads) cache_append_kernel(const CacheRowsArgs a) {
    constexpr int kLanes = D / 8;
    const CacheShare my(a.cache.kv_heads, kLanes);
    const int all = a.B * a.S, step = my.tokens * kCacheTokens;
    for (int t0 = blockIdx.x * step; t0 < all; t0 += gridDim.x * step) {
        long long place[kCacheTokens];
        int batch[kCacheTokens], node[kCacheTokens];
#pragma unroll
        for (int k = 0; k < kCacheTokens; ++k) {
            const int token = t0 + k * my.tokens + my.sub;
            place[k] = -1;
            batch[k] = node[k] = 0;
            if (my.sub >= my.tokens || token >= all) continue;
            const int b = token / a.S, i = token - b * a.S, from = a.select ? __ldg(a.select + token) : i;
            place[k] = cache_place(a, b, i, from, a.N);
            batch[k] = b;
            node[k] = from;
        }
        for (int round = 0; round < my.rounds; ++round) {  // (the whole CTA goes round together: the shuffles take whole warps)
            const int item = my.item(round), g = item / kLanes, part = item % kLanes;
            const size_t within = static_cast<size_t>(g) * D + part * 8;
            uint4 loaded[2][kCacheTokens];
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int k = 0; k < kCacheTokens; ++k) {
                    loaded[w][k] = make_uint4(0, 0, 0, 0);
                    if (place[k] >= 0 && item < my.items)
                        loaded[w][k] = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const T *>(a.src[w]) + batch[k] * a.batch_stride[w] + node[k] * a.token_stride[w] + within));
                }
#pragma unroll
            for (int k = 0; k < kCacheTokens; ++k) {
                const bool live = place[k] >= 0 && item < my.items;
                const size_t to = live ? cache_row(a.cache, place[k], g) : 0;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint4 x = loaded[w][k];
                    if (!Q8) {
                        if (live) *reinterpret_cast<uint4 *>(a.cache.data[w] + (to * D + part * 8) * 2) = x;
                        continue;
                    }
                    // The largest magnitude, as whole numbers: without their signs the elements are ordered as their
                    // bits are, infinities above the finite ones and NaN above those.
                    const uint32_t bits4[4] = {x.x, x.y, x.z, x.w};
                    uint32_t most = __vmaxu2(__vmaxu2(bits4[0] & 0x7fff7fffu, bits4[1] & 0x7fff7fffu), __vmaxu2(bits4[2] & 0x7fff7fffu, bits4[3] & 0x7fff7fffu));
#pragma unroll
                    for (int m = 1; m < kLanes; m *= 2) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, m));
                    const uint32_t largest = max(most & 0xffffu, most >> 16);
                    // max = c 2^(E - 127), 1 <= c < 2 (a subnormal maximum has E = 0 and is far below the least e)
                    const uint32_t bits = __float_as_uint(Elt<T>::to_float2(largest).x);
                    const int e = min(max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), Elt<T>::kLeastExp), Elt<T>::kTopExp);
                    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                    float v[8];
                    unpack8<T>(x, v);
#pragma unroll
                    for (int h = 0; h < 8; ++h) v[h] *= inv;
                    if (e >= Elt<T>::kTopExp)  // 256 2^e would not come back
#pragma unroll
                        for (int h = 0; h < 8; ++h) v[h] = fminf(fmaxf(v[h], -240.0f), 240.0f);
                    uint32_t q[2] = {0, 0};
#pragma unroll
                    for (int h = 0; h < 8; h += 2)
                        q[h / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(v[h], v[h + 1]), __NV_SATFINITE, __NV_E4M3)) << (h % 4 * 8);
                    if (live) {
                        *reinterpret_cast<uint2 *>(a.cache.data[w] + to * D + part * 8) = make_uint2(q[0], q[1]);
                        if (part == 0) a.cache.scale[w][to] = largest >= Elt<T>::kInfinity ? 255 : static_cast<uint8_t>(e + 127);
                    }
                }
            }
        }
    }
}

template <typename T, int D, bool Q8, int kCacheTokens>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheRowsArgs a) {
    constexpr int kEach = Q8 ? 16 : 8, kLanes = D / kEach;  // values of a lane
    const CacheShare my(a.cache.kv_heads, kLanes);
    const int all = a.B * a.S, step = my.tokens * kCacheTokens;
    for (int t0 = blockIdx.x * step; t0 < all; t0 += gridDim.x * step) {
        long long place[kCacheTokens];
#pragma unroll
        for (int k = 0; k < kCacheTokens; ++k) {
            const int token = t0 + k * my.tokens + my.sub;
            place[k] = my.sub < my.tokens && token < all ? cache_place(a, token / a.S, token % a.S, 0, 1) : -1;
        }
        for (int round = 0; round < my.rounds; ++round) {
            const int item = my.item(round), g = item / kLanes, part = item % kLanes;
            if (item >= my.items) continue;
            uint4 x[2][kCacheTokens];
            uint32_t scale[2][kCacheTokens];
#pragma unroll
            for (int k = 0; k < kCacheTokens; ++k) {
                if (place[k] < 0) continue;
                const size_t at = cache_row(a.cache, place[k], g);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    x[w][k] = *reinterpret_cast<const uint4 *>(a.cache.data[w] + (at * D + part * kEach) * (Q8 ? 1 : 2));
                    if (Q8) scale[w][k] = a.cache.scale[w][at];
                }
            }
#pragma unroll
            for (int k = 0; k < kCacheTokens; ++k) {
                if (place[k] < 0) continue;
                const size_t token = static_cast<size_t>(t0) + k * my.tokens + my.sub, at = (token * a.cache.kv_heads + g) * (D / 8) + part * (kEach / 8);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint4 *to = reinterpret_cast<uint4 *>(a.dst[w]) + at;
                    if (!Q8) {
                        *to = x[w][k];
                        continue;
                    }
                    const float s = scale_of(scale[w][k]);
                    const uint32_t q[4] = {x[w][k].x, x[w][k].y, x[w][k].z, x[w][k].w};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float2 f = e4m3x2(q[2 * h + e / 4] >> (e % 4 * 8));
                            v[e] = f.x * s;
                            v[e + 1] = f.y * s;
                        }
                        to[h] = pack8<T>(v);
                    }
                }
            }
        }
    }
}

}  // namespace context
}  // namespace spec
