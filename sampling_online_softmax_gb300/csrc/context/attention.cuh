// attention.cuh -- attention of drafted tokens over the paged cache and their own tree.
//
// One warp a row (b, n, h): it goes over the keys one by one, each lane holding D / 32 values of the
// query and of the weighted sum, with a running maximum and sum.
#pragma once

#include "cache.cuh"
#include "attention.h"

namespace spec {
namespace context {

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(128) attention_kernel(const AttentionArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.B) * a.N * a.heads) return;
    const int h = static_cast<int>(row % a.heads), n = static_cast<int>(row / a.heads % a.N), b = static_cast<int>(row / a.heads / a.N);
    const int g = h / (a.heads / a.cache.kv_heads);
    int len = __ldg(a.lens + b);
    if (len < 0) return;
    bool bad_page = false;
    if (len < a.shared_len || len > a.cache.table_width << a.cache.page_bits) {
        if (lane == 0) atomicOr(a.status, SPEC_DEV_BAD_LENGTH);
        len = min(max(len, a.shared_len), a.cache.table_width << a.cache.page_bits);
    }
    float q[E], o[E], m = -INFINITY, l = 0.0f;
    const T *qr = reinterpret_cast<const T *>(a.q) + b * a.stride[0] + n * a.stride[1] + static_cast<size_t>(h) * D + lane * E;
    for (int e = 0; e < E; ++e) q[e] = static_cast<float>(qr[e]) * a.scale, o[e] = 0.0f;
    auto key = [&](const float *k, const float *v) {
        float s = 0.0f;
        for (int e = 0; e < E; ++e) s += q[e] * k[e];
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float top = fmaxf(m, s);
        const float was = m == -INFINITY ? 0.0f : expf(m - top), p = s == -INFINITY ? 0.0f : expf(s - top);
        l = l * was + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * was + p * v[e];
        m = top;
    };
    for (int j = 0; j < len; ++j) {
        const int owner = j < a.shared_len ? 0 : b;
        const int page = __ldg(a.cache.table + static_cast<size_t>(owner) * a.cache.table_width + (j >> a.cache.page_bits));
        if (page < 0 || page >= a.cache.pages) {
            bad_page = true;
            continue;
        }
        const size_t at = cache_row(a.cache, (static_cast<long long>(page) << a.cache.page_bits) + (j & ((1 << a.cache.page_bits) - 1)), g);
        float x[2][E];
        for (int w = 0; w < 2; ++w) {
            const float s = Q8 ? scale_of(a.cache.scale[w][at]) : 1.0f;
            for (int e = 0; e < E; ++e) {
                if (Q8) x[w][e] = Elt<T>::clamp(e4m3x2(a.cache.data[w][at * D + lane * E + e]).x * s);
                else x[w][e] = static_cast<float>(reinterpret_cast<const T *>(a.cache.data[w])[at * D + lane * E + e]);
            }
        }
        key(x[0], x[1]);
    }
    const int words = (a.N + 31) / 32;
    for (int j = 0; j < a.N; ++j) {
        const bool on = a.mask ? (a.mask[static_cast<size_t>(n) * words + (j >> 5)] >> (j & 31)) & 1 : j <= n;
        if (!on) continue;
        float x[2][E];
        for (int e = 0; e < E; ++e) {
            x[0][e] = static_cast<float>((reinterpret_cast<const T *>(a.k) + b * a.stride[2] + j * a.stride[3] + static_cast<size_t>(g) * D)[lane * E + e]);
            x[1][e] = static_cast<float>((reinterpret_cast<const T *>(a.v) + b * a.stride[4] + j * a.stride[5] + static_cast<size_t>(g) * D)[lane * E + e]);
        }
        key(x[0], x[1]);
    }
    if (bad_page && lane == 0) atomicOr(a.status, SPEC_DEV_BAD_PAGE);
    T *out = reinterpret_cast<T *>(a.out) + row * D + lane * E;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int e = 0; e < E; ++e) out[e] = static_cast<T>(o[e] * inv);
    if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace context
}  // namespace spec
