// adjust.cuh -- penalties for repeated tokens, biases and grammar masks on rows of logits.
//
// A CTA takes one slice of the vocabulary of one sequence and some of its rows.  It counts the
// history once into a table of the slice in shared memory (one word a token: bit 31 says that the
// prompt holds it, the rest count the generated occurrences), with a bit a token that anything may
// change.  Then it streams the slice of its rows: a 16-byte vector without such a bit is copied
// under its mask bits, the others are computed token by token.  The drafted tokens of a row's own
// path are added to the table before the row and taken out behind it, by integer atomics on shared
// memory, whose order changes nothing.
//
// Bound by HBM: each logit read and written once, a bit of mask a logit.  A vector whose mask lets
// nothing through is not read; in place, only vectors that change are touched at all.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "../host.h"

namespace spec {
namespace vocab {

constexpr int kAdjustThreads = 256;
constexpr int kMinSlice = 1024, kMaxSlice = 8192;  // tokens of a CTA

struct AdjustArgs {
    const unsigned char *in;
    unsigned char *out;
    int B, N, V, L, M;
    int slice, slices;        // tokens a slice, slices a row
    int rows, groups;         // rows a CTA, groups of rows a sequence
    const int32_t *tokens, *prompt_len, *total_len, *nodes;
    const uint32_t *mask;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_ids;
    const float *bias;
    const uint32_t *allowed;
    uint32_t *status;
};

template <int EB>
__device__ __forceinline__ float load_one(const unsigned char *p) {
    if (EB == 4) return *reinterpret_cast<const float *>(p);
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
}
template <int EB>
__device__ __forceinline__ void store_one(unsigned char *p, float x) {
    if (EB == 4) *reinterpret_cast<float *>(p) = x;
    else *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(x);
}
// EPV bits from bit `at` of a bit array that has one word to spare behind them.
template <int EPV>
__device__ __forceinline__ uint32_t bits_at(const uint32_t *words, int at) {
    return __funnelshift_r(words[at >> 5], words[(at >> 5) + 1], at & 31) & ((1u << EPV) - 1);
}

template <int EB, bool VEC, bool INPLACE>
__global__ void __launch_bounds__(kAdjustThreads) adjust_kernel(const AdjustArgs a) {
    constexpr int EPV = VEC ? 16 / EB : 1;  // tokens of a vector
    constexpr uint32_t kAll = (1u << EPV) - 1;
    constexpr int kBatch = 4;               // vectors of a thread under way at once
    extern __shared__ uint32_t smem[];
    const int tid = threadIdx.x;
    const int s = blockIdx.x % a.slices;
    const int group = blockIdx.x / a.slices % a.groups;
    const int b = blockIdx.x / a.slices / a.groups;
    const int t0 = s * a.slice, len = min(a.V - t0, a.slice);

    // the sequence's penalties; one out of range is none
    float r = a.repetition ? a.repetition[b] : 1.0f, f = a.frequency ? a.frequency[b] : 0.0f, p = a.presence ? a.presence[b] : 0.0f;
    bool bad = false;
    if (!(r > 0.0f && r < INFINITY)) r = 1.0f, bad = true;
    if (!isfinite(f)) f = 0.0f, bad = true;
    if (!isfinite(p)) p = 0.0f, bad = true;
    if (bad && tid == 0) atomicOr(a.status, SPEC_DEV_BAD_PARAM);
    const bool counts = r != 1.0f || f != 0.0f || p != 0.0f;
    const bool paths = counts && a.nodes && a.N > 1;

    uint32_t *touched = smem;                                       // slice bits and one spare word
    uint32_t *count = touched + a.slice / 32 + 1;                   // [slice], where a penalty is given
    float *bias = reinterpret_cast<float *>(count + (a.repetition || a.frequency || a.presence ? a.slice : 0));  // [slice], where M > 0
    for (int i = tid; i <= a.slice / 32; i += kAdjustThreads) touched[i] = 0;
    if (counts)
        for (int i = tid; i < len; i += kAdjustThreads) count[i] = 0;
    if (a.M)
        for (int i = tid; i < len; i += kAdjustThreads) bias[i] = 0.0f;
    __syncthreads();

    const int32_t *nodes = a.nodes ? a.nodes + static_cast<size_t>(b) * a.N : nullptr;
    if (counts) {
        int total = a.total_len ? a.total_len[b] : a.L, prompt = a.prompt_len ? a.prompt_len[b] : 0;
        const int total_in = total, prompt_in = prompt;
        total = min(max(total, 0), a.L);
        prompt = min(max(prompt, 0), total);
        bool odd = false;
        const int32_t *history = a.tokens + static_cast<size_t>(b) * a.L;
        constexpr int kAhead = 8;
        for (int i = tid; i < total; i += kAhead * kAdjustThreads) {
            int t[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) t[k] = i + k * kAdjustThreads < total ? __ldg(history + i + k * kAdjustThreads) : -1;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t u = static_cast<uint32_t>(t[k]) - t0;  // (a token below t0 wraps past the slice's end)
                odd |= t[k] < -1 || t[k] >= a.V;
                if (t[k] >= 0 && u < static_cast<uint32_t>(len)) {
                    if (i + k * kAdjustThreads < prompt) atomicOr(&count[u], 0x80000000u);
                    else atomicAdd(&count[u], 1u);
                    atomicOr(&touched[u >> 5], 1u << (u & 31));
                }
            }
        }
        if (paths)
            for (int m = 1 + tid; m < a.N; m += kAdjustThreads) {
                const int t = nodes[m];
                odd |= t < -1 || t >= a.V;
                if (t >= t0 && t < t0 + len) atomicOr(&touched[(t - t0) >> 5], 1u << ((t - t0) & 31));
            }
        if (s == 0) {
            if (odd) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
            if (tid == 0 && (total != total_in || prompt != prompt_in)) atomicOr(a.status, SPEC_DEV_BAD_LENGTH);
        }
    }
    // The first slot that names a token adds the later ones' values, in their order.
    for (int i = tid; i < a.M; i += kAdjustThreads) {
        const int32_t *ids = a.bias_ids + static_cast<size_t>(b) * a.M;
        const int t = ids[i];
        if (s == 0 && (t < -1 || t >= a.V)) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
        if (t < t0 || t >= t0 + len) continue;
        bool first = true;
        for (int k = 0; k < i && first; ++k) first = ids[k] != t;
        if (!first) continue;
        const float *values = a.bias + static_cast<size_t>(b) * a.M;
        float sum = values[i];
        for (int k = i + 1; k < a.M; ++k)
            if (ids[k] == t) sum += values[k];
        bias[t - t0] = sum;
        atomicOr(&touched[(t - t0) >> 5], 1u << ((t - t0) & 31));
    }
    __syncthreads();

    auto adjusted = [&](float x, int u) {
        if (a.M) x = __fadd_rn(x, bias[u]);
        if (counts) {
            const uint32_t c = count[u], made = c & 0x7fffffffu;
            if (c) x = x > 0.0f ? __fdiv_rn(x, r) : __fmul_rn(x, r);
            if (made) x = __fsub_rn(__fsub_rn(x, __fmul_rn(f, static_cast<float>(made))), p);
        }
        return x;
    };
    // The path's tokens of row n into the table (by 1) or out of it (by -1).
    auto path = [&](int n, uint32_t by) {
        const int words = (a.N + 31) / 32;
        for (int m = 1 + tid; m < a.N; m += kAdjustThreads) {
            const bool on = a.mask ? (__ldg(a.mask + static_cast<size_t>(n) * words + (m >> 5)) >> (m & 31)) & 1 : m <= n;
            const int t = nodes[m];
            if (on && t >= t0 && t < t0 + len) atomicAdd(&count[t - t0], by);
        }
    };

    const int words = (a.V + 31) / 32;
    const int n_end = min(a.N, (group + 1) * a.rows);
    for (int n = group * a.rows; n < n_end; ++n) {
        const size_t row = static_cast<size_t>(b) * a.N + n;
        if (paths) {
            if (n > group * a.rows) {
                __syncthreads();
                path(n - 1, ~0u);
            }
            path(n, 1u);
            __syncthreads();
        }
        const size_t first = (row * a.V + t0) * EB;  // the slice's first byte
        const int off = VEC ? static_cast<int>(reinterpret_cast<uintptr_t>(a.in + first) % 16) / EB : 0;
        const int vectors = (len + off + EPV - 1) / EPV;
        const uint32_t *allowed = a.allowed ? a.allowed + row * words : nullptr;
        for (int j0 = tid; j0 < vectors; j0 += kBatch * kAdjustThreads) {
            uint32_t ok[kBatch], hit[kBatch];
            uint4 v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int u = (j0 + k * kAdjustThreads) * EPV - off;  // the vector's first token in the slice
                ok[k] = kAll;
                hit[k] = 0;
                if (u < 0 || u + EPV > len) continue;
                hit[k] = bits_at<EPV>(touched, u);
                if (allowed) {
                    const int t = t0 + u, w = t >> 5;
                    const uint32_t low = __ldg(allowed + w), high = (t & 31) + EPV > 32 ? __ldg(allowed + w + 1) : 0;
                    ok[k] = __funnelshift_r(low, high, t & 31) & kAll;
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int u = (j0 + k * kAdjustThreads) * EPV - off;
                const bool whole = u >= 0 && u + EPV <= len;
                const bool read = whole && ok[k] != 0 && !(INPLACE && hit[k] == 0 && ok[k] == kAll);
                v[k] = make_uint4(0, 0, 0, 0);
                if (!read) continue;
                const unsigned char *at = a.in + first + static_cast<ptrdiff_t>(u) * EB;
                if (VEC) v[k] = __ldcs(reinterpret_cast<const uint4 *>(at));
                else v[k].x = EB == 4 ? *reinterpret_cast<const uint32_t *>(at) : *reinterpret_cast<const uint16_t *>(at);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int u = (j0 + k * kAdjustThreads) * EPV - off;
                if (u >= len) continue;
                unsigned char *to = a.out + first + static_cast<ptrdiff_t>(u) * EB;
                if (u < 0 || u + EPV > len) {  // a vector that the slice holds in part
                    for (int e = max(0, -u); e < min(EPV, len - u); ++e) {
                        const int t = t0 + u + e;
                        const bool let = !allowed || (__ldg(allowed + (t >> 5)) >> (t & 31)) & 1;
                        const bool touch = (touched[(u + e) >> 5] >> ((u + e) & 31)) & 1;
                        if (INPLACE && let && !touch) continue;
                        float x = -INFINITY;
                        if (let) {
                            x = load_one<EB>(a.in + first + static_cast<ptrdiff_t>(u + e) * EB);
                            if (touch) x = adjusted(x, u + e);
                        }
                        store_one<EB>(to + e * EB, x);
                    }
                    continue;
                }
                if (INPLACE && hit[k] == 0 && ok[k] == kAll) continue;
                union {
                    uint4 q;
                    uint32_t w[4];
                } x;
                x.q = v[k];
                if (hit[k] != 0 || ok[k] != kAll) {
#pragma unroll
                    for (int e = 0; e < EPV; ++e) {
                        const bool let = (ok[k] >> e) & 1, touch = (hit[k] >> e) & 1;
                        if (EB == 4) {
                            if (touch && let) x.w[e] = __float_as_uint(adjusted(__uint_as_float(x.w[e]), u + e));
                            if (!let) x.w[e] = 0xff800000u;
                        } else {
                            const int sh = (e & 1) * 16;
                            uint32_t h = (x.w[e >> 1] >> sh) & 0xffffu;
                            if (touch && let) h = __bfloat16_as_ushort(__float2bfloat16_rn(adjusted(__uint_as_float(h << 16), u + e)));
                            if (!let) h = 0xff80u;
                            x.w[e >> 1] = (x.w[e >> 1] & ~(0xffffu << sh)) | h << sh;
                        }
                    }
                }
                if (VEC) *reinterpret_cast<uint4 *>(to) = x.q;
                else if (EB == 4) *reinterpret_cast<uint32_t *>(to) = x.q.x;
                else *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(x.q.x);
            }
        }
    }
}

}  // namespace vocab
}  // namespace spec
