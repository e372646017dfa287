// adjust.cuh -- penalties for repeated tokens, biases and grammar masks on rows of logits.
//
// A CTA takes one slice of the vocabulary of one sequence and some of its rows.  It counts the
// history once into a table of the slice in shared memory (16 bits a token where history and nodes are fewer than
// 2^15, else 32: the top bit says that the prompt holds it, the rest count the generated occurrences) and lists
// the tokens that anything may change.
// Then, a few rows at a time, it streams the slice under the mask bits, 16 bytes a load, and computes the
// listed tokens over what it streamed.  In text these are a tenth of the tokens here and there: computed
// in the stream they would cost each warp that holds one the whole arithmetic (16 sequences of 64 rows of 32000
// fp32: 156 us, against 76 us so).  The drafted tokens of a row's own path are found through a chain of
// drafted tokens at each listed token.
//
// HBM is the floor: each logit read and written once, a bit of mask a logit.  A vector whose mask lets
// nothing through is not read; in place, only what changes is touched.  512 x 9 rows of 152064 bf16 take 525 us,
// 5.3 TB/s.  Smaller calls are bound by a CTA's fixed part, a chain of trips to L2 and barriers (the tables
// cleared, the history counted, the list made) that other CTAs of the SM hide in part: 64 x 5 rows of
// 128256 bf16 with histories of 4000 take 71 us, 2.3 TB/s; one row of 32000 fp32 5 us.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "../host.h"

namespace spec {
namespace vocab {

constexpr int kAdjustThreads = 256, kAdjustResident = 4;  // threads of a CTA; CTAs of an SM, by registers (with every argument and 8192 tokens, 66 KB, three)
constexpr int kMinSlice = 1024, kMaxSlice = 8192;  // tokens of a CTA
constexpr int kAdjustRows = 4;                     // rows streamed before their listed tokens are computed

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

// Where the parts of a CTA's shared memory begin, in words; those that a call has no use for are empty.
struct AdjustShared {
    int count, bias, list, chain, before, sums, words;
    bool narrow;  // counts of 16 bits
    __host__ __device__ explicit AdjustShared(const AdjustArgs &a) {
        const bool counts = a.repetition || a.frequency || a.presence, lists = counts || a.M, paths = counts && a.nodes && a.N > 1;
        count = lists ? a.slice / 32 : 0;
        narrow = a.L + a.N < 1 << 15;
        bias = count + (counts ? a.slice / (narrow ? 2 : 1) : 0);
        chain = bias + (a.M ? a.slice / 2 : 0);
        list = chain + (paths ? a.slice / 2 : 0);  // (up to here all is zeroed)
        before = list + (lists ? a.slice / 2 : 0);
        sums = before + (paths ? (a.N + 1) / 2 : 0);
        words = sums + a.M;
    }
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
// Vectors of a slice of a row: tid + j0 and every kAdjustThreads-th from there on.
template <int EB, bool VEC, bool INPLACE, int COUNT>
struct Vectors {
    static constexpr int EPV = VEC ? 16 / EB : 1;  // tokens of a vector
    static constexpr uint32_t kAll = (1u << EPV) - 1;
    uint32_t ok[COUNT];  // a bit a token: allowed
    uint4 v[COUNT];
    size_t first;        // the slice's first byte
    int u0;              // the first vector's first token in the slice
    const uint32_t *allowed;

    __device__ __forceinline__ int token(int k) const { return u0 + k * kAdjustThreads * EPV; }
    __device__ __forceinline__ void masks(const AdjustArgs &a, size_t row, int t0, int len, int j0) {
        first = (row * a.V + t0) * EB;
        u0 = j0 * EPV - (VEC ? static_cast<int>(reinterpret_cast<uintptr_t>(a.in + first) % 16) / EB : 0);
        allowed = a.allowed ? a.allowed + row * ((a.V + 31) / 32) : nullptr;
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
            const int u = token(k), t = t0 + u, w = t >> 5;
            ok[k] = kAll;
            if (!allowed || u < 0 || u + EPV > len) continue;
            const uint32_t low = __ldg(allowed + w), high = (t & 31) + EPV > 32 ? __ldg(allowed + w + 1) : 0;
            ok[k] = __funnelshift_r(low, high, t & 31) & kAll;
        }
    }
    __device__ __forceinline__ void load(const AdjustArgs &a, int len) {
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
            const int u = token(k);
            v[k] = make_uint4(0, 0, 0, 0);
            if (u < 0 || u + EPV > len || ok[k] == 0 || (INPLACE && ok[k] == kAll)) continue;
            const unsigned char *from = a.in + first + static_cast<ptrdiff_t>(u) * EB;
            if (VEC) v[k] = *reinterpret_cast<const uint4 *>(from);
            else v[k].x = EB == 4 ? *reinterpret_cast<const uint32_t *>(from) : *reinterpret_cast<const uint16_t *>(from);
        }
    }
    __device__ __forceinline__ void store(const AdjustArgs &a, int t0, int len) {
#pragma unroll
        for (int k = 0; k < COUNT; ++k) {
            const int u = token(k);
            if (u >= len) continue;
            unsigned char *to = a.out + first + static_cast<ptrdiff_t>(u) * EB;
            if (u < 0 || u + EPV > len) {  // a vector that the slice holds in part
                for (int e = max(0, -u); e < min(EPV, len - u); ++e) {
                    const int t = t0 + u + e;
                    const bool let = !allowed || (__ldg(allowed + (t >> 5)) >> (t & 31)) & 1;
                    if (INPLACE && let) continue;
                    store_one<EB>(to + e * EB, let ? load_one<EB>(a.in + first + static_cast<ptrdiff_t>(u + e) * EB) : -INFINITY);
                }
                continue;
            }
            if (INPLACE && ok[k] == kAll) continue;
            if (ok[k] != kAll) {
                uint32_t *x = reinterpret_cast<uint32_t *>(&v[k]);
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    if ((ok[k] >> e) & 1) continue;
                    if (EB == 4) x[e] = 0xff800000u;
                    else x[e >> 1] = (e & 1) ? (x[e >> 1] & 0xffffu) | 0xff800000u : (x[e >> 1] & 0xffff0000u) | 0xff80u;
                }
            }
            if (VEC) *reinterpret_cast<uint4 *>(to) = v[k];
            else if (EB == 4) *reinterpret_cast<uint32_t *>(to) = v[k].x;
            else *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(v[k].x);
        }
    }
};

template <int EB, bool VEC, bool INPLACE>
__global__ void __launch_bounds__(kAdjustThreads, kAdjustResident) adjust_kernel(const AdjustArgs a) {
    constexpr int EPV = VEC ? 16 / EB : 1;  // tokens of a vector
    constexpr int kBatch = 4, kFix = 2;     // vectors of a row, and listed tokens, of a thread under way at once
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ int listed;
    __shared__ float slots[32];
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

    const AdjustShared at(a);
    uint32_t *touched = smem, *count = smem + at.count;  // a bit a token; a count a token, of 16 or of 32 bits
    uint16_t *bias = reinterpret_cast<uint16_t *>(smem + at.bias);    // 1 + where a token's bias is among `sums`
    float *sums = reinterpret_cast<float *>(smem + at.sums);
    const int half = at.narrow ? 1 : 0;
    const uint32_t prompt_bit = at.narrow ? 0x8000u : 0x80000000u;
    uint16_t *list = reinterpret_cast<uint16_t *>(smem + at.list);    // the tokens that are touched
    uint16_t *chain = reinterpret_cast<uint16_t *>(smem + at.chain);  // a token's last drafted node
    uint16_t *before = reinterpret_cast<uint16_t *>(smem + at.before);  // a node's predecessor in its token's chain (0: none)
    if (counts || a.M) {
        for (int i = tid; i < at.list / 4; i += kAdjustThreads) reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) listed = 0;
        __syncthreads();
    }
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
                    const int sh = half ? (u & 1) * 16 : 0;
                    if (i + k * kAdjustThreads < prompt) atomicOr(&count[u >> half], prompt_bit << sh);
                    else atomicAdd(&count[u >> half], 1u << sh);
                    atomicOr(&touched[u >> 5], 1u << (u & 31));
                }
            }
        }
        if (paths && tid < 32)  // one warp, 32 nodes at a time, in order: each node leads to the one before it of its token
            for (int m0 = 1; m0 < a.N; m0 += 32) {
                const int m = m0 + tid, t = m < a.N ? nodes[m] : -1;
                odd |= t < -1 || t >= a.V;
                const bool in = t >= t0 && t < t0 + len;
                if (!__any_sync(0xffffffffu, in)) continue;
                const uint32_t same = __match_any_sync(0xffffffffu, in ? t : -1), lower = same & ((1u << tid) - 1);
                if (in) before[m] = lower ? static_cast<uint16_t>(m0 + 31 - __clz(lower)) : chain[t - t0];
                __syncwarp();
                if (in && same >> tid == 1) {  // the last of its token
                    chain[t - t0] = static_cast<uint16_t>(m);
                    atomicOr(&touched[(t - t0) >> 5], 1u << ((t - t0) & 31));
                }
                __syncwarp();
            }
        if (s == 0) {
            if (odd) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
            if (tid == 0 && (total != total_in || prompt != prompt_in)) atomicOr(a.status, SPEC_DEV_BAD_LENGTH);
        }
    }
    if (a.M) {
        // One warp, 32 slots at a time: the first slot that names a token of the slice holds the sum, and the others' values are
        // added in slot order.  (Each slot compared with all the others: 80 x 10 rows of
        // 4797 bf16 with 89 biases 22 us, this 18.)
        const int32_t *ids = a.bias_ids + static_cast<size_t>(b) * a.M;
        const float *values = a.bias + static_cast<size_t>(b) * a.M;
        if (tid >= 32 && tid < 64) {
            const int lane = tid - 32;
            for (int i0 = 0; i0 < a.M; i0 += 32) {
                const int i = i0 + lane, t = i < a.M ? ids[i] : -1;
                if (s == 0 && (t < -1 || t >= a.V)) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
                const bool in = t >= t0 && t < t0 + len;
                if (!__any_sync(0xffffffffu, in)) continue;
                uint32_t same = __match_any_sync(0xffffffffu, in ? t : -1);
                slots[lane] = in ? values[i] : 0.0f;
                __syncwarp();
                if (in && (same & ((1u << lane) - 1)) == 0) {
                    int at_sum = bias[t - t0];
                    if (at_sum == 0) {
                        at_sum = i + 1;
                        bias[t - t0] = static_cast<uint16_t>(at_sum);
                        atomicOr(&touched[(t - t0) >> 5], 1u << ((t - t0) & 31));
                        sums[i] = slots[lane];
                        same &= same - 1;
                    }
                    float sum = sums[at_sum - 1];
                    for (; same; same &= same - 1) sum += slots[__ffs(same) - 1];
                    sums[at_sum - 1] = sum;
                }
                __syncwarp();
            }
        }
    }
    int n_listed = 0;
    if (counts || a.M) {
        __syncthreads();
        for (int i = tid; i < (len + 31) / 32; i += kAdjustThreads) {
            uint32_t w = touched[i];
            if (!w) continue;
            for (int to = atomicAdd(&listed, __popc(w)); w; w &= w - 1) list[to++] = static_cast<uint16_t>(32 * i + __ffs(w) - 1);
        }
        __syncthreads();
        n_listed = listed;
    }

    const int words = (a.V + 31) / 32, mask_words = (a.N + 31) / 32;
    const int n_end = min(a.N, (group + 1) * a.rows);
    for (int n0 = group * a.rows; n0 < n_end; n0 += kAdjustRows) {
        const int n1 = min(n_end, n0 + kAdjustRows);
        // The stream.  In place and without a mask nothing is copied.
        for (int n = n0; (!INPLACE || a.allowed) && n < n1; ++n) {
            const int most = (len + EPV - 1) / EPV + (VEC ? 1 : 0);  // vectors of a row, wherever it lies on the 16-byte grid
            for (int j0 = tid; j0 < most; j0 += kBatch * kAdjustThreads) {
                Vectors<EB, VEC, INPLACE, kBatch> x;
                x.masks(a, static_cast<size_t>(b) * a.N + n, t0, len, j0);
                x.load(a, len);
                x.store(a, t0, len);
            }
        }
        if (n_listed == 0) continue;
        __syncthreads();  // what was streamed lies under what the listed tokens get
        const int items = n_listed * (n1 - n0);
        for (int i0 = tid; i0 < items; i0 += kFix * kAdjustThreads) {
            uint32_t let[kFix];
            float x[kFix];
            int u[kFix], n[kFix];
            size_t at[kFix];
#pragma unroll
            for (int k = 0; k < kFix; ++k) {
                const int i = i0 + k * kAdjustThreads;
                let[k] = 0;
                if (i >= items) continue;
                n[k] = n0 + i / n_listed;
                u[k] = list[i % n_listed];
                const int t = t0 + u[k];
                const size_t row = static_cast<size_t>(b) * a.N + n[k];
                at[k] = (row * a.V + t) * EB;
                let[k] = a.allowed ? __ldg(a.allowed + row * words + (t >> 5)) >> (t & 31) & 1 : 1;
                x[k] = load_one<EB>(a.in + at[k]);
            }
#pragma unroll
            for (int k = 0; k < kFix; ++k) {
                if (!let[k]) continue;
                if (a.M && bias[u[k]]) x[k] = __fadd_rn(x[k], sums[bias[u[k]] - 1]);
                if (counts) {
                    const uint32_t c = half ? count[u[k] >> 1] >> ((u[k] & 1) * 16) & 0xffffu : count[u[k]];
                    uint32_t made = c & (prompt_bit - 1);
                    if (paths)
                        for (int m = chain[u[k]]; m; m = before[m])
                            made += a.mask ? (__ldg(a.mask + static_cast<size_t>(n[k]) * mask_words + (m >> 5)) >> (m & 31)) & 1 : m <= n[k];
                    if (made || c) x[k] = x[k] > 0.0f ? __fdiv_rn(x[k], r) : __fmul_rn(x[k], r);
                    if (made) x[k] = __fsub_rn(__fsub_rn(x[k], __fmul_rn(f, static_cast<float>(made))), p);
                }
                store_one<EB>(a.out + at[k], x[k]);
            }
        }
    }
}

}  // namespace vocab
}  // namespace spec
