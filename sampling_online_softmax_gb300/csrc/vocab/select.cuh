// select.cuh -- rows of logits kept on the chip: filtered sampling and the
// largest logits.
//
// One thread-block cluster per row.  The row's 16-byte vectors are dealt out to the
// cluster's CTAs in contiguous parts, which stay in shared memory, so HBM is read
// once however many passes the choice takes; what the CTAs have to know of one
// another (the maximum, sums, histograms) goes through distributed shared memory.
#pragma once

#include "cluster.cuh"
#include "rows.h"
#include "weight.cuh"

namespace spec {
namespace vocab {

constexpr int kWarps = kThreads / 32;
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kBinsPerThread = kBins / kThreads;
constexpr uint32_t kAll = 0xffffffffu;
static_assert(kBinsPerThread == 4, "a thread reads its bins of a peer as one 16-byte vector of counts");

// Whole-number keys in the order of the logits (equal for -0 and +0), and back.
__device__ __forceinline__ uint32_t order_key(float l) {
    const int b = __float_as_int(l + 0.f);
    return static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

struct alignas(16) SelectShared {
    unsigned long long mass[kBins];        // histogram: weights
    uint32_t count[kBins];                 // and counts
    unsigned long long list[kMaxList];     // the leader's list: (~key << 32) | index
    unsigned long long slot[2][kMaxCluster];
    unsigned long long seg[2][kMaxCluster * kWarps];
    unsigned long long red[kWarps];
    unsigned long long above;              // a crossing: what lies above its bin,
    uint32_t cross_bin;                    // and the bin (kAll: none)
    uint32_t list_n;
    uint32_t tie_index;
    float2 pow2[kPow2Steps];
};

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += t;
    }
    return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int EB>
struct Row {
    static constexpr int kPer = 16 / EB;  // logits per 16-byte vector
    static constexpr uint32_t kLowest = EB == 2 ? 0x0080u : 0x00800000u;  // the key of the lowest finite logit
    const uint4 *data;  // this CTA's part: n vectors, the row's vectors first .. first + n - 1
    int n, first, lead;  // lead: logits of the row's first vector that belong to the row before
    int tid, lane, warp;
    uint32_t rank, cs;
    int turn;  // which half of the exchange buffers comes next
    SelectShared *sh;

    static __device__ __forceinline__ uint32_t key(float l) { return EB == 2 ? order_key(l) >> 16 : order_key(l); }
    static __device__ __forceinline__ float value(uint32_t k) {
        return EB == 2 ? key_value((k & 0x8000u) ? k << 16 : (k << 16) | 0xffffu) : key_value(k);
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&l)[kPer]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (EB == 4) {
                l[i] = __uint_as_float(w[i]);
            } else {
                l[2 * i] = __uint_as_float(w[i] << 16);
                l[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ int index(int i, int q) const { return (first + i) * kPer + q - lead; }

    // The part of row b, in shared memory, with -inf in place of what lies outside the row.
    __device__ void load(const RowArgs &a, int b, uint4 *buf) {
        const size_t row_bytes = static_cast<size_t>(a.V) * EB;
        const unsigned char *row = a.base + static_cast<size_t>(b) * row_bytes;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
        const unsigned char *win = row - off;
        const int total = static_cast<int>((off + row_bytes + 15) >> 4);
        lead = off / EB;
        first = static_cast<int>(rank) * a.part;
        n = max(0, min(a.part, total - first));
        data = buf;
        for (int i = tid; i < n; i += kThreads) {
            const unsigned char *src = win + (static_cast<size_t>(first + i) << 4);
            if (src >= a.base && src + 16 <= a.end) copy16(smem_u32(buf + i), src);
        }
        copies_commit();
        copies_wait<0>();
        // the row's first and last vector: by logit where the vector leaves the tensor, -inf outside the row
        for (int i = tid; i < n; i += kThreads) {
            const int j = first + i;
            if (j != 0 && j != total - 1) continue;
            const unsigned char *src = win + (static_cast<size_t>(j) << 4);
            const bool whole = src >= a.base && src + 16 <= a.end;
            for (int q = 0; q < kPer; ++q) {
                const int x = index(i, q);
                const bool in = x >= 0 && x < a.V;
                if (EB == 4) {
                    uint32_t *d = reinterpret_cast<uint32_t *>(buf + i) + q;
                    if (!in)
                        *d = 0xff800000u;
                    else if (!whole)
                        *d = *reinterpret_cast<const uint32_t *>(src + 4 * q);
                } else {
                    uint16_t *d = reinterpret_cast<uint16_t *>(buf + i) + q;
                    if (!in)
                        *d = 0xff80u;
                    else if (!whole)
                        *d = *reinterpret_cast<const uint16_t *>(src + 2 * q);
                }
            }
        }
    }

    // f(logit, index) for every logit of the part, a thread's own vectors.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int i = tid; i < n; i += kThreads) {
            float l[kPer];
            unpack(data[i], l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) f(l[q], index(i, q));
        }
    }

    // The sum of v over every thread of the cluster.
    __device__ unsigned long long sum(unsigned long long v) {
        v = warp_sum(v);
        if (lane == 0) sh->red[warp] = v;
        __syncthreads();
        if (warp == 0) {
            v = warp_sum(lane < kWarps ? sh->red[lane] : 0ull);
            if (lane < static_cast<int>(cs)) st_peer(peer(&sh->slot[turn][rank], lane), v);
        }
        cluster_sync();
        v = 0;
        for (uint32_t r = 0; r < cs; ++r) v += sh->slot[turn][r];
        turn ^= 1;
        return v;
    }

    // The largest logit of the row, NaN if there is one.
    __device__ float maximum() {
        float m = -INFINITY;
        each([&](float l, int) { m = max_nan(m, l); });
#pragma unroll
        for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, o));
        if (lane == 0) sh->red[warp] = __float_as_uint(m);
        __syncthreads();
        if (warp == 0) {
            m = lane < kWarps ? __uint_as_float(static_cast<uint32_t>(sh->red[lane])) : -INFINITY;
#pragma unroll
            for (int o = 16; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(kAll, m, o));
            if (lane < static_cast<int>(cs))
                st_peer(peer(&sh->slot[turn][rank], lane), static_cast<unsigned long long>(__float_as_uint(m)));
        }
        cluster_sync();
        m = -INFINITY;
        for (uint32_t r = 0; r < cs; ++r) m = max_nan(m, __uint_as_float(static_cast<uint32_t>(sh->slot[turn][r])));
        turn ^= 1;
        return m;
    }

    // Where, in the order of falling keys, the running sum of weigh(logit, index) over the keys
    // in [lo, hi] reaches target: *key, and *above, the sum over the keys above it.  False if it
    // never does.  Each step counts the keys left into 2048 equal bins and goes on inside the one
    // that crosses: 3 steps from 32 bits, 2 from 16.  COUNT: weigh gives 0 or 1.
    template <bool COUNT, class F>
    __device__ bool reach(uint32_t lo, uint32_t hi, unsigned long long target, F weigh, uint32_t *at, unsigned long long *above) {
        unsigned long long over = 0;
        for (;;) {
            const uint32_t range = hi - lo;
            const int s = max(0, 32 - __clz(range) - kBinBits);
            for (int i = tid; i < kBins; i += kThreads) {
                if (COUNT)
                    sh->count[i] = 0;
                else
                    sh->mass[i] = 0;
            }
            if (tid == 0) sh->cross_bin = kAll;
            __syncthreads();
            each([&](float l, int x) {
                const uint32_t k = key(l);
                if (k < lo || k > hi) return;
                const unsigned long long w = weigh(l, x);
                if (w == 0) return;
                if (COUNT)
                    atomicAdd(&sh->count[(hi - k) >> s], 1u);
                else
                    atomicAdd(&sh->mass[(hi - k) >> s], w);
            });
            cluster_sync();
            unsigned long long v[kBinsPerThread] = {};
            for (uint32_t r = 0; r < cs; ++r) {
                if (COUNT) {
                    const uint4 c = ld_peer4(peer(&sh->count[tid * kBinsPerThread], r));
                    v[0] += c.x, v[1] += c.y, v[2] += c.z, v[3] += c.w;
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 c = ld_peer4(peer(&sh->mass[tid * kBinsPerThread + 2 * h], r));
                        v[2 * h] += c.x | static_cast<unsigned long long>(c.y) << 32;
                        v[2 * h + 1] += c.z | static_cast<unsigned long long>(c.w) << 32;
                    }
                }
            }
            const unsigned long long mine = v[0] + v[1] + v[2] + v[3];
            const unsigned long long incl = warp_scan(mine, lane);
            if (lane == 31) sh->red[warp] = incl;
            __syncthreads();
            unsigned long long run = over + incl - mine;
            for (int w = 0; w < warp; ++w) run += sh->red[w];
#pragma unroll
            for (int i = 0; i < kBinsPerThread; ++i) {
                if (run < target && run + v[i] >= target) {
                    sh->cross_bin = tid * kBinsPerThread + i;
                    sh->above = run;
                }
                run += v[i];
            }
            cluster_sync();  // the crossing is known, and the peers have read this histogram
            const uint32_t bin = sh->cross_bin;
            if (bin == kAll) return false;
            over = sh->above;
            hi -= bin << s;
            const uint32_t width = (1u << s) - 1;
            if (hi - lo > width) lo = hi - width;
            if (s == 0) break;
            __syncthreads();  // cross_bin is reset by the next step
        }
        *at = hi;
        *above = over;
        return true;
    }

    // The first index, in index order, at which the running sum of weigh(logit, index) reaches
    // target: found(index) is called by the one thread of the cluster that holds it.
    template <class F, class G>
    __device__ void locate(unsigned long long target, F weigh, G found) {
        const int per = (n + kWarps - 1) / kWarps;
        const int s0 = min(n, warp * per), s1 = min(n, s0 + per);
        unsigned long long v = 0;
        for (int i = s0 + lane; i < s1; i += 32) {
            float l[kPer];
            unpack(data[i], l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) v += weigh(l[q], index(i, q));
        }
        v = warp_sum(v);
        const uint32_t me = rank * kWarps + warp;
        if (lane < static_cast<int>(cs)) st_peer(peer(&sh->seg[turn][me], lane), v);
        cluster_sync();
        unsigned long long before = 0;
        for (uint32_t g = lane; g < me; g += 32) before += sh->seg[turn][g];
        before = warp_sum(before);
        turn ^= 1;
        if (before >= target || before + v < target) return;  // the whole warp
        for (int base = s0; base < s1; base += 32) {
            const int i = base + lane;
            float l[kPer];
            unsigned long long w[kPer], mine = 0;
            if (i < s1) unpack(data[i], l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                w[q] = i < s1 ? weigh(l[q], index(i, q)) : 0ull;
                mine += w[q];
            }
            const unsigned long long incl = before + warp_scan(mine, lane);
            const uint32_t hit = __ballot_sync(kAll, incl >= target);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    unsigned long long run = incl - mine;
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        if (run < target && run + w[q] >= target) found(index(i, q));
                        run += w[q];
                    }
                }
                return;
            }
            before = __shfl_sync(kAll, incl, 31);
        }
    }

    // The index of the r-th logit of key k, in index order, for every thread of the cluster.
    template <class P>
    __device__ int tie_index(uint32_t k, unsigned long long r, P also) {
        locate(r, [&](float l, int x) { return static_cast<unsigned long long>(key(l) == k && also(l, x)); },
               [&](int x) {
                   for (uint32_t p = 0; p < cs; ++p) st_peer(peer(&sh->tie_index, p), static_cast<uint32_t>(x));
               });
        cluster_sync();
        const int x = static_cast<int>(sh->tie_index);
        cluster_sync();  // read everywhere before it is written again
        return x;
    }
};

// Sorts n (a power of two) entries ascending: a bitonic network.
__device__ inline void sort_list(unsigned long long *v, int n, int tid) {
    for (int k = 2; k <= n; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            __syncthreads();
            for (int p = tid; p < n / 2; p += kThreads) {
                const int i = 2 * p - (p & (j - 1));
                const unsigned long long x = v[i], y = v[i + j];
                if ((x > y) == ((i & k) == 0)) {
                    v[i] = y;
                    v[i + j] = x;
                }
            }
        }
    }
    __syncthreads();
}

// A row's cluster: one CTA's part of it, and the row.
template <int EB>
__device__ __forceinline__ Row<EB> row_setup(const RowArgs &a, SelectShared *sh) {
    const float2 pow2[kPow2Steps] = SPEC_POW2_TABLE;
    Row<EB> r;
    r.tid = threadIdx.x;
    r.lane = threadIdx.x & 31;
    r.warp = threadIdx.x >> 5;
    r.rank = cluster_rank();
    r.cs = a.cluster;
    r.turn = 0;
    r.sh = sh;
    if (r.tid == 0) {
#pragma unroll
        for (int i = 0; i < kPow2Steps; ++i) sh->pow2[i] = pow2[i];
        sh->list_n = 0;
    }
    return r;
}

}  // namespace vocab
}  // namespace spec
