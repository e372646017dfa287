// select.cuh -- rows of logits kept on the chip: filtered sampling and the
// largest logits.
//
// One thread-block cluster per row.  The row's 16-byte vectors are dealt out to the
// cluster's CTAs in contiguous parts, which stay in shared memory, so HBM is read
// once however many passes the choice takes; what the CTAs have to know of one
// another (maxima, sums, histograms) goes through distributed shared memory.
//
// The short way (Row::threshold, Row::collect, and the leader's list): the logits
// are in about 2048 groups, a thread's own vectors, and the k-th largest of the
// groups' maxima is at or below the k-th largest logit, while few logits more than
// k lie at or above it (k groups hold them: 1.4 k of random logits at k = 1024, 1.03 k
// at k = 64).  So two cluster barriers bring every candidate for the k largest into
// one short list in the leader's shared memory, which sorts and weighs it alone.
// Only the threads whose own maximum reaches the bound look at their logits again.
//
// The long way (Row::reach, Row::locate), for rows of which thousands of tokens
// are kept: exact histograms of the whole row.
#pragma once

#include "../ptx.cuh"
#include "part.cuh"
#include "rows.h"
#include "weight.cuh"

namespace spec {
namespace vocab {

constexpr int kWarps = kThreads / 32;
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kBinsPerThread = kBins / kThreads;
constexpr int kGroups = kMaxCluster * kThreads;  // groups of a row's logits, whatever the cluster's size
constexpr int kKeysPerThread = kGroups / kThreads;
constexpr int kFirstGoal = 128;                  // candidates asked for at first where top-p alone limits,
constexpr int kMaxGoal = 1024;                   // and at most
constexpr int kSteps = kThreads;                 // bins of the groups' maxima
constexpr uint32_t kAll = 0xffffffffu;
static_assert(kBinsPerThread % 4 == 0, "a thread reads its bins of a peer in 16-byte vectors");
static_assert(kGroups <= kMaxList && kBins <= kMaxList, "overlaid in SelectShared");

// Whole-number keys in the order of the logits (equal for -0 and +0), and back.
__device__ __forceinline__ uint32_t order_key(float l) {
    const int b = __float_as_int(l + 0.f);
    return static_cast<uint32_t>(b) ^ (static_cast<uint32_t>(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

struct alignas(16) SelectShared {
    union {                                    // the long way's histogram, or the leader's list:
        unsigned long long mass[kBins];
        uint32_t count[kBins];
        unsigned long long list[kMaxList];     // (~key << 32) | index
    };
    union {
        uint32_t maxima[kGroups];              // keys of the groups' maxima, the whole row's
        unsigned long long cum[kMaxList];      // the leader's: running sums of the sorted list's weights
    };
    unsigned long long slot[2][kMaxCluster];
    unsigned long long seg[2][kMaxCluster * kWarps];
    uint32_t hits[2][kMaxCluster * kWarps];    // candidates of each warp of the cluster
    unsigned long long red[kWarps];
    unsigned long long above;                  // a crossing: what lies above its bin,
    uint32_t cross_bin;                        // and the bin (kAll: none)
    uint32_t list_n[2];
    uint32_t tie_index;
    uint32_t verdict;
    unsigned long long W[2];                   // bounds of the row's weight
    uint32_t steps[kSteps];
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
    using P = Part<EB>;
    static constexpr int kPer = P::kPer;
    static constexpr uint32_t kLowest = EB == 2 ? 0x0080u : 0x00800000u;  // the key of the lowest finite logit
    P part;
    const uint4 *data;  // this CTA's part
    int n;              // its vectors
    int tid, lane, warp;
    uint32_t rank, cs;
    int turn;           // which half of the exchange buffers comes next
    float own_max;      // the largest of this thread's vectors (tid, tid + kThreads, ...)
    SelectShared *sh;

    static __device__ __forceinline__ uint32_t key(float l) { return EB == 2 ? order_key(l) >> 16 : order_key(l); }
    static __device__ __forceinline__ float value(uint32_t k) {
        return EB == 2 ? key_value((k & 0x8000u) ? k << 16 : (k << 16) | 0xffffu) : key_value(k);
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&l)[kPer]) { P::unpack(v, l); }
    __device__ __forceinline__ int index(int i, int q) const { return part.index(i, q); }

    __device__ void start_load(const RowArgs &a, int b, uint4 *buf) {
        part.place(a.base, a.end, a.V, b, rank, a.part);
        n = part.n;
        data = buf;
        for (int i = tid; i < n; i += kThreads) part.copy(buf, i);
        copies_commit();
    }
    // The largest logit of a vector, NaN if it holds one.
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float vector_max(const uint4 &v) {
        if (EB == 2) {
            const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
            return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        }
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }

    // Waits for the part; then the largest logit of the row, NaN if there is one, and in
    // sh->maxima, in every CTA, the keys of the groups' maxima.  A thread's vectors make
    // kMaxCluster / cs groups, so that a row has kGroups of them.
    __device__ float maximum(uint4 *buf) {
        copies_wait<0>();
        constexpr int kMost = kMaxCluster;
        const int per = kMost / static_cast<int>(cs);  // groups per thread
        float g[kMost];
#pragma unroll
        for (int j = 0; j < kMost; ++j) g[j] = -INFINITY;
        for (int i0 = tid; i0 < n; i0 += kMost * kThreads) {
#pragma unroll
            for (int j = 0; j < kMost; ++j) {
                const int i = i0 + j * kThreads;
                if (i < n) {
                    part.mend(buf, i);
                    g[j] = max_nan(g[j], vector_max(buf[i]));
                }
            }
        }
        if (per <= 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = max_nan(g[j], g[j + 4]);
        }
        if (per <= 2) g[0] = max_nan(g[0], g[2]), g[1] = max_nan(g[1], g[3]);
        if (per <= 1) g[0] = max_nan(g[0], g[1]);
        own_max = -INFINITY;
        cluster_wait();  // the peers have started
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
            if (j < per) {
                own_max = max_nan(own_max, g[j]);
                const uint32_t k = order_key(g[j]);
                for (uint32_t p = 0; p < cs; ++p) st_peer(peer(&sh->maxima[(rank * per + j) * kThreads + tid], p), k);
            }
        }
        cluster_sync();
        uint32_t k = 0;
#pragma unroll
        for (int j = 0; j < kKeysPerThread; ++j) k = max(k, sh->maxima[j * kThreads + tid]);
        k = __reduce_max_sync(kAll, k);
        if (lane == 0) sh->red[warp] = k;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) k = max(k, static_cast<uint32_t>(sh->red[w]));
        return key_value(k);
    }

    // A logit that at least `goal` groups reach (so at least `goal` logits), near the goal-th largest
    // group's: the maxima are counted by their distance below the row's in steps of the key's upper
    // 16 bits, two powers of two of them first, coarser where that does not reach.  False: too few groups.
    __device__ bool threshold(float m, uint32_t goal, float *at) {
        const uint32_t top = order_key(m) >> 16;
        for (int s = 0; s <= 8; s += 4) {
            __syncthreads();
            sh->steps[tid] = 0;
            if (tid == 0) sh->cross_bin = kAll;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kKeysPerThread; ++j) {
                const uint32_t k = sh->maxima[j * kThreads + tid];
                const uint32_t d = (top - (k >> 16)) >> s;
                if (d < kSteps && k >= 0x00800000u) atomicAdd(&sh->steps[d], 1u);
            }
            __syncthreads();
            const uint32_t c = sh->steps[tid];
            uint32_t incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane == 31) sh->red[warp] = incl;
            __syncthreads();
            for (int w = 0; w < warp; ++w) incl += static_cast<uint32_t>(sh->red[w]);
            if (incl >= goal && incl - c < goal) sh->cross_bin = tid;
            __syncthreads();
            const uint32_t bin = sh->cross_bin;
            if (bin != kAll) {
                const uint32_t below = ((bin + 1) << s) - 1;  // steps below the row's maximum
                const uint32_t k16 = top > below + 0x0080u ? top - below : 0x0080u;
                *at = key_value(k16 << 16);
                return true;
            }
        }
        return false;
    }

    // sum of 2^((l - m) c) over the part, in fp32, posted by warp to every CTA in units of 2^-40;
    // exp_total() after the caller's cluster barrier.  Off by less than 2^-16 relative: 2^-22 an
    // ex2, its argument's rounding (3/2 of 2^-24 |x|, and what lies beyond |x| = 48 adds up to
    // less than 2^-29), and sums of a dozen levels.
    __device__ void exp_sum(float m, float c) {
        float s = 0.f;
        for (int i = tid; i < n; i += kThreads) {
            float l[kPer];
            unpack(data[i], l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) l[q] = ptx::ex2((l[q] - m) * c);
#pragma unroll
            for (int h = kPer / 2; h; h >>= 1)
#pragma unroll
                for (int q = 0; q < h; ++q) l[q] += l[q + h];
            s += l[0];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        const unsigned long long v = __float2ull_rn(s * 0x1p40f);
        if (lane < static_cast<int>(cs)) st_peer(peer(&sh->seg[turn][rank * kWarps + warp], lane), v);
    }
    __device__ unsigned long long exp_total() {
        unsigned long long v = 0;
        for (uint32_t i = lane; i < cs * kWarps; i += 32) v += sh->seg[turn][i];
        turn ^= 1;
        return warp_sum(v);
    }

    // Every logit >= low into the leader's list; what each warp found, into sh->hits of every
    // CTA.  The caller's cluster barrier follows.
    __device__ void collect(float low, int attempt) {
        uint32_t c = 0;
        unsigned long long h[2] = {0, 0};
        auto entry = [&](float l, int x) {
            return static_cast<unsigned long long>(~order_key(l)) << 32 | static_cast<uint32_t>(x);
        };
        const bool mine = own_max >= low;
        if (__any_sync(kAll, mine)) {
            if (mine) {
                for (int i = tid; i < n; i += kThreads) {
                    const uint4 v = data[i];
                    if (!(vector_max(v) >= low)) continue;
                    float l[kPer];
                    unpack(v, l);
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        if (l[q] >= low) {
                            const unsigned long long e = entry(l[q], index(i, q));
                            if (c == 0) h[0] = e;
                            if (c == 1) h[1] = e;
                            ++c;
                        }
                    }
                }
            }
            __syncwarp();
            uint32_t incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += x;
            }
            const uint32_t total = __shfl_sync(kAll, incl, 31);
            uint32_t base = 0;
            if (lane == 0) base = atom_add_peer(peer(&sh->list_n[attempt], 0), total);
            base = __shfl_sync(kAll, base, 0) + incl - c;
            const uint32_t list = peer(sh->list, 0);
            if (c > 0 && base < kMaxList) st_peer(list + base * 8, h[0]);
            if (c > 1 && base + 1 < kMaxList) st_peer(list + base * 8 + 8, h[1]);
            if (c > 2) {
                uint32_t at = 0;
                for (int i = tid; i < n; i += kThreads) {
                    const uint4 v = data[i];
                    if (!(vector_max(v) >= low)) continue;
                    float l[kPer];
                    unpack(v, l);
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        if (l[q] >= low) {
                            if (at >= 2 && base + at < kMaxList) st_peer(list + (base + at) * 8, entry(l[q], index(i, q)));
                            ++at;
                        }
                    }
                }
            }
            __syncwarp();
            c = total;
        }
        if (lane < static_cast<int>(cs)) st_peer(peer(&sh->hits[attempt][rank * kWarps + warp], lane), c);
    }
    // After that barrier: how many there are.
    __device__ uint32_t collected(int attempt) const {
        uint32_t c = 0;
        for (uint32_t i = lane; i < cs * kWarps; i += 32) c += sh->hits[attempt][i];
        return __reduce_add_sync(kAll, c);
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
#pragma unroll
                    for (int h = 0; h < kBinsPerThread / 4; ++h) {
                        const uint4 c = ld_peer4(peer(&sh->count[tid * kBinsPerThread + 4 * h], r));
                        v[4 * h] += c.x, v[4 * h + 1] += c.y, v[4 * h + 2] += c.z, v[4 * h + 3] += c.w;
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < kBinsPerThread / 2; ++h) {
                        const uint4 c = ld_peer4(peer(&sh->mass[tid * kBinsPerThread + 2 * h], r));
                        v[2 * h] += c.x | static_cast<unsigned long long>(c.y) << 32;
                        v[2 * h + 1] += c.z | static_cast<unsigned long long>(c.w) << 32;
                    }
                }
            }
            unsigned long long mine = 0;
#pragma unroll
            for (int i = 0; i < kBinsPerThread; ++i) mine += v[i];
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

// ---- the leader's list: one CTA, all its threads

// Sum over the block of v; red is free again after the caller's next barrier.
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long *red, int lane, int warp) {
    v = warp_sum(v);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w];
    return v;
}

// Sorts n distinct entries ascending.  Up to 128: each entry's rank is counted (2 to 8 threads an
// entry); above: a bitonic network over the next power of two.  (list holds room for it.)
__device__ inline void sort_list(unsigned long long *v, int n, int tid) {
    __syncthreads();
    if (n <= kThreads / 2) {
        const int each = n <= kThreads / 8 ? 8 : n <= kThreads / 4 ? 4 : 2;
        const int i = tid / each;
        const unsigned long long e = i < n ? v[i] : 0ull;
        int rank = 0;
        for (int j = tid & (each - 1); j < n; j += each) rank += v[j] < e;
        for (int o = 1; o < each; o <<= 1) rank += __shfl_xor_sync(kAll, rank, o);
        __syncthreads();
        if (i < n && (tid & (each - 1)) == 0) v[rank] = e;
        __syncthreads();
        return;
    }
    int size = kThreads;
    while (size < n) size <<= 1;
    for (int i = n + tid; i < size; i += kThreads) v[i] = ~0ull;
    for (int k = 2; k <= size; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            __syncthreads();
            for (int p = tid; p < size / 2; p += kThreads) {
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
        sh->list_n[0] = sh->list_n[1] = 0;
    }
    return r;
}

}  // namespace vocab
}  // namespace spec
