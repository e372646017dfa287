// select.cuh -- rows of logits kept on the chip: filtered sampling and the
// largest logits.
//
// A row is read from HBM once: while it streams by, each thread keeps the maxima of
// the groups that its vectors make (about 2048 groups a row) and, where a share of
// the whole row's weight or the log-normaliser is wanted, a running exp-sum.
//
// The short way: the k-th largest of the groups' maxima is at or below the k-th
// largest logit, while few logits more than k lie at or above it (k groups hold
// them all: 1.4 k of random logits at k = 1024, 1.03 k at k = 64).  Those k groups are
// read again, from L2, into one short list of candidates, which one CTA sorts,
// weighs and cuts alone.
//
// The long way, for rows of which thousands of tokens are kept: passes over the
// row in L2.  A histogram of counts brackets the cut, a second one narrows it,
// and the few tokens left are sorted; see cut_row.  In bf16 one histogram of the
// keys is enough; see cut_by_keys.
//
// Many rows: one CTA each, several to an SM, so that some stream while others
// choose.  Few rows: a cluster shares a row through distributed shared memory.
//
// HBM bounds the stream; what follows it is latency (block and cluster barriers, one
// trip to L2, a short sort: 8 to 10 us a row on a busy SM, 6 alone), hidden where an
// SM has other rows to stream.  Measured (kernel alone, GB300): the 64 largest of 2304
// rows of 129280 bf16 134 us, 4.4 TB/s of logits; top-p over 512 such rows of 152064
// 60 us, 2.6 TB/s (all rows under way at once: stream 25 us, then tails); one row of
// 32000 fp32 10.7 us.  The long way is bound by instructions (430 a token in all), by
// their fetching and by its passes' barriers: 48 flat rows of 50257 fp32, 17000 tokens kept, 61 us.
#pragma once

#include "part.cuh"
#include "rows.h"
#include "weight.cuh"

namespace spec {
namespace vocab {

constexpr int kWarps = kThreads / 32;
constexpr int kBinBits = 11;
constexpr int kBins = 1 << kBinBits;
constexpr int kBinsPerThread = kBins / kThreads;
constexpr int kCutBins = 512;                    // bins of cut_row's histograms
constexpr int kCutPerThread = kCutBins / kThreads;
constexpr int kTally = 4096;                     // bins of cut_by_keys' histogram, a bf16 key each
constexpr int kGroups = kMaxCluster * kThreads;  // groups of a row's logits, whatever the cluster's size
constexpr int kKeysPerThread = kGroups / kThreads;
constexpr int kWhole = 128;                      // rows up to this long are listed whole
constexpr int kGoal0 = 64, kGoal1 = 256;         // candidates asked for where top-p alone limits, one after the
constexpr int kMaxGoal = 1024, kGoals = 3;       // other (64 sort in a third of the time that 256 take), at most
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
        uint32_t tally[kTally];
        unsigned long long list[kMaxList];     // (~key << 32) | index
    };
    union {
        unsigned long long cum[kMaxList];      // the leader's: running sums of the sorted list's weights
        uint16_t hit[kGroups];                 // this CTA's groups that reach a bound
        uint32_t scratch[kBins];               // sort_list's
        uint32_t whole[kTally];                // the row's tally
    };
    uint32_t maxima[kGroups];                  // keys of the groups' maxima, the whole row's
    unsigned long long seg[2][kMaxCluster * kWarps], seg2[2][kMaxCluster * kWarps];
    uint32_t hits[kGoals][kMaxCluster * kWarps];    // candidates of each warp of the cluster
    unsigned long long red[kWarps];
    unsigned long long above;                  // a crossing: what lies above its bin,
    uint32_t cross_bin, cross_last;            // and the bin (kAll: none), or the last it may be in
    uint32_t list_n[kGoals];
    uint32_t hit_n;
    uint32_t tie_index;
    uint32_t cut[2];                           // a cut's key and index
    uint32_t verdict;
    uint32_t drawn;                            // a sure draw by near sums (kAll: none)
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
// Sum over the block of v.
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, unsigned long long *red, int lane, int warp) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w];
    return v;
}

template <int EB>
struct Row {
    using P = Part<EB>;
    static constexpr int kPer = P::kPer;
    static constexpr uint32_t kLowest = EB == 2 ? 0x0080u : 0x00800000u;  // the key of the lowest finite logit
    P part;
    int n;              // this CTA's vectors
    int tid, lane, warp;
    uint32_t rank, cs;
    int per;            // groups per thread: a thread's vectors i = tid + r kThreads of equal r mod per
    int turn;           // which half of the exchange buffers comes next
    bool used;          // sh->steps has been
    SelectShared *sh;

    static __device__ __forceinline__ uint32_t key(float l) { return EB == 2 ? order_key(l) >> 16 : order_key(l); }
    static __device__ __forceinline__ float value(uint32_t k) {
        return EB == 2 ? key_value((k & 0x8000u) ? k << 16 : (k << 16) | 0xffffu) : key_value(k);
    }
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&l)[kPer]) { P::unpack(v, l); }
    __device__ __forceinline__ int index(int i, int q) const { return part.index(i, q); }
    // A barrier of all threads that work on the row.
    __device__ __forceinline__ void sync() const {
        if (cs == 1)
            __syncthreads();
        else
            cluster_sync();
    }

    static __device__ __forceinline__ float vector_max(const uint4 &v) { return P::vector_max(v); }
    // 2^(l c - q) of two logits; adds weight times exponent to `b`.
    template <bool BOUND>
    static __device__ __forceinline__ unsigned long long exp_pair(float l0, float l1, unsigned long long c2, unsigned long long q2,
                                                                  unsigned long long &b) {
        const unsigned long long x = fma2(pair(l0, l1), c2, q2);
        float x0, x1;
        split(x, x0, x1);
        const unsigned long long w = pair(ptx::ex2(x0), ptx::ex2(x1));
        if (BOUND) b = fma2(w, pair(fmaxf(x0, -200.f), fmaxf(x1, -200.f)), b);  // (a masked logit's is -inf)
        return w;
    }
    template <bool BOUND>
    static __device__ __forceinline__ unsigned long long vector_exp(const uint4 &v, unsigned long long c2, unsigned long long q2,
                                                                    unsigned long long &b) {
        float l[kPer];
        unpack(v, l);
        unsigned long long s = add2(exp_pair<BOUND>(l[0], l[1], c2, q2, b), exp_pair<BOUND>(l[2], l[3], c2, q2, b));
        if (kPer == 8) s = add2(s, add2(exp_pair<BOUND>(l[4 % kPer], l[5 % kPer], c2, q2, b), exp_pair<BOUND>(l[6 % kPer], l[7 % kPer], c2, q2, b)));
        return s;
    }

    // Reads the part; then the largest logit of the row (returned; NaN if there is one), the keys of
    // the groups' maxima in sh->maxima of every CTA, and with kSum what exp_total() takes: a sum s of
    // 2^x, x = l c - q, for every warp, its q, and (kBounded) b, the sum of 2^x |x|, for the error.  q is a rounded
    // maximum times c and counts as exact, so a term is off by 2.25 |x| 2^-24 ln 2 (x, c and its log2 e round) + 2^-22
    // (ex2) relative; rebasing a sum to a larger q by (6 + |change|) 2^-24, which counts as 4 more of
    // |x|; and the sums by 2 + 3 (trees), 2 (pairs of floats), 5 + 5 levels of 2^-24.
    enum Sums : int { kNone = 0, kSum = 1, kBounded = 2 };  // kBounded: b too
    static constexpr int kStream = 8;  // vectors of a batch: one of each group
    __device__ __forceinline__ void load(int i0, uint4 (&v)[kStream]) const {
        if (i0 > 0 && i0 + (kStream - 1) * kThreads < n - 1) {
            const uint4 *p = reinterpret_cast<const uint4 *>(part.at(i0));
#pragma unroll
            for (int j = 0; j < kStream; ++j) v[j] = __ldg(p + j * kThreads);
        } else {  // the row's first and last vectors may hold a neighbour's logits
#pragma unroll
            for (int j = 0; j < kStream; ++j) {
                const int i = i0 + j * kThreads;
                v[j] = nothing();
                if (i < n) v[j] = part.fetch(i);
            }
        }
    }
    // v: load(tid), ahead of what the caller waits for.
    template <int SUM>
    __device__ __forceinline__ float stream(float c, uint4 (&v)[kStream]) {
        constexpr int kBatch = kStream;
        static_assert(kBatch == kMaxCluster, "a batch's vectors are one of each group");
        float g[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) g[j] = -INFINITY;
        float top = -INFINITY, q = -INFINITY;
        unsigned long long s = pair(0.f, 0.f), less = s, b = s;  // the sum, its rounding errors, the exponents'
        const unsigned long long c2 = pair(c, c);
        auto take = [&](const uint4(&v)[kBatch]) {
            float m = -INFINITY;
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float x = vector_max(v[j]);
                g[j] = max_nan(g[j], x);
                if (SUM) m = fmaxf(m, x);
            }
            if (SUM) {
                if (m > top) {
                    // (the rounded product, as it is subtracted below: not to be fused into q - to)
                    const float to = __fmul_rn(m, c), f = top > -INFINITY ? ptx::ex2(q - to) : 0.f, d = top > -INFINITY ? q - to - 4.f : 0.f;
                    const unsigned long long none = pair(0.f, 0.f), f2 = pair(f, f);
                    if (SUM == kBounded) b = fma2(fma2(s, pair(d, d), b), f2, none);
                    s = fma2(s, f2, none);
                    less = fma2(less, f2, none);
                    top = m;
                    q = to;
                }
                if (top > -INFINITY) {
                    const unsigned long long q2 = pair(-q, -q);
                    unsigned long long t[kBatch];
#pragma unroll
                    for (int j = 0; j < kBatch; ++j) t[j] = vector_exp<SUM == kBounded>(v[j], c2, q2, b);
#pragma unroll
                    for (int h = kBatch / 2; h; h >>= 1)
#pragma unroll
                        for (int j = 0; j < h; ++j) t[j] = add2(t[j], t[j + h]);
                    const unsigned long long minus = pair(-1.f, -1.f), sum = add2(s, t[0]);  // TwoSum, s or t larger
                    const unsigned long long bb = fma2(s, minus, sum);
                    less = add2(less, add2(fma2(fma2(bb, minus, sum), minus, s), fma2(bb, minus, t[0])));
                    s = sum;
                }
            }
        };
        for (int i0 = tid; i0 < n;) {
            take(v);
            i0 += kBatch * kThreads;
            if (i0 < n) load(i0, v);
        }
        if (per <= 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) g[j] = max_nan(g[j], g[j + 4]);
        }
        if (per <= 2) g[0] = max_nan(g[0], g[2]), g[1] = max_nan(g[1], g[3]);
        if (per <= 1) g[0] = max_nan(g[0], g[1]);
        unsigned long long warp_sums = 0;
        float warp_bound = 0.f;
        if (SUM) {
            float Q = q;
#pragma unroll
            for (int o = 16; o; o >>= 1) Q = fmaxf(Q, __shfl_xor_sync(kAll, Q, o));
            float x, y;
            split(s, x, y);
            float e0, e1, b0, b1;
            split(less, e0, e1);
            split(b, b0, b1);
            const float f = q > -INFINITY ? ptx::ex2(q - Q) : 0.f, d = q > -INFINITY ? 4.f + Q - q : 0.f;
            x = (x + y) + (e0 + e1);
            y = (x * d - (b0 + b1)) * f;
            x *= f;
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                x += __shfl_xor_sync(kAll, x, o);
                y += __shfl_xor_sync(kAll, y, o);
            }
            warp_sums = pair(Q, x);
            warp_bound = y;
        }
        if (cs > 1) cluster_wait();  // the peers have started
        if (SUM && lane < static_cast<int>(cs)) {
            st_peer(peer(&sh->seg[turn][rank * kWarps + warp], lane), warp_sums);
            st_peer(peer(&sh->seg2[turn][rank * kWarps + warp], lane), static_cast<unsigned long long>(__float_as_uint(warp_bound)));
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (j < per) {
                const uint32_t k = order_key(g[j]);
                for (uint32_t p = 0; p < cs; ++p) st_peer(peer(&sh->maxima[(rank * per + j) * kThreads + tid], p), k);
            }
        }
        sync();
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
    // The row's sum of 2^(l c - *q), its q, and a bound of its error, relative, after stream<kSum or kBounded>
    // (the bound: kBounded).
    __device__ __forceinline__ float exp_total(float *q, float *off) {
        constexpr int kEach = (kMaxCluster * kWarps + 31) / 32;
        float Q = -INFINITY, s = 0.f, b = 0.f, e[kEach][3];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const uint32_t g = i * 32 + lane;
            e[i][0] = -INFINITY;
            e[i][1] = e[i][2] = 0.f;
            if (g < cs * kWarps) {
                split(sh->seg[turn][g], e[i][0], e[i][1]);
                e[i][2] = __uint_as_float(static_cast<uint32_t>(sh->seg2[turn][g]));
            }
            Q = fmaxf(Q, e[i][0]);
        }
        turn ^= 1;
#pragma unroll
        for (int o = 16; o; o >>= 1) Q = fmaxf(Q, __shfl_xor_sync(kAll, Q, o));
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (e[i][0] == -INFINITY) continue;
            const float f = ptx::ex2(e[i][0] - Q);
            s += e[i][1] * f;
            b += (e[i][2] + e[i][1] * (4.f + Q - e[i][0])) * f;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s += __shfl_xor_sync(kAll, s, o);
            b += __shfl_xor_sync(kAll, b, o);
        }
        *q = Q;
        *off = (1.6f * (b / s) + 24.f) * (1.01f * 0x1p-24f);
        return s;
    }
    // The smallest of the groups' maxima that is finite (the row's largest if there is no other).
    __device__ __forceinline__ float least_maximum() {
        uint32_t k = kAll;
#pragma unroll
        for (int j = 0; j < kKeysPerThread; ++j) {
            const uint32_t x = sh->maxima[j * kThreads + tid];
            if (x >= 0x00800000u) k = min(k, x);
        }
        k = __reduce_min_sync(kAll, k);
        __syncthreads();
        if (lane == 0) sh->red[warp] = k;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) k = min(k, static_cast<uint32_t>(sh->red[w]));
        return key_value(k);
    }

    // A logit that at least `goal` groups reach (so at least `goal` logits), near the goal-th largest
    // group's: the maxima are counted by their distance below the row's in steps of the key's upper
    // 16 bits, two powers of two of them first, coarser where that does not reach.  False: too few groups.
    __device__ __forceinline__ bool threshold(float m, uint32_t goal, float *at) {
        const uint32_t top = order_key(m) >> 16;
        for (int s = 0; s <= 8; s += 4) {
            if (used) {  // (the first time: cleared by row_setup)
                __syncthreads();
                sh->steps[tid] = 0;
                if (tid == 0) sh->cross_bin = kAll;
                __syncthreads();
            }
            used = true;
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

    static __device__ __forceinline__ uint4 nothing() { return P::nothing(); }
    // f(vectors, number) for the vectors of the groups whose maximum reaches `low`, spread over all
    // threads, kGather at a time, whole warps together; number(j) is vector j's (-1: none, a vector of -inf).
    // `low` is finite.
    static constexpr int kGather = 8;
    template <class F>
    __device__ __forceinline__ void gather(float low, F f) {
        const uint32_t bound = order_key(low);
        if (tid == 0) sh->hit_n = 0;
        __syncthreads();
        for (int j = 0; j < per; ++j)
            if (sh->maxima[(rank * per + j) * kThreads + tid] >= bound) sh->hit[atomicAdd(&sh->hit_n, 1u)] = static_cast<uint16_t>(j * kThreads + tid);
        __syncthreads();
        // (group, round) pairs, the rounds padded to a power of two: no division in number()
        const int rounds = max(1, ((n + kThreads - 1) / kThreads + per - 1) / per);  // vectors of a group, at most
        const int bits = 32 - __clz(rounds - 1);
        const int total = static_cast<int>(sh->hit_n) << bits;
        for (int e0 = tid; e0 - lane < total; e0 += kGather * kThreads) {
            auto number = [&](int j) {
                const int e = e0 + j * kThreads;
                if (e >= total) return -1;
                const int group = sh->hit[e >> bits];
                const int i = ((e & ((1 << bits) - 1)) * per + group / kThreads) * kThreads + group % kThreads;
                return i < n ? i : -1;
            };
            uint4 v[kGather];
#pragma unroll
            for (int j = 0; j < kGather; ++j) {
                v[j] = nothing();
                if (e0 - lane + j * kThreads < total) {  // the whole warp
                    const int i = number(j);
                    if (i >= 0) v[j] = part.fetch(i);
                }
            }
            f(v, number);
        }
        __syncwarp();
    }
    // One bit for each logit of a vector that is at least `low` (finite: elements outside the row are -inf).
    static __device__ __forceinline__ uint32_t reaching(const uint4 &v, float low) {
        if (!(vector_max(v) >= low)) return 0;
        float l[kPer];
        unpack(v, l);
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) m |= static_cast<uint32_t>(l[q] >= low) << q;
        return m;
    }
    static __device__ __forceinline__ unsigned long long entry(float l, int x) {
        return static_cast<unsigned long long>(~order_key(l)) << 32 | static_cast<uint32_t>(x);
    }
    // Appends to the leader's list, for a whole warp, the logits of the bits (bit j * kPer + q: element q
    // of vector number(j)); returns how many the warp had.
    template <class N>
    __device__ __forceinline__ uint32_t append(unsigned long long bits, int attempt, N number) {
        if (!__any_sync(kAll, bits != 0)) return 0;
        const uint32_t c = __popcll(bits);
        uint32_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += x;
        }
        const uint32_t total = __shfl_sync(kAll, incl, 31);
        uint32_t base = 0;
        if (lane == 0) base = cs == 1 ? atomicAdd(&sh->list_n[attempt], total) : atom_add_peer(peer(&sh->list_n[attempt], 0), total);
        base = __shfl_sync(kAll, base, 0) + incl - c;
        const uint32_t list = peer(sh->list, 0);
        for (; bits; bits &= bits - 1, ++base) {
            const int e = __ffsll(bits) - 1, i = number(e / kPer);
            if (base < kMaxList) st_peer(list + base * 8, entry(P::logit(part.at(i), e % kPer), index(i, e % kPer)));
        }
        __syncwarp();
        return total;
    }
    // Every logit >= low into the leader's list; returns, after a barrier of the row, how many there are.
    __device__ __forceinline__ uint32_t collect(float low, int attempt) {
        uint32_t c = 0;
        gather(low, [&](const uint4(&v)[kGather], auto number) {
            unsigned long long bits = 0;
#pragma unroll
            for (int j = 0; j < kGather; ++j) bits |= static_cast<unsigned long long>(reaching(v[j], low)) << (j * kPer);
            c += append(bits, attempt, number);
        });
        return collected(c, attempt);
    }
    __device__ __forceinline__ uint32_t collected(uint32_t c, int attempt) {
        if (lane < static_cast<int>(cs)) st_peer(peer(&sh->hits[attempt][rank * kWarps + warp], lane), c);
        sync();
        c = 0;
        for (uint32_t i = lane; i < cs * kWarps; i += 32) c += sh->hits[attempt][i];
        return __reduce_add_sync(kAll, c);
    }

    // f(vectors, the first's number) for the vectors of the part, a thread's own (i, i + kThreads,
    // ...; -inf beyond the last), kBatch at a time, whole warps together.
    static constexpr int kBatch = 4;
    template <class F>
    __device__ __forceinline__ void vectors(F f) const {
        for (int i0 = tid; i0 - lane < n; i0 += kBatch * kThreads) {
            uint4 v[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = i0 + j * kThreads;
                v[j] = nothing();
                if (i < n) v[j] = part.fetch(i);
            }
            f(v, i0);
        }
        __syncwarp();
    }
    // v[j], for loops that are not unrolled.
    static __device__ __forceinline__ uint4 pick(const uint4 (&v)[kBatch], int j) { return j == 0 ? v[0] : j == 1 ? v[1] : j == 2 ? v[2] : v[3]; }
    // f(logit, index) for every logit of the part (and for some -inf of no index).
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        vectors([&](const uint4(&v)[kBatch], int i0) {
#pragma unroll 1
            for (int j = 0; j < kBatch; ++j) {
                float l[kPer];
                unpack(pick(v, j), l);
#pragma unroll
                for (int q = 0; q < kPer; ++q) f(l[q], index(i0 + j * kThreads, q));
            }
        });
    }

    // The sums of v and w over every thread of the row.
    __device__ __forceinline__ void sum2(unsigned long long &v, unsigned long long &w) {
        v = warp_sum(v);
        w = warp_sum(w);
        if (lane < static_cast<int>(cs)) {
            st_peer(peer(&sh->seg[turn][rank * kWarps + warp], lane), v);
            st_peer(peer(&sh->seg2[turn][rank * kWarps + warp], lane), w);
        }
        sync();
        v = w = 0;
        for (uint32_t g = lane; g < cs * kWarps; g += 32) {
            v += sh->seg[turn][g];
            w += sh->seg2[turn][g];
        }
        v = warp_sum(v);
        w = warp_sum(w);
        turn ^= 1;
    }
    __device__ __forceinline__ unsigned long long sum(unsigned long long v) {
        unsigned long long none = 0;
        sum2(v, none);
        return v;
    }
    // The summed weights 2^((l - m) c) of the groups' maxima that reach `low`, roughly.
    __device__ __forceinline__ float weight_of_maxima(float m, float c, float low) {
        const uint32_t bound = order_key(low);
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kKeysPerThread; ++j) {
            const uint32_t k = sh->maxima[j * kThreads + tid];
            if (k >= bound) s += ptx::ex2((key_value(k) - m) * c);
        }
        return static_cast<float>(block_sum(__float2ull_rn(s * 0x1p24f), sh->red, lane, warp)) * 0x1p-24f;
    }

    // The row's histogram: this thread's kBinsPerThread bins, summed over the CTAs.
    template <bool COUNT>
    __device__ __forceinline__ void bins(unsigned long long (&v)[kBinsPerThread]) const {
#pragma unroll
        for (int i = 0; i < kBinsPerThread; ++i) v[i] = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {  // unrolled: the peers' loads overlap
            if (r >= cs) break;
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
    }
    // The same of cut_row's.
    __device__ __forceinline__ void cut_bins(unsigned long long (&v)[kCutPerThread]) const {
        static_assert(kCutPerThread == 2, "read as a pair");
        v[0] = v[1] = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            if (r >= cs) break;
            const uint2 c = ld_peer2(peer(&sh->count[2 * tid], r));
            v[0] += c.x, v[1] += c.y;
        }
    }
    // The block's running sum before this thread's v, and its whole sum.
    __device__ __forceinline__ unsigned long long sum_before(unsigned long long v, unsigned long long *all = nullptr) const {
        const unsigned long long incl = warp_scan(v, lane);
        __syncthreads();
        if (lane == 31) sh->red[warp] = incl;
        __syncthreads();
        unsigned long long run = incl - v, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) run += sh->red[w];
            total += sh->red[w];
        }
        if (all) *all = total;
        return run;
    }

    // Where, in the order of falling keys, the running sum of weigh(logit, index) over the keys
    // in [lo, hi] reaches target: *key, and *above, the sum over the keys above it.  False if it
    // never does.  Each step counts the keys left into 2048 equal bins and goes on inside the one
    // that crosses: 3 steps from 32 bits, 2 from 16.  COUNT: weigh gives 0 or 1.
    template <bool COUNT, class F>
    __device__ __forceinline__ bool reach(uint32_t lo, uint32_t hi, unsigned long long target, F weigh, uint32_t *at, unsigned long long *above) {
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
            sync();
            unsigned long long v[kBinsPerThread], mine = 0;
            bins<COUNT>(v);
#pragma unroll
            for (int i = 0; i < kBinsPerThread; ++i) mine += v[i];
            unsigned long long run = over + sum_before(mine);
#pragma unroll
            for (int i = 0; i < kBinsPerThread; ++i) {
                if (run < target && run + v[i] >= target) {
                    sh->cross_bin = tid * kBinsPerThread + i;
                    sh->above = run;
                }
                run += v[i];
            }
            sync();  // the crossing is known, and the peers have read this histogram
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

    // Where, in index order, the running sum of weigh(vector, number) reaches aim(the row's sum):
    // found(vector, number, the sum before it, target, ...) is called by the one thread of the row that
    // has it; with it the sums of off(), a thread's after its weights, over the runs up to and from its.  By warps over runs of the row, then by the warps of the CTA that has it over parts of that
    // run, then by one warp.
    template <class F, class O, class A, class G>
    __device__ __forceinline__ void locate(F weigh, O off, A aim, G found) {
        auto run_sum = [&](int s0, int s1) {
            unsigned long long v = 0;
            for (int i0 = s0 + lane; i0 - lane < s1; i0 += kBatch * 32) {
                uint4 w[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    w[j] = nothing();
                    if (i0 + 32 * j < s1) w[j] = part.fetch(i0 + 32 * j);
                }
#pragma unroll 1
                for (int j = 0; j < kBatch; ++j) v += weigh(pick(w, j), i0 + 32 * j);
            }
            return warp_sum(v);
        };
        const int run = (n + kWarps - 1) / kWarps;
        const unsigned long long mine = run_sum(min(n, warp * run), min(n, (warp + 1) * run));
        const unsigned long long bound = warp_sum(off());
        if (lane < static_cast<int>(cs)) {
            st_peer(peer(&sh->seg[turn][rank * kWarps + warp], lane), mine);
            st_peer(peer(&sh->seg2[turn][rank * kWarps + warp], lane), bound);
        }
        sync();
        // the runs' sums, two to a lane in order
        static_assert(kMaxCluster * kWarps == 64, "two runs a lane");
        const uint32_t g0 = 2 * lane;
        const unsigned long long a0 = g0 < cs * kWarps ? sh->seg[turn][g0] : 0ull, a1 = g0 + 1 < cs * kWarps ? sh->seg[turn][g0 + 1] : 0ull;
        const unsigned long long b = (g0 < cs * kWarps ? sh->seg2[turn][g0] : 0ull) + (g0 + 1 < cs * kWarps ? sh->seg2[turn][g0 + 1] : 0ull);
        const unsigned long long incl = warp_scan(a0 + a1, lane), b_incl = warp_scan(b, lane);
        turn ^= 1;
        const unsigned long long target = aim(__shfl_sync(kAll, incl, 31));
        const uint32_t hits = __ballot_sync(kAll, incl >= target);
        if (!hits) return;  // (no row that aims within its sum)
        const int owner = __ffs(hits) - 1;
        const unsigned long long b_upto = __shfl_sync(kAll, b_incl, owner);
        const unsigned long long b_from = __shfl_sync(kAll, b_incl, 31) - __shfl_sync(kAll, b_incl - b, owner);
        const bool second = incl - a1 < target;
        const uint32_t g = __shfl_sync(kAll, g0 + second, owner);
        unsigned long long before = __shfl_sync(kAll, incl - a1 - (second ? 0ull : a0), owner);
        if (g / kWarps != rank) return;  // the whole CTA
        int s0 = min(n, static_cast<int>(g % kWarps) * run), s1 = min(n, s0 + run);
        const int piece = (s1 - s0 + kWarps - 1) / kWarps;
        const unsigned long long part_sum = run_sum(min(s1, s0 + warp * piece), min(s1, s0 + (warp + 1) * piece));
        __syncthreads();
        if (lane == 0) sh->red[warp] = part_sum;
        __syncthreads();
        int w = 0;
        for (; w < kWarps - 1; ++w) {
            if (before + sh->red[w] >= target) break;
            before += sh->red[w];
        }
        if (w != warp) return;
        s1 = min(s1, s0 + (w + 1) * piece);
        s0 = min(s1, s0 + w * piece);
        for (int base = s0; base < s1; base += 32) {
            const int i = base + lane;
            uint4 v = nothing();
            if (i < s1) v = part.fetch(i);
            const unsigned long long x = weigh(v, i), incl = before + warp_scan(x, lane);
            const uint32_t hit = __ballot_sync(kAll, incl >= target);
            if (hit) {
                if (lane == __ffs(hit) - 1) found(v, i, incl - x, target, b_upto, b_from);
                return;
            }
            before = __shfl_sync(kAll, incl, 31);
        }
    }

    // The index of the r-th logit of key k, in index order, among those up to `last`, for every thread
    // of the row.
    __device__ __forceinline__ int tie_index(uint32_t k, unsigned long long r, int last) {
        auto is = [&](float l, int x) { return key(l) == k && x <= last; };
        const uint32_t twin = EB == 2 ? (__float_as_uint(value(k)) >> 16) * 0x10001u : 0u;
        locate(
            [&](const uint4 &v, int i) {
                unsigned long long c = 0;
                // (few vectors hold one: bf16 pairs are compared with it first, but for the two zeros)
                if (EB == 2 && k != 0x8000u && !(__vcmpeq2(v.x, twin) | __vcmpeq2(v.y, twin) | __vcmpeq2(v.z, twin) | __vcmpeq2(v.w, twin)))
                    return c;
                float l[kPer];
                unpack(v, l);
#pragma unroll
                for (int q = 0; q < kPer; ++q) c += is(l[q], index(i, q));
                return c;
            },
            []() { return 0ull; }, [&](unsigned long long) { return r; },
            [&](const uint4 &v, int i, unsigned long long before, unsigned long long target, unsigned long long, unsigned long long) {
                float l[kPer];
                unpack(v, l);
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    if (!is(l[q], index(i, q))) continue;
                    if (++before == target)
                        for (uint32_t p = 0; p < cs; ++p) st_peer(peer(&sh->tie_index, p), static_cast<uint32_t>(index(i, q)));
                }
            });
        sync();
        const int x = static_cast<int>(sh->tie_index);
        sync();  // read everywhere before it is written again
        return x;
    }
};

// ---- the leader's list: one CTA, all its threads

// Sorts n distinct entries ascending.  Up to 128: each entry's rank is counted (2 to 8 threads an
// entry).  Above: by 2048 equal steps of the upper halves' range, each entry then counts its rank in
// its own bin; a bitonic network where a bin holds too many for that (equal logits in their hundreds).
// `scratch` holds kBins counts.
__device__ inline void sort_list(unsigned long long *v, int n, uint32_t *scratch, unsigned long long *red, int tid) {
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
    constexpr int kEach = kMaxList / kThreads;
    const int lane = tid & 31, warp = tid >> 5;
    unsigned long long e[kEach];
    uint32_t least = kAll, most = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = tid + j * kThreads;
        e[j] = i < n ? v[i] : 0ull;
        if (i < n) {
            least = min(least, static_cast<uint32_t>(e[j] >> 32));
            most = max(most, static_cast<uint32_t>(e[j] >> 32));
        }
        scratch[i] = 0;
    }
    least = __reduce_min_sync(kAll, least);
    most = __reduce_max_sync(kAll, most);
    if (lane == 0) red[warp] = static_cast<unsigned long long>(least) << 32 | most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        least = min(least, static_cast<uint32_t>(red[w] >> 32));
        most = max(most, static_cast<uint32_t>(red[w]));
    }
    const float scale = 2047.f / fmaxf(static_cast<float>(most - least), 1.f);
    auto bin = [&](unsigned long long x) {
        return min(kBins - 1, static_cast<int>(static_cast<float>(static_cast<uint32_t>(x >> 32) - least) * scale));
    };
    uint32_t at[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (tid + j * kThreads < n) at[j] = atomicAdd(&scratch[bin(e[j])], 1u);
    __syncthreads();
    uint32_t own[kBinsPerThread], sum = 0, large = 0;
#pragma unroll
    for (int j = 0; j < kBinsPerThread; ++j) {
        own[j] = scratch[tid * kBinsPerThread + j];
        sum += own[j];
        large = max(large, own[j]);
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += x;
    }
    large = __syncthreads_or(large > 192);
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    uint32_t run = incl - sum;
    for (int w = 0; w < warp; ++w) run += static_cast<uint32_t>(red[w]);
    if (!large) {
#pragma unroll
        for (int j = 0; j < kBinsPerThread; ++j) {
            scratch[tid * kBinsPerThread + j] = run;
            run += own[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (tid + j * kThreads < n) v[scratch[bin(e[j])] + at[j]] = e[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            if (tid + j * kThreads >= n) continue;
            const int b = bin(e[j]);
            const uint32_t from = scratch[b], upto = b + 1 < kBins ? scratch[b + 1] : static_cast<uint32_t>(n);
            uint32_t rank = from;
            for (uint32_t i = from; i < upto; ++i) rank += v[i] < e[j];
            at[j] = rank;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            if (tid + j * kThreads < n) v[at[j]] = e[j];
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
__device__ __forceinline__ Row<EB> row_setup(const RowArgs &a, SelectShared *sh, int b) {
    static __constant__ const float2 pow2[kPow2Steps] = SPEC_POW2_TABLE;
    Row<EB> r;
    r.tid = threadIdx.x;
    r.lane = threadIdx.x & 31;
    r.warp = threadIdx.x >> 5;
    r.cs = a.cluster;
    r.rank = r.cs == 1 ? 0u : cluster_rank();
    r.per = kMaxCluster / static_cast<int>(r.cs);
    r.turn = 0;
    r.used = false;
    r.sh = sh;
    sh->steps[r.tid] = 0;
    if (r.tid == 0) sh->cross_bin = kAll;
    if (r.tid < kPow2Steps) sh->pow2[r.tid] = pow2[r.tid];
    if (r.tid < kGoals) sh->list_n[r.tid] = 0;
    r.part.place(a.base, a.end, a.V, b, static_cast<int>(r.rank), a.part);
    r.n = r.part.n;
    return r;
}

}  // namespace vocab
}  // namespace spec
