// row_kernels.cuh -- the kernels on rows of logits and their launcher; each
// (element size, operation) is instantiated in a unit of its own (rows_*.cu).
#pragma once

#include <cfloat>
#include <climits>

#include "select.cuh"

namespace spec {
namespace vocab {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

enum Verdict : uint32_t { kDone = 0, kWeigh = 1, kMore = 2 };

// One row's request, after the checks.
struct Request {
    float p, min_p, u;
    unsigned long long least;  // the weight that min-p asks for (0: none),
    uint32_t min_key;          // or, where by_weight() is false, the least key that has it
    int k;                     // 0: no limit
};

// The smallest whole number of units that is at least f times W (f in [0, 1]), and at least 1.
__device__ __forceinline__ unsigned long long share_of(unsigned long long W, float f) {
    if (f >= 1.f) return W;
    bool rest;
    const unsigned long long t = scaled_floor(W, f, &rest);
    return max(t + (rest ? 1ull : 0ull), 1ull);
}

// Whether whole units tell which tokens min-p keeps as well as weights are known: half of one is 2^-37 of
// its weight or less.  (Smaller ones are asked about by key: rows of equal logits next to min-p would be
// kept or not by a unit's rounding, all of them alike.)
__device__ __forceinline__ bool by_weight(const Request &q) { return q.least >> 36; }
// u = 0 draws the first kept token, whatever its weight: also one below half a unit, which the whole
// numbers have as 0.  A weight that is 0 in 64 bits (below 2^-1075, which rounds to 0) is not drawn.
__device__ __forceinline__ bool drawn_at_zero(float l, const Scale &sc) { return (l - sc.m) * sc.ch > -1075.f; }

// The leader's part of a row whose kept tokens are among the n entries of its list, which holds the
// row's n largest logits: sorts them, cuts, draws.  W0, W1: bounds of the weight of all tokens that
// top-p is a share of, in units of 2^-U; 0: the list's own first k.  kWeigh: the bounds leave the
// cut open; kMore: the cut lies past the list.  need: what it has to weigh, nearly
// (0: not known); again: the list is sorted and weighed, its bounds are new.
template <int EB>
__device__ __forceinline__ Verdict draw_from_list(Row<EB> &r, const Scale &sc, const Request &q, int n, unsigned long long W0, unsigned long long W1,
                                  float need, bool again, int32_t *token) {
    SelectShared *sh = r.sh;
    const int tid = r.tid, lane = r.lane, warp = r.warp;
    if (need > 0.f) {
        float s = 0.f;
        for (int i = tid; i < n; i += kThreads) s += ptx::ex2((key_value(~static_cast<uint32_t>(sh->list[i] >> 32)) - sc.m) * sc.ch);
        if (static_cast<float>(block_sum(__float2ull_rn(s * 0x1p24f), sh->red, lane, warp)) * (1.001f * 0x1p-24f) < need) return kMore;
    }
    if (!again) sort_list(sh->list, n, sh->scratch, sh->red, tid);
    int nk = q.k > 0 ? min(n, q.k) : n;
    auto value = [&](int i) { return key_value(~static_cast<uint32_t>(sh->list[i] >> 32)); };
    auto index = [&](int i) { return static_cast<uint32_t>(sh->list[i]); };
    auto weight = [&](int i) { return sh->cum[i] - (i ? sh->cum[i - 1] : 0ull); };

    // running sums of the sorted weights, a run of entries per thread
    const int per = (nk + kThreads - 1) / kThreads;
    const int i0 = min(nk, tid * per), i1 = min(nk, i0 + per);
    if (!again) {
        unsigned long long mine = 0;
        for (int i = i0; i < i1; ++i) {
            mine += fixed_weight(value(i), sc, sh->pow2);
            sh->cum[i] = mine;
        }
        const unsigned long long before = r.sum_before(mine);
        for (int i = i0; i < i1; ++i) sh->cum[i] += before;
        __syncthreads();
    }

    if (q.p < 1.f || q.least) {
        const bool weighed = by_weight(q);
        const unsigned long long total = sh->cum[nk - 1];
        const unsigned long long t0 = share_of(W0 ? W0 : total, q.p), t1 = share_of(W1 ? W1 : total, q.p);
        unsigned long long c = 0;  // entries below the two cuts of top-p, and entries that min-p keeps
        for (int i = i0; i < i1; ++i)
            c += static_cast<unsigned long long>(sh->cum[i] < t0) | static_cast<unsigned long long>(sh->cum[i] < t1) << 16 |
                 static_cast<unsigned long long>(weighed ? weight(i) >= q.least : Row<EB>::key(value(i)) >= q.min_key) << 32;
        c = block_sum(c, sh->red, lane, warp);
        if (q.p < 1.f) {
            const int a = static_cast<int>(c & 0xffff) + 1, b = static_cast<int>((c >> 16) & 0xffff) + 1;
            if (b > nk) return kMore;
            if (a != b) return kWeigh;
            nk = a;
        }
        nk = min(nk, static_cast<int>(c >> 32));
    }
    if (nk == 1) {
        if (tid == 0) *token = static_cast<int32_t>(index(0));
        return kDone;
    }
    if (q.u == 0.f) {
        uint32_t x = kAll;
        for (int i = tid; i < nk; i += kThreads)
            if (drawn_at_zero(value(i), sc)) x = min(x, index(i));
        x = __reduce_min_sync(kAll, x);
        __syncthreads();
        if (lane == 0) sh->red[warp] = x;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kWarps; ++w) x = min(x, static_cast<uint32_t>(sh->red[w]));
            *token = static_cast<int32_t>(x);
        }
        return kDone;
    }
    bool rest;
    const unsigned long long target = scaled_floor(sh->cum[nk - 1], q.u, &rest) + 1;
    if (nk <= kThreads / 2) {  // each token's sum up to its own index, 2 to 8 threads a token
        const int each = nk <= kThreads / 8 ? 8 : nk <= kThreads / 4 ? 4 : 2;
        const int i = tid / each;
        unsigned long long s = 0;
        if (i < nk) {
            const uint32_t x = index(i);
            for (int j = tid & (each - 1); j < nk; j += each)
                if (index(j) <= x) s += weight(j);
        }
        for (int o = 1; o < each; o <<= 1) s += __shfl_xor_sync(kAll, s, o);
        if (i < nk && (tid & (each - 1)) == 0 && s >= target && s - weight(i) < target) *token = static_cast<int32_t>(index(i));
        return kDone;
    }
    // by index: (index << 32 | place in the order)
    __syncthreads();
    for (int i = tid; i < nk; i += kThreads) sh->list[i] = static_cast<unsigned long long>(index(i)) << 32 | static_cast<uint32_t>(i);
    sort_list(sh->list, nk, sh->maxima, sh->red, tid);  // (cum holds the weights; the maxima have served)
    const int pn = (nk + kThreads - 1) / kThreads;
    const int j0 = min(nk, tid * pn), j1 = min(nk, j0 + pn);
    unsigned long long s = 0;
    for (int j = j0; j < j1; ++j) s += weight(static_cast<int>(index(j)));
    unsigned long long run = r.sum_before(s);
    for (int j = j0; j < j1; ++j) {
        const unsigned long long w = weight(static_cast<int>(index(j)));
        if (run < target && run + w >= target) *token = static_cast<int32_t>(sh->list[j] >> 32);
        run += w;
    }
    return kDone;
}

// What a row keeps: the keys above `key`, and of that key the indices up to `index`.
struct Cut {
    uint32_t key;
    int index;
};

// Weights of a vector's kept tokens.  Near: 2^((l - m) c) by ex2, off by at most
//   3.25 2^-24 |x| ln 2 (difference, product, c and its log2 e round) + 2^-22 (ex2) + 3 2^-24 (sums of eight)
// relative, which bound() adds up; in units of 2^-40.  Exact: fixed_weight, in units of 2^-U.
template <int EB>
struct Weigh {
    static constexpr int kPer = Row<EB>::kPer;
    static constexpr float kPerBit = 2.3f * 0x1p-24f, kFlat = 7.5f * 0x1p-24f;
    const Scale &sc;
    const float2 *pow2;
    float floor;
    int last;

    __device__ __forceinline__ Weigh(const Scale &s, const float2 *p, const Cut &cut) : sc(s), pow2(p) {
        floor = Row<EB>::value(cut.key);
        last = cut.index;
    }
    __device__ __forceinline__ bool kept(float l, int x) const { return l > floor || (l == floor && x <= last); }
    __device__ __forceinline__ float near(float l, float *b) const {
        const float x = fmaxf((l - sc.m) * sc.ch, -200.f), w = ptx::ex2(x);  // (bounded: 0 times infinity is no bound)
        *b = fmaf(w, fmaf(-x, kPerBit, kFlat), *b);
        return w;
    }
    // The sum of a vector's weights, three roundings deep.  (Sums over the row that share their tokens'
    // errors are off from one another by no more than the whole's: the cut compares A with p W.)
    static __device__ __forceinline__ float tree(const float (&w)[kPer]) {
        const float s = (w[0] + w[1]) + (w[2] + w[3]);
        return kPer == 4 ? s : s + ((w[4 % kPer] + w[5 % kPer]) + (w[6 % kPer] + w[7 % kPer]));
    }
    // The kept weights of a vector, and in *b their error's bound.
    __device__ __forceinline__ unsigned long long near_sum(const Row<EB> &r, const uint4 &v, int i, float *b) const {
        if (!(Row<EB>::vector_max(v) >= floor)) return 0ull;
        float l[kPer];
        Row<EB>::unpack(v, l);
#pragma unroll
        for (int q = 0; q < kPer; ++q) l[q] = kept(l[q], r.index(i, q)) ? near(l[q], b) : 0.f;
        return __float2ull_rn(tree(l) * 0x1p40f);
    }
    __device__ __forceinline__ unsigned long long exact(float l, int x) const {
        const unsigned long long w = fixed_weight(l, sc, pow2);
        return kept(l, x) ? w : 0ull;
    }
    __device__ __forceinline__ unsigned long long exact_sum(const Row<EB> &r, const uint4 &v, int i) const {
        if (!(Row<EB>::vector_max(v) >= floor)) return 0ull;
        float l[kPer];
        Row<EB>::unpack(v, l);
        unsigned long long s = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) s += exact(l[q], r.index(i, q));
        return s;
    }
    // A thread's summed bound in units of 2^-40, and half a unit for each rounding to them.
    static __device__ __forceinline__ unsigned long long bound(float b, int vectors) {
        return __float2ull_ru(b * (1.001f * 0x1p40f)) + vectors;
    }
};

constexpr uint32_t kOpen = 1;  // in place of a cut's key (keys are larger): the near sums leave it open

// Where the kept tokens, in the order of falling logits, reach COUNT: the k-th; else: p times
// their weight.  False: fewer than k, or (with near sums) open.
//   1  a histogram of counts over 512 equal steps below the maximum.  A bin's weight lies between
//      its edges', 7 % apart at most, so its running sums bracket the cut's bin (COUNT: find it).
//   2  the weights above the bracket and in all, and a histogram of the bracket's inside.
//   3  the weights between, and the tokens of the narrowed bracket: a few, or equal ones, which one
//      CTA sorts and weighs.
// The sums are near ones, by ex2 with a bound of the error (about 2^-20 of the whole), at a tenth of
// the exact weights' time, where the tokens at the cut weigh enough (2^-14 of the whole) for that to
// decide which comes last in most rows; where it leaves that open the caller comes again with
// `exact`.  Where more than the list holds are left (equal logits in their thousands), reach() finds
// the cut by keys.
// (Always inlined, as all that takes a Row is: a pointer to one would keep it in memory.)
template <bool COUNT, int EB>
__device__ __forceinline__ bool cut_row(Row<EB> &r, const Scale &sc, int k, float p, bool exact, Cut *cut) {
    using W_ = Weigh<EB>;
    constexpr int kPer = Row<EB>::kPer;
    SelectShared *sh = r.sh;
    const int tid = r.tid;
    const Cut had = *cut;
    const W_ weigh(sc, sh->pow2, had);
    // 48 steps of two hold every weight that counts; narrower rows get finer bins
    const float span = fminf(48.f / sc.ch, 2.f * (sc.m - r.least_maximum()));
    const float scale = (kCutBins - 1) / fmaxf(span, 1e-30f);
    auto place = [&](float l) { return fminf((sc.m - l) * scale, 0x1.fffffep8f); };  // in bins below the maximum; < kCutBins
    auto clear = [&]() {
        r.sync();  // the histogram before this one has been read, by the peers too
        for (int i = tid; i < kCutBins; i += kThreads) sh->count[i] = 0;
        if (tid == 0) sh->cross_bin = kAll, sh->cross_last = kCutBins - 1;
        __syncthreads();
    };
    unsigned long long v[kCutPerThread];
    const int first = tid * kCutPerThread;
    const float per_bin = sc.ch / scale;
    // the weight of a logit that lies `at` bins below the maximum, in units of 2^-40
    auto edge = [&](float at) { return __float2ull_rn(ptx::ex2(-at * per_bin) * 0x1p40f); };
    // this thread's bins' weights at most and at least, their counts times their edges' give or take 2^-slack;
    // a last bin without end: 0
    auto weights = [&](float at, float step, int slack, bool endless, unsigned long long (&lo)[kCutPerThread],
                       unsigned long long (&hi)[kCutPerThread]) {
        unsigned long long e = edge(at);
#pragma unroll
        for (int i = 0; i < kCutPerThread; ++i) {
            const unsigned long long below = edge(at + static_cast<float>(i + 1) * step);
            hi[i] = v[i] * (e + (e >> slack) + 1);
            lo[i] = endless && tid == kThreads - 1 && i == kCutPerThread - 1 ? 0ull : v[i] * (below - (below >> slack));
            e = below;
        }
    };
    // the bin of the histogram in which the count from `over` on reaches `goal`
    auto counted = [&](unsigned long long over, unsigned long long goal) {
        unsigned long long mine = 0;
#pragma unroll
        for (int i = 0; i < kCutPerThread; ++i) mine += v[i];
        unsigned long long run = over + r.sum_before(mine);
#pragma unroll
        for (int i = 0; i < kCutPerThread; ++i) {
            if (run < goal && run + v[i] >= goal) {
                sh->cross_bin = first + i;
                sh->above = run;
            }
            run += v[i];
        }
        __syncthreads();
    };

    clear();
    uint32_t deep = 0;  // in the last bin, which may hold most of a cold row
    r.vectors([&](const uint4(&vec)[Row<EB>::kBatch], int i0) {
#pragma unroll 1
        for (int j = 0; j < Row<EB>::kBatch; ++j) {
            const uint4 one = Row<EB>::pick(vec, j);
            if (!(Row<EB>::vector_max(one) >= weigh.floor)) continue;
            float l[kPer];
            Row<EB>::unpack(one, l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                if (!weigh.kept(l[q], r.index(i0 + j * kThreads, q))) continue;
                const int y = static_cast<int>(place(l[q]));
                if (y == kCutBins - 1)
                    ++deep;
                else
                    atomicAdd(&sh->count[y], 1u);
            }
        }
    });
    deep = __reduce_add_sync(kAll, deep);
    if (r.lane == 0 && deep) atomicAdd(&sh->count[kCutBins - 1], deep);
    r.sync();
    r.cut_bins(v);
    uint32_t b0, b1;              // the cut's bin is in [b0, b1]
    unsigned long long A = 0;     // what lies above b0
    if (COUNT) {
        counted(0, k);
        b0 = b1 = sh->cross_bin;
        if (b0 == kAll) return false;
        A = sh->above;
    } else {
        unsigned long long lo[kCutPerThread], hi[kCutPerThread], low = 0, high = 0, all_l, all_h;
        weights(static_cast<float>(first), 1.f, 12, true, lo, hi);
#pragma unroll
        for (int i = 0; i < kCutPerThread; ++i) low += lo[i], high += hi[i];
        unsigned long long run_l = r.sum_before(low, &all_l), run_h = r.sum_before(high, &all_h);
        // a bin's end lies at or past the cut where (1 - p) of what lies up to it is at least p of what lies
        // behind it (closer than its share of a sum that is known to 7 %): perhaps, and for certain
        const float rest = 1.f - p;
        uint32_t maybe = kCutBins - 1, sure = kCutBins - 1;
#pragma unroll
        for (int i = 0; i < kCutPerThread; ++i) {
            run_h += hi[i];
            run_l += lo[i];
            if (share_of(run_h, rest) >= share_of(all_l - run_l, p)) maybe = min(maybe, first + i);
            if (share_of(run_l, rest) >= share_of(all_h - run_h, p)) sure = min(sure, first + i);
        }
        maybe = __reduce_min_sync(kAll, maybe);
        sure = __reduce_min_sync(kAll, sure);
        if (r.lane == 0) atomicMin(&sh->cross_bin, maybe), atomicMin(&sh->cross_last, sure);
        __syncthreads();
        b0 = sh->cross_bin;
        b1 = sh->cross_last;
        exact |= edge(static_cast<float>(b1)) < all_l >> 14;
    }

    const float from = static_cast<float>(b0), upto = static_cast<float>(b1 + 1);
    const float fine = kCutBins / (upto - from);
    auto sub = [&](float at) { return min(kCutBins - 1, static_cast<int>((at - from) * fine)); };
    // no logit of the bracket lies below (the last bin has no end)
    const float edge_l = b1 == kCutBins - 1 ? -FLT_MAX : sc.m - upto / scale - (fabsf(sc.m) + span) * 0x1p-20f;
    unsigned long long W = 0, B = 0, target = static_cast<unsigned long long>(k);
    float b = 0.f;
    int vectors = 0;
    clear();
    r.vectors([&](const uint4(&vec)[Row<EB>::kBatch], int i0) {
#pragma unroll 1
        for (int j = 0; j < Row<EB>::kBatch; ++j) {
            const uint4 one = Row<EB>::pick(vec, j);
            const float top = Row<EB>::vector_max(one);
            if (!(top >= (COUNT ? fmaxf(weigh.floor, edge_l) : weigh.floor))) continue;
            float l[kPer], w[kPer], a[kPer];
            Row<EB>::unpack(one, l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const bool in = weigh.kept(l[q], r.index(i0 + j * kThreads, q));
                const float at = place(l[q]);
                if (!COUNT && !exact) {
                    w[q] = in ? weigh.near(l[q], &b) : 0.f;
                    a[q] = at < from ? w[q] : 0.f;
                }
                if (in && at >= from && at < upto) atomicAdd(&sh->count[sub(at)], 1u);
            }
            if (!COUNT && exact) {
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    const unsigned long long w = weigh.exact(l[q], r.index(i0 + j * kThreads, q));
                    W += w;
                    A += place(l[q]) < from ? w : 0ull;
                }
            } else if (!COUNT) {
                W += __float2ull_rn(W_::tree(w) * 0x1p40f);
                A += __float2ull_rn(W_::tree(a) * 0x1p40f);
                ++vectors;
            }
        }
    });
    if (COUNT) {
        r.sync();
    } else {
        r.sum2(W, A);
        if (!exact) B = r.sum(W_::bound(b, 2 * vectors));
        target = share_of(W, p);
    }
    r.cut_bins(v);
    uint32_t s0, s1;
    if (COUNT) {
        counted(A, target);
        s0 = s1 = sh->cross_bin;
        A = sh->above;
    } else {
        const float step = 1.f / fine;
        const int drop = exact ? sc.U - 40 : 0;  // from the sums' units to 2^-40
        const unsigned long long unit = A >> drop, aim = target >> drop, slack = B + 1;
        unsigned long long lo[kCutPerThread], hi[kCutPerThread], low = 0, high = 0;
        weights(from + static_cast<float>(first) * step, step, 14, b1 == kCutBins - 1, lo, hi);
#pragma unroll
        for (int i = 0; i < kCutPerThread; ++i) low += lo[i], high += hi[i];
        unsigned long long run_h = unit + slack + r.sum_before(high);
        unsigned long long run_l = unit + r.sum_before(low);
#pragma unroll
        for (int i = 0; i < kCutPerThread; ++i) {
            if (run_h < aim && run_h + hi[i] >= aim) sh->cross_bin = first + i;
            if (run_l < aim + slack && run_l + lo[i] >= aim + slack) sh->cross_last = first + i;
            run_h += hi[i];
            run_l += lo[i];
        }
        __syncthreads();
        s0 = sh->cross_bin == kAll ? 0u : sh->cross_bin;  // the first bin may be reached from the start
        s1 = sh->cross_last;
    }
    if (tid == 0) sh->list_n[1] = 0, sh->cut[0] = 0;
    r.sync();
    uint32_t found = 0;
    unsigned long long between = 0;
    r.vectors([&](const uint4(&vec)[Row<EB>::kBatch], int i0) {
        unsigned long long bits = 0;
#pragma unroll 1
        for (int j = 0; j < Row<EB>::kBatch; ++j) {
            const uint4 one = Row<EB>::pick(vec, j);
            const float top = Row<EB>::vector_max(one);
            if (!(top >= fmaxf(weigh.floor, edge_l))) continue;
            float l[kPer], w[kPer];
            Row<EB>::unpack(one, l);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const float at = place(l[e]);
                w[e] = 0.f;
                if (!(at >= from && at < upto) || !weigh.kept(l[e], r.index(i0 + j * kThreads, e))) continue;
                const int y = sub(at);
                if (y < static_cast<int>(s0)) {
                    if (!COUNT && !exact) w[e] = weigh.near(l[e], &b);
                    if (!COUNT && exact) between += fixed_weight(l[e], sc, weigh.pow2);
                } else if (y <= static_cast<int>(s1)) {
                    bits |= 1ull << (j * kPer + e);
                }
            }
            if (!COUNT && !exact) between += __float2ull_rn(W_::tree(w) * 0x1p40f);
        }
        found += r.append(bits, 1, [&](int j) { return i0 + j * kThreads; });
    });
    if (!COUNT) A += r.sum(between);
    const uint32_t n = r.collected(found, 1);
    if (n <= kMaxList) {
        if (r.rank == 0) {
            sort_list(sh->list, n, sh->scratch, sh->red, tid);
            const int per = (n + kThreads - 1) / kThreads;
            const int i0 = min(static_cast<int>(n), tid * per), i1 = min(static_cast<int>(n), i0 + per);
            auto weight = [&](int i) -> unsigned long long {
                if (COUNT) return 1ull;
                const unsigned long long w = fixed_weight(key_value(~static_cast<uint32_t>(sh->list[i] >> 32)), sc, weigh.pow2);
                return exact ? w : w >> (sc.U - 40);
            };
            const unsigned long long slack = !COUNT && !exact ? B + n + 2 : 0ull;
            unsigned long long mine = 0;
            for (int i = i0; i < i1; ++i) mine += weight(i);
            unsigned long long run = A + r.sum_before(mine);
            for (int i = i0; i < i1; ++i) {
                const unsigned long long w = weight(i);
                if (run < target && run + w >= target) {
                    const bool sure = run + slack < target && run + w >= target + slack;
                    const uint32_t key = Row<EB>::key(key_value(~static_cast<uint32_t>(sh->list[i] >> 32)));
                    for (uint32_t c = 0; c < r.cs; ++c) {
                        st_peer(peer(&sh->cut[0], c), !COUNT && !exact && !sure ? kOpen : key);
                        st_peer(peer(&sh->cut[1], c), static_cast<uint32_t>(sh->list[i]));
                    }
                }
                run += w;
            }
        }
        r.sync();
        const Cut c = {sh->cut[0], static_cast<int>(sh->cut[1])};
        r.sync();  // read everywhere before it is written again
        if (c.key > kOpen) {
            *cut = c;
            return true;
        }
    }
    if (!COUNT && !exact) return false;
    uint32_t at;
    unsigned long long above;
    auto each = [&](float l, int x) -> unsigned long long {
        return !weigh.kept(l, x) ? 0ull : COUNT ? 1ull : fixed_weight(l, sc, weigh.pow2);
    };
    if (!r.template reach<COUNT>(had.key, Row<EB>::key(sc.m), target, each, &at, &above)) return false;
    const unsigned long long w = COUNT ? 1ull : fixed_weight(Row<EB>::value(at), sc, weigh.pow2);
    cut->index = r.tie_index(at, (target - above + w - 1) / w, at == had.key ? had.index : INT_MAX);
    cut->key = at;
    return true;
}

// The same cut by top-p for bf16 rows, whose logits are few different ones (128 in each power of two): one
// histogram of their keys and one exact weight a key, not a token.  Its 4096 bins are the keys from the
// maximum's downwards, but for those of the 2 `skip` magnitudes next to 0 where the bins would not
// reach to weights that count.  The few tokens of these, and those below the last bin, are weighed one by
// one.  False where the cut is among them.  One row of 128256 in 8 CTAs: 10 us for the histogram, which the
// shared atomics bound (a lane a clock), 6 to merge, weigh and find, 8 for the tie; by cut_row with exact
// weights 45.
__device__ __forceinline__ bool cut_by_keys(Row<2> &r, const Scale &sc, float p, Cut *cut) {
    constexpr int kPer = Row<2>::kPer;
    SelectShared *sh = r.sh;
    const int tid = r.tid;
    const Cut had = *cut;
    const Weigh<2> weigh(sc, sh->pow2, had);
    const float span = fminf(48.f / sc.ch, 2.f * (sc.m - r.least_maximum()));
    const int top = static_cast<int>(Row<2>::key(sc.m)), end = static_cast<int>(Row<2>::key(fmaxf(sc.m - span, -FLT_MAX)));
    int skip = 0;  // magnitudes (as bf16's bits) below it, where the bins lie on both sides of 0
    if (top >= 0x8000 && end < 0x8000) {
        skip = max(0, (top - end + 2 - kTally + 1) / 2);
        if (top - 0x8000 < skip) return false;
    }
    const int last = top - 0x8000 - skip;  // the last bin above 0
    r.sync();  // the histogram before this one has been read, by the peers too
    for (int i = tid; i < kTally; i += kThreads) sh->tally[i] = 0;
    if (tid == 0) sh->cross_bin = kAll;
    __syncthreads();
    unsigned long long near = 0, deep = 0;  // the weights next to 0, and below the last bin
    r.vectors([&](const uint4(&vec)[Row<2>::kBatch], int i0) {
#pragma unroll 1
        for (int j = 0; j < Row<2>::kBatch; ++j) {
            uint4 one = Row<2>::pick(vec, j);
            if (!(Row<2>::vector_max(one) >= weigh.floor)) continue;
            uint32_t rest = 0;
#pragma unroll 1  // (the atomics set the pace)
            for (int e = 0; e < kPer; e += 2) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float l = __uint_as_float(h ? one.x & 0xffff0000u : one.x << 16);
                    const int k = static_cast<int>(Row<2>::key(l));
                    const int d = top - k - (k < 0x8000 - skip ? 2 * skip : 0);
                    const bool in = weigh.kept(l, r.index(i0 + j * kThreads, e + h)), out = d >= kTally || (k >= 0x8000 - skip && k < 0x8000 + skip);
                    if (in && !out) atomicAdd(&sh->tally[d], 1u);
                    if (in && out && (l - sc.m) * sc.ch > -60.f) rest |= 1u << (e + h);
                }
                one.x = one.y, one.y = one.z, one.z = one.w;
            }
            for (; rest; rest &= rest - 1) {
                const float x = Part<2>::logit(r.part.at(i0 + j * kThreads), __ffs(rest) - 1);
                const unsigned long long w = fixed_weight(x, sc, weigh.pow2);
                if (top - static_cast<int>(Row<2>::key(x)) - 2 * skip >= kTally)
                    deep += w;
                else
                    near += w;
            }
        }
    });
    r.sum2(near, deep);
    // Each CTA sums and weighs its share of the bins; the one that has the cut tells it to the others.
    const int per = kTally / kThreads / static_cast<int>(r.cs), base = static_cast<int>(r.rank) * per * kThreads;
    uint32_t *whole = sh->whole + tid * per;
    const int first = base + tid * per;
    for (int h = 0; h < per; h += 2) {
        uint2 v = make_uint2(0, 0);
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c) {
            if (c >= r.cs) break;
            const uint2 x = ld_peer2(peer(&sh->tally[first + h], c));
            v.x += x.x, v.y += x.y;
        }
        *reinterpret_cast<uint2 *>(whole + h) = v;
    }
    auto key_of = [&](int d) { return static_cast<uint32_t>(top - d - (d > last ? 2 * skip : 0)); };
    auto weight = [&](int d) {
        const uint32_t c = whole[d - first];
        return c ? c * fixed_weight(Row<2>::value(key_of(d)), sc, weigh.pow2) : 0ull;
    };
    unsigned long long mine = 0, all;
#pragma unroll 1
    for (int d = first; d < first + per; ++d) mine += weight(d);
    unsigned long long run = r.sum_before(mine, &all);
    if (tid < static_cast<int>(r.cs)) st_peer(peer(&sh->seg[r.turn][r.rank], tid), all);
    r.sync();
    all = near + deep;
    for (uint32_t c = 0; c < r.cs; ++c) {
        const unsigned long long x = sh->seg[r.turn][c];
        if (c < r.rank) run += x;
        all += x;
    }
    r.turn ^= 1;
    const unsigned long long target = share_of(all, p);
    if (run < target && run + mine + near >= target) {
#pragma unroll 1
        for (int d = first; d < first + per; ++d) {
            const unsigned long long w = weight(d), before = run + (d > last ? near : 0ull);
            if (before < target && before + w >= target) {
                for (uint32_t c = 0; c < r.cs; ++c) {
                    st_peer(peer(&sh->cross_bin, c), static_cast<uint32_t>(d));
                    st_peer(peer(&sh->cross_last, c), whole[d - first]);
                    st_peer(peer(&sh->above, c), target - before);
                }
            }
            run += w;
        }
    }
    r.sync();
    const uint32_t d = sh->cross_bin, count = sh->cross_last;
    if (d == kAll) return false;
    const uint32_t key = key_of(d);
    const unsigned long long w = fixed_weight(Row<2>::value(key), sc, weigh.pow2), kept = (sh->above + w - 1) / w;
    cut->index = key == had.key ? had.index : INT_MAX;
    if (kept < count) cut->index = r.tie_index(key, kept, cut->index);
    cut->key = key;
    return true;
}
__device__ __forceinline__ bool cut_by_keys(Row<4> &, const Scale &, float, Cut *) { return false; }

// The key of the least logit whose weight is at least min_p; a warp's lanes try 32 keys at a time.
// (Out of line and without the Row: rarely called, and the rest's registers and code are as without it.)
template <int EB>
__device__ __noinline__ uint32_t least_key(const Scale sc, const float2 *pow2, float min_p) {
    uint32_t lo = Row<EB>::kLowest, hi = Row<EB>::key(sc.m);  // hi's weight suffices; the answer is in [lo, hi]
    const uint32_t lane = threadIdx.x & 31;
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 32 + 1, k = min(hi, lo + lane * step);
        const uint32_t ok = __ballot_sync(kAll, weight_reaches(Row<EB>::value(k), sc, min_p, pow2));
        if (!ok) {  // above the last key tried
            lo = min(hi, lo + 31 * step + 1);
            continue;
        }
        const uint32_t j = __ffs(ok) - 1, at = min(hi, lo + j * step);
        if (j > 0) lo = min(hi, lo + (j - 1) * step + 1);
        hi = at;
        if (j == 0) break;
    }
    return hi;
}

// The long way: the kept tokens are cut out of the whole row, and the draw runs over it.
template <int EB>
__device__ __forceinline__ void draw_from_row(Row<EB> &r, const Scale &sc, const Request &q, int32_t *token) {
    constexpr int kPer = Row<EB>::kPer;
    SelectShared *sh = r.sh;
    Cut cut = {Row<EB>::kLowest, INT_MAX};
    if (q.k > 0) cut_row<true>(r, sc, q.k, 1.f, false, &cut);
    if (q.p < 1.f && !cut_by_keys(r, sc, q.p, &cut)) {
        for (int again = 0; again < 2; ++again)
            if (cut_row<false>(r, sc, 0, q.p, again, &cut)) break;
    }
    if (q.least) {
        const uint32_t x = by_weight(q) ? least_key<EB>(sc, sh->pow2, q.min_p) : q.min_key;
        if (x > cut.key) cut = {x, INT_MAX};
    }
    const Weigh<EB> weigh(sc, sh->pow2, cut);
    if (q.u == 0.f) {
        r.locate(
            [&](const uint4 &v, int i) {
                float l[kPer];
                Row<EB>::unpack(v, l);
                unsigned long long c = 0;
#pragma unroll
                for (int e = 0; e < kPer; ++e) c += weigh.kept(l[e], r.index(i, e)) && drawn_at_zero(l[e], sc);
                return c;
            },
            []() { return 0ull; }, [](unsigned long long) { return 1ull; },
            [&](const uint4 &v, int i, unsigned long long, unsigned long long, unsigned long long, unsigned long long) {
                float l[kPer];
                Row<EB>::unpack(v, l);
                int x = -1;
#pragma unroll
                for (int e = kPer - 1; e >= 0; --e)
                    if (weigh.kept(l[e], r.index(i, e)) && drawn_at_zero(l[e], sc)) x = r.index(i, e);
                *token = x;
            });
        return;
    }
    auto aim = [&](unsigned long long W) {
        bool rest;
        return scaled_floor(W, q.u, &rest) + 1;
    };
    // First by near sums.  u's place is u W - C_v: the errors of what lies up to v count (1 - u) times,
    // of what lies behind u times.  The draw is sure where it is further than that from the token's ends.
    float b = 0.f;
    int vectors = 0;
    if (r.tid == 0) sh->drawn = kAll;
    __syncthreads();
    bool counting = true;
    r.locate(
        [&](const uint4 &v, int i) {
            float more = 0.f;
            const unsigned long long w = weigh.near_sum(r, v, i, &more);
            if (counting) b += more, ++vectors;
            return w;
        },
        [&]() {
            counting = false;
            return Weigh<EB>::bound(b, vectors);
        },
        aim,
        [&](const uint4 &v, int i, unsigned long long before, unsigned long long target, unsigned long long b_upto, unsigned long long b_from) {
            float l[kPer], none = 0.f;
            Row<EB>::unpack(v, l);
            const unsigned long long off = __float2ull_ru(((1.f - q.u) * static_cast<float>(b_upto) + q.u * static_cast<float>(b_from)) * 1.001f) + kPer + 2;
            unsigned long long run = before;
            uint32_t x = kAll;
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const bool in = weigh.kept(l[e], r.index(i, e));
                const unsigned long long w = in ? __float2ull_rn(weigh.near(l[e], &none) * 0x1p40f) : 0ull;
                if (run < target && run + w >= target && target > run + off && run + w > target + off) x = static_cast<uint32_t>(r.index(i, e));
                run += w;
            }
            for (uint32_t c = 0; c < r.cs; ++c) st_peer(peer(&sh->drawn, c), x);
        });
    r.sync();
    if (sh->drawn != kAll) {
        if (r.rank == 0 && r.tid == 0) *token = static_cast<int32_t>(sh->drawn);
        return;
    }
    r.locate([&](const uint4 &v, int i) { return weigh.exact_sum(r, v, i); }, []() { return 0ull; }, aim,
             [&](const uint4 &v, int i, unsigned long long before, unsigned long long target, unsigned long long, unsigned long long) {
                 float l[kPer];
                 Row<EB>::unpack(v, l);
#pragma unroll
                 for (int e = 0; e < kPer; ++e) {
                     const unsigned long long w = weigh.exact(l[e], r.index(i, e));
                     if (before < target && before + w >= target) *token = r.index(i, e);
                     before += w;
                 }
             });
}

// Filtered sampling of row b.
template <int EB>
__device__ __forceinline__ void sample_row(const RowArgs &a, Row<EB> &r, int b) {
    SelectShared *sh = r.sh;
    uint4 first[Row<EB>::kStream];
    r.load(r.tid, first);
    Request q;
    q.u = a.u[b];
    float T = a.temperature[b];
    q.k = a.top_k ? a.top_k[b] : 0;
    q.p = a.top_p ? a.top_p[b] : 1.f;
    q.min_p = a.min_p ? a.min_p[b] : 0.f;
    q.least = 0;
    q.min_key = 0;
    const bool greedy = T == 0.f;
    const bool bad = !(greedy || (T >= kMinTemperature && T <= kMaxTemperature)) ||
                     !(greedy || (q.p >= 0.f && q.p <= 1.f && q.min_p >= 0.f && q.min_p <= 1.f && q.u >= 0.f && q.u < 1.f));
    if (bad) {
        if (r.rank == 0 && r.tid == 0) {
            a.tokens[b] = -1;
            atomicOr(a.status, SPEC_DEV_BAD_PARAM);
        }
        if (r.cs > 1) cluster_wait();
        return;
    }
    const bool one = greedy || q.k == 1;  // the argmax, whatever the other filters keep
    if (greedy) T = 1.f;
    if (q.k < 0 || q.k >= a.V) q.k = 0;
    Scale sc;
    sc.U = a.U;
    {   // log2(e) / T as a pair
        constexpr float kH = 0x1.715476p+0f, kL = 0x1.4ae0c0p-26f;
        sc.ch = kH / T;
        sc.cl = (fmaf(-sc.ch, T, kH) + kL) / T;
    }
    const bool share = q.p < 1.f && q.k == 0;  // top-p is a share of the whole row
    const bool sums = share && a.V > kWhole && !one;
    sc.m = sums ? r.template stream<Row<EB>::kBounded>(sc.ch, first) : r.template stream<Row<EB>::kNone>(sc.ch, first);
    if (!(fabsf(sc.m) < INFINITY)) {  // NaN, +inf, or nothing but -inf
        if (r.rank == 0 && r.tid == 0) {
            a.tokens[b] = -1;
            atomicOr(a.status, SPEC_DEV_NONFINITE);
        }
        return;
    }
    if (one) {  // the lowest index of the maximum: each warp's first, to the leader
        uint32_t x = kAll;
        r.gather(sc.m, [&](const uint4(&v)[Row<EB>::kGather], auto number) {
#pragma unroll
            for (int j = 0; j < Row<EB>::kGather; ++j) {
                const uint32_t m = Row<EB>::reaching(v[j], sc.m);
                if (m) x = min(x, static_cast<uint32_t>(r.index(number(j), __ffs(m) - 1)));
            }
        });
        x = __reduce_min_sync(kAll, x);
        if (r.lane == 0) st_peer(peer(&sh->hits[0][r.rank * kWarps + r.warp], 0), x);
        r.sync();
        if (r.rank == 0 && r.warp == 0) {
            x = kAll;
            for (uint32_t i = r.lane; i < r.cs * kWarps; i += 32) x = min(x, sh->hits[0][i]);
            x = __reduce_min_sync(kAll, x);
            if (r.lane == 0) a.tokens[b] = static_cast<int32_t>(x);
        }
        return;
    }
    if (q.min_p > 0.f) {
        q.least = share_of(1ull << sc.U, q.min_p);
        if (!by_weight(q)) q.min_key = least_key<EB>(sc, sh->pow2, q.min_p);
    }

    // The short way: the list holds the logits from `low` on; all: that is every token.
    float low = -FLT_MAX;
    bool all = true;
    int attempts = sums ? kGoals : 1;
    unsigned long long W0 = 0, W1 = 0;
    float need = 0.f;  // what a list has to weigh for top-p
    if (a.V > kWhole) {
        if (sums) {  // bounds of the row's weight
            float Q, off, s = r.exp_total(&Q, &off);
            const float d = fmaf(-sc.m, sc.ch, Q);
            s *= ptx::ex2(d);
            off += (fabsf(d) + 8.f) * 0x1p-24f;
            const bool sound = s >= 0.5f && s <= static_cast<float>(a.V) * 1.01f && off < 0x1p-10f;  // not: logits whose products overflow
            const float unit = bits_float((sc.U + 127) << 23);
            const unsigned long long w = __float2ull_rn(sound ? s * unit : 0.f), e = __float2ull_ru(sound ? s * off * unit : 0.f);
            W0 = sound ? w - e : 1ull;
            W1 = sound ? w + e : 1ull << 62;
            need = sound ? q.p * s : 0.f;
        }
        if (q.k > kMaxGoal || (q.k == 0 && !share && q.min_p == 0.f)) {
            attempts = 0;
        } else if (q.k > 0) {  // too few groups for it: few tokens that are not masked
            all = !r.threshold(sc.m, q.k, &low);
        } else if (!share) {   // from a little below what min-p asks for
            low = logit_under(sc.m, -log2f(q.min_p) / sc.ch);
            all = false;
        }
    }
    for (int attempt = 0; attempt < attempts; ++attempt) {
        if (sums) {
            const int goal = attempt == 0 ? kGoal0 : attempt == 1 ? kGoal1 : kMaxGoal;
            // a list of the largest n logits weighs at most n, and a little more than its groups' maxima
            if (need > 2.f * static_cast<float>(goal)) continue;
            all = !r.threshold(sc.m, goal, &low);
            if (!all && 1.15f * r.weight_of_maxima(sc.m, sc.ch, low) < need) continue;
        }
        if (all) low = -FLT_MAX;
        const bool part = share && !all;
        const uint32_t n = r.collect(low, attempt);
        if (n > kMaxList) break;
        uint32_t v = kDone;
        for (int weighed = 0; weighed < 3; ++weighed) {
            if (r.rank == 0) {
                v = draw_from_list(r, sc, q, n, part ? W0 : 0ull, part ? W1 : 0ull, part && n > kThreads / 2 && weighed == 0 ? need : 0.f,
                                   weighed > 0, a.tokens + b);
                if (part && r.tid < static_cast<int>(r.cs)) st_peer(peer(&sh->verdict, r.tid), v);
            }
            if (!part) return;
            r.sync();
            v = sh->verdict;
            if (v != kWeigh || weighed == 2) break;
            if (weighed == 0) {  // the list's weights are exact, in the leader's hands: the error is the rest's alone
                const Weigh<EB> weigh(sc, sh->pow2, Cut{Row<EB>::kLowest, INT_MAX});
                unsigned long long rest = 0, bound = 0;
                float e = 0.f;
                int vectors = 0;
                r.vectors([&](const uint4(&v)[Row<EB>::kBatch], int) {
#pragma unroll 1
                    for (int j = 0; j < Row<EB>::kBatch; ++j) {
                        float l[Row<EB>::kPer];
                        Row<EB>::unpack(Row<EB>::pick(v, j), l);
#pragma unroll
                        for (int x = 0; x < Row<EB>::kPer; ++x) l[x] = l[x] >= low || l[x] == -INFINITY ? 0.f : weigh.near(l[x], &e);
                        rest += __float2ull_rn(Weigh<EB>::tree(l) * 0x1p40f);
                        ++vectors;
                    }
                });
                bound = Weigh<EB>::bound(e, vectors);
                r.sum2(rest, bound);
                const unsigned long long listed = sh->cum[n - 1];
                W0 = listed + ((rest - min(rest, bound)) << (sc.U - 40));
                W1 = listed + ((rest + bound) << (sc.U - 40));
            } else {
                unsigned long long w = 0;
                r.each([&](float l, int) { w += fixed_weight(l, sc, sh->pow2); });
                W0 = W1 = r.sum(w);
            }
        }
        if (v == kDone) return;
    }
    draw_from_row(r, sc, q, a.tokens + b);
}

// The K largest logits of row b.
template <int EB>
__device__ __forceinline__ void top_row(const RowArgs &a, Row<EB> &r, int b) {
    SelectShared *sh = r.sh;
    const float c = kLog2e / a.temp;
    uint4 first[Row<EB>::kStream];
    r.load(r.tid, first);
    const float m = a.lse ? r.template stream<Row<EB>::kSum>(c, first) : r.template stream<Row<EB>::kNone>(c, first);
    const size_t out = static_cast<size_t>(b) * a.K;
    if (!(m < INFINITY)) {  // NaN or +inf
        if (r.rank == 0) {
            for (int i = r.tid; i < a.K; i += kThreads) {
                a.values[out + i] = NAN;
                a.ids[out + i] = -1;
            }
            if (r.tid == 0) {
                if (a.lse) a.lse[b] = NAN;
                atomicOr(a.status, SPEC_DEV_NONFINITE);
            }
        }
        return;
    }
    const bool empty = m == -INFINITY;  // every token masked: an empty list, no error
    if (a.lse) {
        float Q, off, z = -INFINITY;
        const float s = r.exp_total(&Q, &off);
        if (!empty) {
            z = fmaf(Q, kLn2, logf(s));
            if (!(fabsf(z) < INFINITY) || !(s >= 0.25f)) {  // logits whose products with c overflow
                float d = 0.f;
                r.each([&](float l, int) { d += ptx::ex2((l - m) * c); });
                z = m / a.temp + logf(static_cast<float>(r.sum(__float2ull_rn(d * 0x1p40f))) * 0x1p-40f);
            }
        }
        if (r.rank == 0 && r.tid == 0) a.lse[b] = z;
    }
    uint32_t n = 0;
    if (!empty) {
        float low = -FLT_MAX;
        if (a.V > kWhole && !r.threshold(m, a.K, &low)) low = -FLT_MAX;  // few tokens that are not masked
        n = r.collect(low, 0);
    }
    if (n > kMaxList) {  // equal logits in their thousands
        uint32_t at;
        unsigned long long above;
        Cut cut = {Row<EB>::kLowest, INT_MAX};
        if (r.template reach<true>(cut.key, Row<EB>::key(m), a.K, [](float, int) { return 1ull; }, &at, &above)) {
            cut.index = r.tie_index(at, a.K - above, INT_MAX);
            cut.key = at;
        }
        uint32_t found = 0;
        r.vectors([&](const uint4(&v)[Row<EB>::kBatch], int i0) {
            constexpr int kPer = Row<EB>::kPer;
            unsigned long long bits = 0;
#pragma unroll
            for (int j = 0; j < Row<EB>::kBatch; ++j) {
                float l[kPer];
                Row<EB>::unpack(v[j], l);
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const uint32_t y = Row<EB>::key(l[e]);
                    if (y > cut.key || (y == cut.key && r.index(i0 + j * kThreads, e) <= cut.index)) bits |= 1ull << (j * kPer + e);
                }
            }
            found += r.append(bits, 1, [&](int j) { return i0 + j * kThreads; });
        });
        n = r.collected(found, 1);
    }
    if (r.rank != 0) return;
    sort_list(sh->list, n, sh->scratch, sh->red, r.tid);
    for (int i = r.tid; i < a.K; i += kThreads) {
        const unsigned long long e = i < n ? sh->list[i] : 0ull;
        a.values[out + i] = i < n ? key_value(~static_cast<uint32_t>(e >> 32)) : -INFINITY;
        a.ids[out + i] = i < n ? static_cast<int32_t>(static_cast<uint32_t>(e)) : -1;
    }
}

template <int EB, int OP>
__global__ void __launch_bounds__(kThreads, kRowCtas) row_kernel(const RowArgs a) {
    extern __shared__ uint4 dyn[];
    SelectShared *sh = reinterpret_cast<SelectShared *>(dyn);
    const int b = blockIdx.x / a.cluster;
    Row<EB> r = row_setup<EB>(a, sh, b);
    if (r.cs > 1)
        cluster_arrive();  // the first peer access waits for it
    else
        __syncthreads();
    if (OP == kSampleRows)
        sample_row<EB>(a, r, b);
    else
        top_row<EB>(a, r, b);
}

// CTAs per row and vectors per CTA.  The largest logits: the row is shared while all CTAs run at once
// and each has 64 KB of it (16 KB where a long list is to be gathered, or the rows are few).  64 rows of 32000 fp32, us with
// 1, 2, 4, 8 CTAs a row: 8.5, 8.8, 8.7, 14.8; 1 row of 152064 bf16: 15.2, 11.7, 10.0, 9.3; the 777
// largest of 12 rows of 50257 bf16: 20.2, 16.3, 14.9, 14.3.
// Sampling, whose long way is passes over the row: shared while that leaves fewer than two CTAs an SM
// (four where no filter is given at all) and each has four vectors a thread, by 8 only where all run at
// once (a tenth of the places lie where no cluster of 8 fits).  64 rows of 152064 bf16: short way 14.1, 13.8,
// 13.8, 21.7, unfiltered 128, 74, 46, 46; 48 flat rows of 50257 fp32, all the long way: 186, 108, 75, 61; 512
// rows of 152064, short way: 61, 70, 95, 173.
inline void row_split(RowArgs *a, int EB, int sms, bool top) {
    const long long vecs = (static_cast<long long>(a->V) * EB + 14) / 16 + 1;  // at the worst alignment
    const long long B = a->B;
    int cs = 1;
    if (top) {
        while (cs < kMaxCluster && 2 * cs * B <= kRowCtas * sms && vecs / cs > (a->K > 256 || 4 * cs * B <= sms ? 1024 : 4096)) cs *= 2;
    } else {
        const bool unfiltered = !a->top_k && !a->top_p && !a->min_p;
        const long long want = (unfiltered && vecs > 8192 ? 4ll : 2ll) * sms;
        while (cs < kMaxCluster && B * cs < want && vecs / cs > 4 * kThreads && (cs < 4 || 10 * 2 * cs * B <= 9 * kRowCtas * sms)) cs *= 2;
    }
    a->cluster = cs;
    a->part = static_cast<int>((vecs + cs - 1) / cs);
}

template <int EB, int OP>
spec_status launch_rows(const RowArgs &a0, cudaStream_t stream) {
    RowArgs a = a0;
    DeviceInfo di;
    int dev = 0;
    spec_status st = device_info(&di, &dev);
    if (st != SPEC_OK) return st;
    auto kernel = row_kernel<EB, OP>;
    st = allow_max_dyn_smem(dev, reinterpret_cast<const void *>(kernel), &di);
    if (st != SPEC_OK) return st;
    row_split(&a, EB, di.sms, OP == kTopRows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(SelectShared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(SPEC_ERR_CUDA, "row kernel launch (B=%d, cluster=%d): %s", a.B, a.cluster, cudaGetErrorString(e));
    return SPEC_OK;
}

}  // namespace vocab
}  // namespace spec
