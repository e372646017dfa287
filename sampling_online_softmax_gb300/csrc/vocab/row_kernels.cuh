// row_kernels.cuh -- the kernels on rows of logits and their launcher; each
// (element size, operation) is instantiated in a unit of its own (rows_*.cu).
#pragma once

#include <cfloat>
#include <climits>

#include "select.cuh"

namespace spec {
namespace vocab {

constexpr float kLog2e = 1.4426950408889634f;

enum Verdict : uint32_t { kDone = 0, kWeighAll = 1, kMore = 2 };

// One row's request, after the checks.
struct Request {
    float T, p, low, u;  // low: the least logit that min-p keeps
    int k;               // 0: no limit
};

// The leader's part of a row whose kept tokens are among the n entries of its list, which holds the
// row's n largest logits: sorts them, cuts, draws.  W0, W1: bounds of the weight of all tokens that
// top-p is a share of, in units of 2^-U; 0: the list's own first k.  kWeighAll: the bounds leave the
// cut open; kMore: the cut lies past the list.
template <int EB>
__device__ Verdict draw_from_list(Row<EB> &r, const Scale &sc, const Request &q, int n, unsigned long long W0, unsigned long long W1,
                                  int32_t *token) {
    SelectShared *sh = r.sh;
    const int tid = r.tid, lane = r.lane, warp = r.warp;
    sort_list(sh->list, n, tid);
    int nk = q.k > 0 ? min(n, q.k) : n;
    auto value = [&](int i) { return key_value(~static_cast<uint32_t>(sh->list[i] >> 32)); };

    // running sums of the sorted weights, a run of entries per thread
    const int per = (nk + kThreads - 1) / kThreads;
    const int i0 = min(nk, tid * per), i1 = min(nk, i0 + per);
    unsigned long long mine = 0;
    for (int i = i0; i < i1; ++i) {
        mine += fixed_weight(value(i), sc, sh->pow2);
        sh->cum[i] = mine;
    }
    const unsigned long long incl = warp_scan(mine, lane);
    if (lane == 31) sh->red[warp] = incl;
    __syncthreads();
    unsigned long long before = incl - mine;
    for (int w = 0; w < warp; ++w) before += sh->red[w];
    for (int i = i0; i < i1; ++i) sh->cum[i] += before;
    __syncthreads();

    if (q.p < 1.f || q.low > -INFINITY) {
        const unsigned long long total = sh->cum[nk - 1];
        unsigned long long t0 = 0, t1 = 0;
        if (q.p < 1.f) {
            bool rest;
            t0 = scaled_floor(W0 ? W0 : total, q.p, &rest);
            t0 = max(t0 + (rest ? 1ull : 0ull), 1ull);
            t1 = scaled_floor(W1 ? W1 : total, q.p, &rest);
            t1 = max(t1 + (rest ? 1ull : 0ull), 1ull);
        }
        unsigned long long c = 0;  // entries below the two cuts of top-p, and entries that min-p keeps
        for (int i = i0; i < i1; ++i)
            c += static_cast<unsigned long long>(sh->cum[i] < t0) | static_cast<unsigned long long>(sh->cum[i] < t1) << 16 |
                 static_cast<unsigned long long>(value(i) >= q.low) << 32;
        c = block_sum(c, sh->red, lane, warp);
        if (q.p < 1.f) {
            const int a = static_cast<int>(c & 0xffff) + 1, b = static_cast<int>((c >> 16) & 0xffff) + 1;
            if (b > nk) return kMore;
            if (a != b) return kWeighAll;
            nk = a;
        }
        nk = min(nk, static_cast<int>(c >> 32));
    }
    const unsigned long long W = sh->cum[nk - 1];
    auto index = [&](int i) { return static_cast<uint32_t>(sh->list[i]); };
    if (nk == 1) {
        if (tid == 0) *token = static_cast<int32_t>(index(0));
        return kDone;
    }
    if (q.u == 0.f) {  // the first kept token, however small its weight (a double's least is 2^-1074)
        uint32_t x = kAll;
        for (int i = tid; i < nk; i += kThreads)
            if ((value(i) - sc.m) * sc.ch > -1074.f) x = min(x, index(i));
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
    const unsigned long long target = scaled_floor(W, q.u, &rest) + 1;
    auto weight = [&](int i) { return sh->cum[i] - (i ? sh->cum[i - 1] : 0ull); };
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
    sort_list(sh->list, nk, tid);
    const int pn = (nk + kThreads - 1) / kThreads;
    const int j0 = min(nk, tid * pn), j1 = min(nk, j0 + pn);
    unsigned long long s = 0;
    for (int j = j0; j < j1; ++j) s += weight(static_cast<int>(static_cast<uint32_t>(sh->list[j])));
    const unsigned long long upto = warp_scan(s, lane);
    if (lane == 31) sh->red[warp] = upto;
    __syncthreads();
    unsigned long long run = upto - s;
    for (int w = 0; w < warp; ++w) run += sh->red[w];
    for (int j = j0; j < j1; ++j) {
        const unsigned long long w = weight(static_cast<int>(static_cast<uint32_t>(sh->list[j])));
        if (run < target && run + w >= target) *token = static_cast<int32_t>(sh->list[j] >> 32);
        run += w;
    }
    return kDone;
}

// The long way: the kept tokens are cut out of the whole row, and the draw runs over it.
template <int EB>
__device__ void draw_from_row(const RowArgs &a, Row<EB> &r, const Scale &sc, const Request &q, int32_t *token) {
    const float2 *pow2 = r.sh->pow2;
    // the kept tokens: those of a key above ck, and those of key ck up to index ci
    uint32_t ck = Row<EB>::kLowest;
    int ci = INT_MAX;
    const uint32_t top = Row<EB>::key(sc.m);
    auto kept = [&](float l, int x) {
        const uint32_t y = Row<EB>::key(l);
        return y > ck || (y == ck && x <= ci);
    };
    auto weight = [&](float l, int x) { return kept(l, x) ? fixed_weight(l, sc, pow2) : 0ull; };
    auto total = [&]() {
        unsigned long long v = 0;
        r.each([&](float l, int x) { v += weight(l, x); });
        return r.sum(v);
    };
    if (q.k > 0) {
        uint32_t at;
        unsigned long long above;
        if (r.template reach<true>(ck, top, q.k, [&](float, int) { return 1ull; }, &at, &above)) {
            ci = r.tie_index(at, q.k - above, [](float, int) { return true; });
            ck = at;
        }
    }
    if (q.p < 1.f) {
        bool rest;
        unsigned long long target = scaled_floor(total(), q.p, &rest);
        target = max(target + (rest ? 1ull : 0ull), 1ull);
        uint32_t at;
        unsigned long long above;
        if (r.template reach<false>(ck, top, target, weight, &at, &above)) {
            const unsigned long long w = fixed_weight(Row<EB>::value(at), sc, pow2);
            const int old = ci;
            const bool same = at == ck;
            const int x = r.tie_index(at, (target - above + w - 1) / w, [&](float, int y) { return !same || y <= old; });
            ck = at;
            ci = x;
        }
    }
    if (q.low > -INFINITY) {
        uint32_t y = Row<EB>::key(q.low);
        if (EB == 2 && Row<EB>::value(y) < q.low) ++y;
        if (y > ck) ck = y, ci = INT_MAX;
    }
    if (q.u == 0.f) {  // the first kept token, however small its weight (a double's least is 2^-1074)
        auto any = [&](float l, int x) {
            return static_cast<unsigned long long>(kept(l, x) && (l - sc.m) * sc.ch > -1074.f);
        };
        r.locate(1ull, any, [&](int x) { *token = x; });
        return;
    }
    bool rest;
    const unsigned long long target = scaled_floor(total(), q.u, &rest) + 1;
    r.locate(target, weight, [&](int x) { *token = x; });
}

// Filtered sampling of row b.
template <int EB>
__device__ void sample_row(const RowArgs &a, Row<EB> &r, int b, uint4 *buf) {
    SelectShared *sh = r.sh;
    r.start_load(a, b, buf);
    Request q;
    q.u = a.u[b];
    q.T = a.temperature[b];
    q.k = a.top_k ? a.top_k[b] : 0;
    q.p = a.top_p ? a.top_p[b] : 1.f;
    q.low = -INFINITY;
    const float mp = a.min_p ? a.min_p[b] : 0.f;
    const bool greedy = q.T == 0.f;
    const bool bad = !(greedy || (q.T >= kMinTemperature && q.T <= kMaxTemperature)) ||
                     !(greedy || (q.p >= 0.f && q.p <= 1.f && mp >= 0.f && mp <= 1.f && q.u >= 0.f && q.u < 1.f));
    if (bad) {
        copies_wait<0>();
        cluster_wait();
        if (r.rank == 0 && r.tid == 0) {
            a.tokens[b] = -1;
            atomicOr(a.status, SPEC_DEV_BAD_PARAM);
        }
        return;
    }
    const bool one = greedy || q.k == 1;  // the argmax, whatever the other filters keep
    if (greedy) q.T = 1.f;
    if (q.k < 0 || q.k >= a.V) q.k = 0;
    const double c = 1.4426950408889634074 / static_cast<double>(q.T);
    Scale sc;
    sc.ch = static_cast<float>(c);
    sc.cl = static_cast<float>(c - static_cast<double>(sc.ch));
    sc.U = a.U;
    const double below = mp > 0.f && !one ? static_cast<double>(q.T) * log(static_cast<double>(mp)) : 0.0;
    sc.m = r.maximum(buf);
    if (!(fabsf(sc.m) < INFINITY)) {  // NaN, +inf, or nothing but -inf
        if (r.rank == 0 && r.tid == 0) {
            a.tokens[b] = -1;
            atomicOr(a.status, SPEC_DEV_NONFINITE);
        }
        return;
    }
    if (one) {  // the lowest index of the maximum: each warp's first, to the leader
        uint32_t x = kAll;
        if (r.own_max == sc.m) r.each([&](float l, int y) { if (l == sc.m) x = min(x, static_cast<uint32_t>(y)); });
        x = __reduce_min_sync(kAll, x);
        if (r.lane == 0) st_peer(peer(&sh->hits[0][r.rank * kWarps + r.warp], 0), x);
        cluster_sync();
        if (r.rank == 0 && r.warp == 0) {
            x = kAll;
            for (uint32_t i = r.lane; i < r.cs * kWarps; i += 32) x = min(x, sh->hits[0][i]);
            x = __reduce_min_sync(kAll, x);
            if (r.lane == 0) a.tokens[b] = static_cast<int32_t>(x);
        }
        return;
    }
    // w >= min_p as a bound on the logit: only the least logit at or above the bound matters
    if (mp > 0.f) q.low = __double2float_ru(static_cast<double>(sc.m) + below);

    // The list holds the logits from `low` on; all: that is every token.
    const bool share = q.p < 1.f && q.k == 0;  // top-p is a share of the whole row
    const int attempts = share && a.V > kMaxList ? 2 : 1;
    float low[2] = {-FLT_MAX, -FLT_MAX};
    bool all[2] = {true, true};
    if (a.V > kMaxList) {
        if (q.k > kMaxGoal || (q.k == 0 && !share && !(mp > 0.f))) {
            draw_from_row(a, r, sc, q, a.tokens + b);
            return;
        }
        if (q.k > 0 || share) {  // fewer groups than asked for: few tokens that are not masked
            all[0] = !r.threshold(sc.m, q.k > 0 ? q.k : kFirstGoal, &low[0]);
            if (share && !all[0]) all[1] = !r.threshold(sc.m, kMaxGoal, &low[1]);
        } else {
            low[0] = q.low;
            all[0] = false;
        }
    }
    const bool sums = share && !all[0];
    if (sums) r.exp_sum(sc.m, sc.ch);
    for (int attempt = 0; attempt < attempts; ++attempt) {
        r.collect(low[attempt], attempt);
        cluster_sync();
        const uint32_t n = r.collected(attempt);
        if (sums && attempt == 0) {
            const unsigned long long W = r.exp_total() << (sc.U - 40);
            sh->W[0] = W - (W >> 16);
            sh->W[1] = W + (W >> 16);
        }
        if (n > kMaxList) break;
        if (!share || all[attempt]) {
            if (r.rank == 0) draw_from_list(r, sc, q, n, 0ull, 0ull, a.tokens + b);
            return;
        }
        __syncthreads();
        uint32_t v = kDone;
        for (int exact = 0; exact < 2; ++exact) {
            if (r.rank == 0) {
                v = draw_from_list(r, sc, q, n, sh->W[0], sh->W[1], a.tokens + b);
                if (r.tid < static_cast<int>(r.cs)) st_peer(peer(&sh->verdict, r.tid), v);
            }
            cluster_sync();
            v = sh->verdict;
            if (v != kWeighAll) break;
            unsigned long long w = 0;
            r.each([&](float l, int) { w += fixed_weight(l, sc, sh->pow2); });
            w = r.sum(w);
            sh->W[0] = sh->W[1] = w;
            __syncthreads();
        }
        if (v == kDone) return;
    }
    draw_from_row(a, r, sc, q, a.tokens + b);
}

// The K largest logits of row b.
template <int EB>
__device__ void top_row(const RowArgs &a, Row<EB> &r, int b, uint4 *buf) {
    SelectShared *sh = r.sh;
    r.start_load(a, b, buf);
    const float m = r.maximum(buf);
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
    if (a.lse && !empty) r.exp_sum(m, kLog2e / a.temp);
    float low = -FLT_MAX;
    if (!empty && a.V > kMaxList && !r.threshold(m, a.K, &low)) low = -FLT_MAX;  // few tokens that are not masked
    bool shorter = !empty;
    if (shorter) r.collect(low, 0);
    cluster_sync();
    if (a.lse) {
        const float S = empty ? 0.f : static_cast<float>(r.exp_total()) * 0x1p-40f;
        if (r.rank == 0 && r.tid == 0) a.lse[b] = empty ? -INFINITY : m / a.temp + logf(S);
    }
    int n = 0;
    if (shorter) {
        const uint32_t c = r.collected(0);
        shorter = c <= kMaxList;
        n = static_cast<int>(c);
    }
    if (!shorter && !empty) {
        uint32_t ck = Row<EB>::kLowest;
        int ci = INT_MAX;
        uint32_t at;
        unsigned long long above;
        if (r.template reach<true>(ck, Row<EB>::key(m), a.K, [](float, int) { return 1ull; }, &at, &above)) {
            ci = r.tie_index(at, a.K - above, [](float, int) { return true; });
            ck = at;
        }
        const uint32_t n_at = peer(&sh->list_n[1], 0), list_at = peer(sh->list, 0);
        r.each([&](float l, int x) {
            const uint32_t y = Row<EB>::key(l);
            if (y > ck || (y == ck && x <= ci)) {
                const uint32_t i = atom_add_peer(n_at, 1);
                if (i < kMaxList) st_peer(list_at + i * 8, static_cast<unsigned long long>(~order_key(l)) << 32 | static_cast<uint32_t>(x));
            }
        });
        cluster_sync();
        n = static_cast<int>(sh->list_n[1]);
    }
    if (r.rank != 0) return;
    sort_list(sh->list, n, r.tid);
    for (int i = r.tid; i < a.K; i += kThreads) {
        const unsigned long long e = i < n ? sh->list[i] : 0ull;
        a.values[out + i] = i < n ? key_value(~static_cast<uint32_t>(e >> 32)) : -INFINITY;
        a.ids[out + i] = i < n ? static_cast<int32_t>(static_cast<uint32_t>(e)) : -1;
    }
}

template <int EB, int OP>
__global__ void __launch_bounds__(kThreads) row_kernel(const RowArgs a) {
    extern __shared__ uint4 dyn[];
    SelectShared *sh = reinterpret_cast<SelectShared *>(dyn);
    uint4 *buf = dyn + sizeof(SelectShared) / 16;
    Row<EB> r = row_setup<EB>(a, sh);
    cluster_arrive();  // the first peer access waits for it
    const int b = blockIdx.x / a.cluster;
    if (OP == kSampleRows)
        sample_row<EB>(a, r, b, buf);
    else
        top_row<EB>(a, r, b, buf);
}

// CTAs per row and vectors per CTA.
inline spec_status row_split(RowArgs *a, int EB, size_t fixed, size_t max_dyn) {
    const long long vecs = (static_cast<long long>(a->V) * EB + 14) / 16 + 1;  // at the worst alignment
    int cs = 1;
    while (cs < kMaxCluster && (vecs + cs - 1) / cs * 16 > 40 * 1024) cs *= 2;
    while (cs < kMaxCluster && static_cast<long long>(a->B) * cs < 152 && vecs / cs > kThreads) cs *= 2;
    a->cluster = cs;
    a->part = static_cast<int>((vecs + cs - 1) / cs);
    if (fixed + static_cast<size_t>(a->part) * 16 > max_dyn)
        return fail(SPEC_ERR_UNSUPPORTED, "V = %d: a row does not fit the shared memory of %d SMs", a->V, cs);
    return SPEC_OK;
}

template <int EB, int OP>
spec_status launch_rows(const RowArgs &a0, cudaStream_t stream) {
    static_assert(sizeof(SelectShared) % 16 == 0, "the row follows in 16-byte vectors");
    RowArgs a = a0;
    DeviceInfo di;
    int dev = 0;
    spec_status st = device_info(&di, &dev);
    if (st != SPEC_OK) return st;
    auto kernel = row_kernel<EB, OP>;
    st = allow_max_dyn_smem(dev, reinterpret_cast<const void *>(kernel), &di);
    if (st != SPEC_OK) return st;
    st = row_split(&a, EB, sizeof(SelectShared), di.max_dyn);
    if (st != SPEC_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(SelectShared) + static_cast<size_t>(a.part) * 16;
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
        return fail(SPEC_ERR_CUDA, "row kernel launch (B=%d, cluster=%d, smem=%zu): %s", a.B, a.cluster, (size_t)cfg.dynamicSmemBytes,
                    cudaGetErrorString(e));
    return SPEC_OK;
}

}  // namespace vocab
}  // namespace spec
