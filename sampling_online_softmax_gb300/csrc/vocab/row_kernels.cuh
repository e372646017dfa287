// row_kernels.cuh -- the kernels on rows of logits and their launcher; each
// (element size, operation) is instantiated in a unit of its own (rows_*.cu).
#pragma once

#include "select.cuh"

namespace spec {
namespace vocab {

constexpr float kLog2e = 1.4426950408889634f;

// Filtered sampling of row b.
template <int EB>
__device__ void sample_row(const RowArgs &a, Row<EB> &r, int b, uint4 *buf) {
    const float u = a.u ? a.u[b] : 0.f;
    float T = a.temperature[b];
    int k = a.top_k ? a.top_k[b] : 0;
    float p = a.top_p ? a.top_p[b] : 1.f;
    float mp = a.min_p ? a.min_p[b] : 0.f;
    const bool greedy = T == 0.f;
    const bool bad = !(greedy || (T >= kMinTemperature && T <= kMaxTemperature)) || !(p >= 0.f && p <= 1.f) ||
                     !(mp >= 0.f && mp <= 1.f) || !(greedy || (u >= 0.f && u < 1.f));
    if (bad) {
        cluster_wait();
        if (r.rank == 0 && r.tid == 0) {
            a.tokens[b] = -1;
            atomicOr(a.status, SPEC_DEV_BAD_PARAM);
        }
        return;
    }
    if (greedy) T = 1.f, k = 1, p = 1.f, mp = 0.f;
    r.load(a, b, buf);
    cluster_wait();
    Scale sc;
    sc.m = r.maximum();
    if (!(fabsf(sc.m) < INFINITY)) {  // NaN, +inf, or nothing but -inf
        if (r.rank == 0 && r.tid == 0) {
            a.tokens[b] = -1;
            atomicOr(a.status, SPEC_DEV_NONFINITE);
        }
        return;
    }
    const double c = 1.4426950408889634074 / static_cast<double>(T);
    sc.ch = static_cast<float>(c);
    sc.cl = static_cast<float>(c - static_cast<double>(sc.ch));
    sc.U = a.U;
    const float2 *pow2 = r.sh->pow2;

    // the kept tokens: those of a key above ck, and those of key ck up to index ci
    uint32_t ck = Row<EB>::kLowest;
    int ci = INT_MAX;
    const uint32_t top = Row<EB>::key(sc.m);
    auto kept = [&](float l, int x) {
        const uint32_t q = Row<EB>::key(l);
        return q > ck || (q == ck && x <= ci);
    };
    auto weight = [&](float l, int x) { return kept(l, x) ? fixed_weight(l, sc, pow2) : 0ull; };
    auto total = [&]() {
        unsigned long long v = 0;
        r.each([&](float l, int x) { v += weight(l, x); });
        return r.sum(v);
    };
    if (k > 0 && k < a.V) {
        uint32_t at;
        unsigned long long above;
        if (r.template reach<true>(ck, top, k, [&](float, int) { return 1ull; }, &at, &above)) {
            ci = r.tie_index(at, k - above, [](float, int) { return true; });
            ck = at;
        }
    }
    if (p < 1.f) {
        bool rest;
        unsigned long long target = scaled_floor(total(), p, &rest);
        target = max(target + (rest ? 1ull : 0ull), 1ull);
        uint32_t at;
        unsigned long long above;
        if (r.template reach<false>(ck, top, target, weight, &at, &above)) {
            const unsigned long long w = fixed_weight(Row<EB>::value(at), sc, pow2);
            const int old = ci;
            const bool same = at == ck;
            const int x = r.tie_index(at, (target - above + w - 1) / w, [&](float, int x) { return !same || x <= old; });
            ck = at;
            ci = x;
        }
    }
    if (mp > 0.f) {
        // w >= min_p as a bound on the logit; only the smallest logit at or above the bound matters
        const float low = __double2float_ru(static_cast<double>(sc.m) + static_cast<double>(T) * log(static_cast<double>(mp)));
        uint32_t q = Row<EB>::key(low);
        if (EB == 2 && Row<EB>::value(q) < low) ++q;
        if (q > ck) ck = q, ci = INT_MAX;
    }
    if (u == 0.f || greedy) {  // the first kept token, however small its weight (a double's least is 2^-1074)
        auto any = [&](float l, int x) {
            return static_cast<unsigned long long>(kept(l, x) && (l - sc.m) * sc.ch > -1074.f);
        };
        r.locate(1ull, any, [&](int x) { a.tokens[b] = x; });
        return;
    }
    const unsigned long long W = total();
    bool rest;
    const unsigned long long target = scaled_floor(W, u, &rest) + 1;
    r.locate(target, weight, [&](int x) { a.tokens[b] = x; });
}

// The K largest logits of row b.
template <int EB>
__device__ void top_row(const RowArgs &a, Row<EB> &r, int b, uint4 *buf) {
    SelectShared *sh = r.sh;
    r.load(a, b, buf);
    cluster_wait();
    const float m = r.maximum();
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
        float s = 0.f;
        if (!empty) {
            const float c = kLog2e / a.temp;
            r.each([&](float l, int) { s += exp2f((l - m) * c); });
        }
        const unsigned long long S = r.sum(__float2ull_rn(s * 0x1p40f));
        if (r.rank == 0 && r.tid == 0) a.lse[b] = empty ? -INFINITY : m / a.temp + logf(static_cast<float>(S) * 0x1p-40f);
    }
    uint32_t ck = Row<EB>::kLowest;
    int ci = INT_MAX;
    if (!empty && a.K < a.V) {
        uint32_t at;
        unsigned long long above;
        if (r.template reach<true>(ck, Row<EB>::key(m), a.K, [](float, int) { return 1ull; }, &at, &above)) {
            ci = r.tie_index(at, a.K - above, [](float, int) { return true; });
            ck = at;
        }
    }
    const uint32_t n_at = peer(&sh->list_n, 0), list_at = peer(sh->list, 0);
    r.each([&](float l, int x) {
        const uint32_t q = Row<EB>::key(l);
        if (q > ck || (q == ck && x <= ci)) {
            const uint32_t i = atom_add_peer(n_at, 1);
            if (i < kMaxList) st_peer(list_at + i * 8, static_cast<unsigned long long>(~order_key(l)) << 32 | static_cast<uint32_t>(x));
        }
    });
    cluster_sync();
    if (r.rank != 0) return;
    const int n = min(static_cast<int>(sh->list_n), a.K);
    int size = 1;
    while (size < n) size <<= 1;
    for (int i = n + r.tid; i < size; i += kThreads) sh->list[i] = ~0ull;
    sort_list(sh->list, size, r.tid);
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
    while (cs < kMaxCluster && (vecs + cs - 1) / cs * 16 > 72 * 1024) cs *= 2;
    while (cs < kMaxCluster && static_cast<long long>(a->B) * cs < 152 && vecs / cs > 512) cs *= 2;
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
