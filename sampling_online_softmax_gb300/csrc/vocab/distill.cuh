// distill.cuh -- distillation from a teacher's largest logits: the loss of each
// row and its gradient.
//
//   q = softmax(s / T),  p_k = exp(t_k / T - lse)  (or the softmax of the K entries),  P = sum_k p_k
//   loss = w sum_k p_k (log p_k - log q_{id_k}),   d loss / d s_v = (w / T) (P q_v - sum_{k: id_k = v} p_k)
//
// HBM bounds all three forms.  Loss and gradient in one call read each logit once:
// a cluster keeps the row in its CTAs' shared memory between the exp-sum and the
// gradient.  A CTA writes its share of P q_v densely and then, after a block
// barrier, the columns of its own teacher entries over it; an entry's column
// is written by one thread (the first slot that names it), which adds the slots
// that name it too in their order, so the gradient does not depend on timing.
#pragma once

#include <algorithm>

#include "distill.h"
#include "part.cuh"

namespace spec {
namespace vocab {

constexpr int kDWarps = kDThreads / 32;
constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr float kLog2ef = 1.4426950408889634f;

// SLOTS teacher entries per thread: 1 where K <= kDThreads, else 4.
template <int SLOTS>
struct alignas(16) DistillShared {
    int32_t id[SLOTS * kDThreads];  // teacher entries in this CTA's part (-1: none, elsewhere, or out of range)
    float p[SLOTS * kDThreads];
    float red[5][kDWarps];
    float4 slot[kMaxCluster];       // of each CTA: its maximum, exp-sum, sum of p (log p - (s - m) / T), sum of p
    int twice;                      // some column is named by two entries
};

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAllLanes, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAllLanes, v, o));
    return v;
}

// Beyond it a maximum's product with c is taken for overflowing, and (l - m) c is computed as that.
constexpr float kHuge = 1e38f;

template <int EB, int SLOTS>
struct Distill {
    using P = Part<EB>;
    static constexpr int kPer = P::kPer;
    const DistillArgs &a;
    DistillShared<SLOTS> *sh;
    P part;
    int b, tid, lane, warp;
    float c, invT;    // log2(e) / T, 1 / T
    float sum_p;      // P; NaN where the teacher holds NaN or infinity
    int32_t id[SLOTS];
    float t[SLOTS];   // the teacher's logits, then log p

    __device__ __forceinline__ Distill(const DistillArgs &a_, DistillShared<SLOTS> *s, int row, uint32_t rank) : a(a_), sh(s) {
        b = row;
        tid = threadIdx.x;
        lane = tid & 31;
        warp = tid >> 5;
        c = kLog2ef / a.T;
        invT = 1.f / a.T;
        part.place(a.student, a.student_end, a.V, b, rank, a.part);
    }
    template <class F>
    __device__ __forceinline__ float block(float v, float none, int which, F join) {
        if (lane == 0) sh->red[which][warp] = v;
        __syncthreads();
        v = none;
#pragma unroll
        for (int i = 0; i < kDWarps; ++i) v = join(v, sh->red[which][i]);
        return v;
    }
    __device__ __forceinline__ float block_add(float v, int which) {
        return block(warp_add(v), 0.f, which, [](float x, float y) { return x + y; });
    }
    __device__ __forceinline__ float block_max(float v, int which) {
        return block(warp_max(v), -INFINITY, which, [](float x, float y) { return fmaxf(x, y); });
    }

    // The teacher's entries, on their way while the copies of the logits are issued.
    __device__ __forceinline__ void ask_teacher() {
        const size_t at = static_cast<size_t>(b) * a.K;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const int k = tid + j * kDThreads;
            id[j] = -1;
            t[j] = -INFINITY;
            if (k < a.K) {
                id[j] = __ldg(a.ids + at + k);
                t[j] = __ldg(a.top + at + k);
            }
        }
    }
    // Every CTA of a row weighs all K entries (P has to be the same everywhere) and keeps those in its
    // part, marked in a bitmap, one bit a logit; sh->twice: a column was marked before.  `bits` has been
    // cleared, a block barrier ago.
    __device__ __forceinline__ void teacher(uint32_t *bits) {
        float top = -INFINITY;
        bool wrong = false, off = false;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            if (id[j] >= a.V || id[j] < -1) off = true, id[j] = -1;
            if (id[j] < 0) t[j] = -INFINITY;
            if (!(t[j] < INFINITY)) wrong = true;
            top = fmaxf(top, t[j]);
        }
        float norm;  // log p = (t - top) / T - norm
        if (a.lse) {
            top = 0.f;
            norm = __ldg(a.lse + b);
            if (!(fabsf(norm) < INFINITY)) wrong = true;
        } else {
            top = block_max(top, 0);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
                if (t[j] > -INFINITY) s += expf((t[j] - top) * invT);
            s = block_add(s, 1);
            norm = s > 0.f ? logf(s) : 0.f;
        }
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const bool any = t[j] > -INFINITY;
            t[j] = any ? (t[j] - top) * invT - norm : 0.f;
            const float p = any ? expf(t[j]) : 0.f;
            sum += p;
            const int k = tid + j * kDThreads;
            const int o = id[j] >= 0 ? part.offset(id[j]) : -1;
            if (o < 0 || o >= part.n * kPer) id[j] = -1;
            sh->id[k] = id[j];
            sh->p[k] = p;
            if (bits && id[j] >= 0 && (atomicOr(&bits[o >> 5], 1u << (o & 31)) >> (o & 31) & 1u)) sh->twice = 1;
        }
        if (off) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
        sum_p = block_add(wrong ? NAN : sum, 2);
    }
    __device__ __forceinline__ void clear(uint32_t *bits) {
        for (int i = tid; i < (part.n * kPer + 31) / 32; i += kDThreads) bits[i] = 0;
        if (tid == 0) sh->twice = 0;
    }

    __device__ __forceinline__ void store(int i, const float (&v)[kPer], bool same) const {
        unsigned char *d = a.grad + (part.at(i) - a.student);
        if (same && !part.edge(i)) {
            uint4 o;
            if (EB == 4) {
                o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            } else {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[q]) : "f"(v[(2 * q + 1) % kPer]), "f"(v[(2 * q) % kPer]));
                o = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4 *>(d) = o;
        } else {
            store_each(i, v);
        }
    }
    __device__ __forceinline__ void store_each(int i, const float (&v)[kPer]) const {
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const int x = part.index(i, q);
            if (x >= 0 && x < a.V) store_one(x, v[q]);
        }
    }
    __device__ __forceinline__ void store_one(int x, float v) const {
        const size_t e = static_cast<size_t>(b) * a.V + x;
        if (EB == 4)
            reinterpret_cast<float *>(a.grad)[e] = v;
        else
            reinterpret_cast<__nv_bfloat16 *>(a.grad)[e] = __float2bfloat16_rn(v);
    }
    // The two tensors' vectors lie alike, so a vector of logits gives a vector of gradients.
    __device__ __forceinline__ bool alike() const {
        return ((reinterpret_cast<uintptr_t>(a.grad) ^ reinterpret_cast<uintptr_t>(a.student)) & 15) == 0;
    }
    __device__ __forceinline__ void fill(float v) const {
        float g[kPer];
#pragma unroll
        for (int q = 0; q < kPer; ++q) g[q] = v;
        const bool same = alike();
        for (int i = tid; i < part.n; i += kDThreads) store(i, g, same);
    }
    // (w / T) P q_v for every column of the part (logits from `get`), then the teacher's columns.
    // g: w / T; m, S: the row's maximum and exp-sum.
    template <class G, class L>
    __device__ __forceinline__ void gradient(float g, float m, float S, G get, L logit_at) {
        // exponents as l c - q, q the rounded m c, whose rounding goes into the factor
        const float q = m * c, A = g * sum_p / S;
        const bool plain = fabsf(q) < kHuge;
        const float A_ = plain ? A * (1.f - 0.6931471805599453f * fmaf(-m, c, q)) : A;
        const bool same = alike();
        float own[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) own[j] = id[j] >= 0 ? logit_at(id[j]) : 0.f;  // before anything is written: grad may be student
        __syncthreads();
        const bool twice = sh->twice != 0;
        const unsigned long long A2 = pair(A_, A_), c2 = pair(c, c), q2 = pair(-q, -q);
#pragma unroll 4
        for (int i = tid; i < part.n; i += kDThreads) {
            float l[kPer];
            P::unpack(get(i), l);
#pragma unroll
            for (int e = 0; e < kPer; e += 2) {
                float x, y;
                const unsigned long long two = pair(l[e], l[e + 1]);
                split(plain ? fma2(two, c2, q2) : mul2(add2(two, pair(-m, -m)), c2), x, y);
                split(mul2(pair(ptx::ex2(x), ptx::ex2(y)), A2), l[e], l[e + 1]);
            }
            store(i, l, same);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const int x = id[j];
            if (x < 0) continue;
            const int k = tid + j * kDThreads;
            float p = sh->p[k];
            if (twice) {
                bool lower = false;
                for (int o = 0; o < a.K; ++o) {
                    if (o == k || sh->id[o] != x) continue;
                    if (o < k) lower = true;
                    p += sh->p[o];
                }
                if (lower) continue;
            }
            store_one(x, A * ptx::ex2((own[j] - m) * c) - g * p);
        }
    }
};

// A thread's running maximum m and sum of 2^((l - m) c): as 2^(l c - q), q the rounded m c, one fused
// operation a pair; at the end the rounding of q goes into the sum.
template <int EB>
struct Running {
    using P = Part<EB>;
    float m = -INFINITY, q = -INFINITY;
    unsigned long long s = 0;  // a pair

    template <int N>
    __device__ __forceinline__ void add(const uint4 (&v)[N], float c) {
        float top = P::vector_max(v[0]);  // NaN if there is one
#pragma unroll
        for (int j = 1; j < N; ++j) top = max_nan(top, P::vector_max(v[j]));
        if (!(top <= m) && m == m) {      // (a NaN stays)
            const float to = top * c;
            const float f = m > -INFINITY ? ptx::ex2(fabsf(to) < kHuge ? q - to : (m - top) * c) : 0.f;
            s = mul2(s, pair(f, f));
            m = top;
            q = to;
        }
        if (m == -INFINITY) return;  // masked so far
        const bool plain = fabsf(q) < kHuge;
        const unsigned long long c2 = pair(c, c), q2 = pair(-q, -q);
        unsigned long long sum = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float l[P::kPer];
            P::unpack(v[j], l);
            unsigned long long e[P::kPer / 2];
#pragma unroll
            for (int i = 0; i < P::kPer / 2; ++i) {
                float x, y;
                const unsigned long long two = pair(l[2 * i], l[2 * i + 1]);
                split(plain ? fma2(two, c2, q2) : mul2(add2(two, pair(-m, -m)), c2), x, y);
                e[i] = pair(ptx::ex2(x), ptx::ex2(y));
            }
#pragma unroll
            for (int h = P::kPer / 4; h; h >>= 1)
#pragma unroll
                for (int i = 0; i < h; ++i) e[i] = add2(e[i], e[i + h]);
            sum = j ? add2(sum, e[0]) : e[0];
        }
        s = add2(s, sum);
    }
    __device__ __forceinline__ float sum(float c) const {
        float x, y;
        split(s, x, y);
        return (x + y) * (fabsf(q) < kHuge ? 1.f + 0.6931471805599453f * fmaf(-m, c, q) : 1.f);
    }
};

// Loss and row statistics, and with GRAD the gradient: a cluster per row.
template <int EB, int SLOTS, bool GRAD>
__global__ void __launch_bounds__(kDThreads, 4) distill_kernel(const DistillArgs a) {
    extern __shared__ uint4 dyn[];
    DistillShared<SLOTS> *sh = reinterpret_cast<DistillShared<SLOTS> *>(dyn);
    uint4 *buf = dyn + sizeof(DistillShared<SLOTS>) / 16;
    uint32_t *bits = GRAD ? reinterpret_cast<uint32_t *>(buf + a.part) : nullptr;
    const uint32_t rank = cluster_rank();
    const int b = blockIdx.x / a.cluster;
    Distill<EB, SLOTS> d(a, sh, b, rank);
    const int tid = d.tid;
    const float w = a.weight ? __ldg(a.weight + b) : 1.f;
    if (w == 0.f) {  // an ignored row: its logits are not read
        if (GRAD) d.fill(0.f);
        if (rank == 0 && tid == 0) {
            a.loss[b] = 0.f;
            a.stats[2 * static_cast<size_t>(b)] = 0.f;
            a.stats[2 * static_cast<size_t>(b) + 1] = 0.f;
        }
        return;
    }
    cluster_arrive();
    d.ask_teacher();
    const int n = d.part.n;
    if (GRAD) {
        d.part.copy_all(buf, tid, kDThreads);
        copies_commit();
        d.clear(bits);
        __syncthreads();
    }
    d.teacher(bits);
    Running<EB> r;
    if (GRAD) {
        copies_wait<0>();
        d.part.mend_all(buf, tid, kDThreads);
        int i = tid;
        for (; i + kDThreads < n; i += 2 * kDThreads) {
            const uint4 v[2] = {buf[i], buf[i + kDThreads]};
            r.add(v, d.c);
        }
        if (i < n) {
            const uint4 v[1] = {buf[i]};
            r.add(v, d.c);
        }
    } else {
        int i = tid;
        for (; i + 3 * kDThreads < n; i += 4 * kDThreads) {
            uint4 v[4];
            if (i > 0 && i + 3 * kDThreads < n - 1) {
                const uint4 *src = reinterpret_cast<const uint4 *>(d.part.at(i));
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = __ldg(src + j * kDThreads);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = d.part.fetch(i + j * kDThreads);
            }
            r.add(v, d.c);
        }
        for (; i < n; i += kDThreads) {
            const uint4 v[1] = {d.part.fetch(i)};
            r.add(v, d.c);
        }
    }
    // the block's, then the cluster's.  NaN passes through the sums.
    const float bm = d.block_max(r.m, 3);
    float s = r.m == -INFINITY ? 0.f : r.sum(d.c) * ptx::ex2((r.m - bm) * d.c);
    // (after that barrier the part is in shared memory for every thread)
    auto logit_at = [&](int x) {
        return GRAD ? Part<EB>::logit(buf, d.part.offset(x)) : Part<EB>::logit(a.student + (static_cast<size_t>(b) * a.V + x) * EB, 0);
    };
    float dot = 0.f, ps = 0.f;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        const float p = d.id[j] >= 0 ? sh->p[tid + j * kDThreads] : 0.f;
        if (p == 0.f) continue;
        const float l = logit_at(d.id[j]);
        dot += p * (d.t[j] - (l == -INFINITY ? l : (l - bm) * d.invT));  // a masked token the teacher wants: +inf
        ps += p;
    }
    s = warp_add(s);
    dot = warp_add(dot);
    ps = warp_add(ps);
    if (d.lane == 0) {
        sh->red[0][d.warp] = s;
        sh->red[1][d.warp] = dot;
        sh->red[4][d.warp] = ps;
    }
    __syncthreads();
    s = dot = ps = 0.f;
#pragma unroll
    for (int i = 0; i < kDWarps; ++i) {
        s += sh->red[0][i];
        dot += sh->red[1][i];
        ps += sh->red[4][i];
    }
    cluster_wait();
    if (tid < a.cluster) st_peer(peer(&sh->slot[rank], tid), make_float4(bm, s, dot, ps));
    cluster_sync();
    float m = -INFINITY;
    for (int i = 0; i < a.cluster; ++i) m = fmaxf(m, sh->slot[i].x);
    s = 0.f;
    dot = 0.f;
    for (int i = 0; i < a.cluster; ++i) {
        const float4 v = sh->slot[i];
        s += v.x == -INFINITY ? v.y : v.y * ptx::ex2((v.x - m) * d.c);  // a part of masked logits has sum 0 (or NaN)
        if (v.w != 0.f) dot += v.z + v.w * ((m - v.x) * d.invT);
    }
    const bool bad = !(d.sum_p == d.sum_p) || !(m < INFINITY && s > 0.f && s < INFINITY);  // NaN, +inf, or nothing but -inf
    if (rank == 0 && tid == 0) {
        a.loss[b] = bad ? NAN : d.sum_p > 0.f ? w * (dot + d.sum_p * logf(s)) : 0.f;
        a.stats[2 * static_cast<size_t>(b)] = bad ? NAN : m;
        a.stats[2 * static_cast<size_t>(b) + 1] = bad ? NAN : s;
        if (bad) atomicOr(a.status, SPEC_DEV_NONFINITE);
    }
    if (!GRAD) return;
    if (bad)
        d.fill(NAN);
    else
        d.gradient(w * d.invT, m, s, [&](int i) { return buf[i]; }, logit_at);
}

// The gradient alone, from the logits and a forward call's statistics: a CTA per part of a row.
template <int EB, int SLOTS>
__global__ void __launch_bounds__(kDThreads, 4) distill_backward_kernel(const DistillArgs a) {
    extern __shared__ uint4 dyn[];
    DistillShared<SLOTS> *sh = reinterpret_cast<DistillShared<SLOTS> *>(dyn);
    uint32_t *bits = reinterpret_cast<uint32_t *>(dyn + sizeof(DistillShared<SLOTS>) / 16);
    const int b = blockIdx.x / a.cluster;
    Distill<EB, SLOTS> d(a, sh, b, blockIdx.x % a.cluster);
    const float up = (a.weight ? __ldg(a.weight + b) : 1.f) * __ldg(a.grad_loss + b);
    if (up == 0.f) {
        d.fill(0.f);
        return;
    }
    d.ask_teacher();
    const float2 ms = __ldg(reinterpret_cast<const float2 *>(a.stats) + b);
    d.clear(bits);
    __syncthreads();
    d.teacher(bits);
    if (!(d.sum_p == d.sum_p) || !(fabsf(ms.x) < INFINITY && ms.y > 0.f && ms.y < INFINITY)) {
        if (d.tid == 0) atomicOr(a.status, SPEC_DEV_NONFINITE);
        d.fill(NAN);
        return;
    }
    d.gradient(up * d.invT, ms.x, ms.y, [&](int i) { return d.part.fetch(i); },
               [&](int x) { return Part<EB>::logit(a.student + (static_cast<size_t>(b) * a.V + x) * EB, 0); });
}

template <class Kernel>
spec_status go(Kernel kernel, DistillArgs a, int eb, int slots, int form, cudaStream_t stream) {
    DeviceInfo di;
    int dev = 0;
    spec_status st = device_info(&di, &dev);
    if (st != SPEC_OK) return st;
    st = allow_max_dyn_smem(dev, reinterpret_cast<const void *>(kernel), &di);
    if (st != SPEC_OK) return st;
    const long long vecs = (static_cast<long long>(a.V) * eb + 14) / 16 + 1;  // at the worst alignment
    const long long most = (form == kLossGrad ? kPartBytes : 48 * 1024);
    const long long limit = form == kBackward ? 1 << 20 : kMaxCluster;
    long long cs = std::min(limit, (vecs * 16 + most - 1) / most);
    while (2 * cs <= kMaxCluster && a.N * cs < 2 * di.sms && vecs / cs > 2 * kDThreads) cs *= 2;
    a.cluster = static_cast<int>(cs);
    a.part = static_cast<int>((vecs + cs - 1) / cs);
    const size_t fixed = slots == 1 ? sizeof(DistillShared<1>) : sizeof(DistillShared<4>);
    const size_t row = form == kLossGrad ? static_cast<size_t>(a.part) * 16 : 0;
    const size_t bits = form == kLoss ? 0 : (static_cast<size_t>(a.part) * (16 / eb) + 31) / 32 * 4;
    const size_t smem = fixed + row + bits;
    if (smem > di.max_dyn) return fail(SPEC_ERR_UNSUPPORTED, "V = %d: a row does not fit the shared memory of %lld SMs", a.V, cs);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N * cs));
    cfg.blockDim = dim3(kDThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = form == kBackward ? 0 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(SPEC_ERR_CUDA, "distillation launch (N=%d, cluster=%lld, smem=%zu): %s", a.N, cs, smem, cudaGetErrorString(e));
    return SPEC_OK;
}

template <int EB>
spec_status launch_distill(const DistillArgs &a, int form, cudaStream_t stream) {
    if (a.K <= kDThreads) {
        if (form == kLoss) return go(distill_kernel<EB, 1, false>, a, EB, 1, form, stream);
        if (form == kLossGrad) return go(distill_kernel<EB, 1, true>, a, EB, 1, form, stream);
        return go(distill_backward_kernel<EB, 1>, a, EB, 1, form, stream);
    }
    if (form == kLoss) return go(distill_kernel<EB, 4, false>, a, EB, 4, form, stream);
    if (form == kLossGrad) return go(distill_kernel<EB, 4, true>, a, EB, 4, form, stream);
    return go(distill_backward_kernel<EB, 4>, a, EB, 4, form, stream);
}

}  // namespace vocab
}  // namespace spec
