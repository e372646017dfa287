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

#include "../ptx.cuh"
#include "distill.h"
#include "part.cuh"

namespace spec {
namespace vocab {

constexpr int kDWarps = kDThreads / 32;
constexpr int kSlots = SPEC_MAX_TOP / kDThreads;  // teacher entries per thread
constexpr uint32_t kAllLanes = 0xffffffffu;
constexpr float kLog2ef = 1.4426950408889634f;

struct alignas(16) DistillShared {
    int32_t id[SPEC_MAX_TOP];   // teacher entries in this CTA's part (-1: none, elsewhere, or out of range)
    float p[SPEC_MAX_TOP];
    float red[4][kDWarps];
    float4 slot[kMaxCluster];   // of each CTA: its maximum, exp-sum, sum of p (log p - (s - m) / T), sum of p
    int twice;                  // some column is named by two entries
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

template <int EB>
struct Distill {
    using P = Part<EB>;
    static constexpr int kPer = P::kPer;
    const DistillArgs &a;
    DistillShared *sh;
    P part;
    int b, tid, lane, warp;
    float c;          // log2(e) / T
    float sum_p;      // P
    bool bad;         // a teacher entry that is NaN or +inf

    __device__ __forceinline__ Distill(const DistillArgs &a_, DistillShared *s, int row, uint32_t rank) : a(a_), sh(s) {
        b = row;
        tid = threadIdx.x;
        lane = tid & 31;
        warp = tid >> 5;
        c = kLog2ef / a.T;
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

    // The teacher: every CTA of a row weighs all K entries (P has to be the same everywhere) and
    // keeps those in its part.  logp[j] is slot tid + j * kDThreads's log p.
    __device__ void teacher(float (&logp)[kSlots]) {
        const size_t at = static_cast<size_t>(b) * a.K;
        int32_t id[kSlots];
        float t[kSlots];
        float top = -INFINITY;
        bool wrong = false, off = false;
        const float invT = 1.f / a.T;
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int k = tid + j * kDThreads;
            id[j] = -1;
            t[j] = -INFINITY;
            if (k < a.K) {
                id[j] = a.ids[at + k];
                if (id[j] >= a.V || id[j] < -1) off = true, id[j] = -1;
                if (id[j] >= 0) {
                    t[j] = a.top[at + k];
                    if (!(t[j] < INFINITY)) wrong = true;
                }
            }
            top = fmaxf(top, t[j]);
        }
        float norm;  // log p = (t - top) / T - norm
        if (a.lse) {
            top = 0.f;
            norm = a.lse[b];
            if (!(fabsf(norm) < INFINITY)) wrong = true;
        } else {
            top = block_max(top, 0);
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (t[j] > -INFINITY) s += expf((t[j] - top) * invT);
            s = block_add(s, 1);
            norm = s > 0.f ? logf(s) : 0.f;
        }
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const bool any = t[j] > -INFINITY || t[j] != t[j];
            logp[j] = any ? (t[j] - top) * invT - norm : 0.f;
            const float p = any ? expf(logp[j]) : 0.f;
            sum += p;
            const int k = tid + j * kDThreads;
            const int o = id[j] >= 0 ? part.offset(id[j]) : -1;
            sh->id[k] = o >= 0 && o < part.n * kPer ? id[j] : -1;
            sh->p[k] = p;
        }
        if (__any_sync(kAllLanes, off) && lane == 0) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
        bad = __syncthreads_or(wrong);
        sum_p = block_add(sum, 2);
    }

    // Marks the part's columns in a bitmap, one bit a logit; sh->twice: a column was marked before.
    __device__ void mark(uint32_t *bits) {
        for (int i = tid; i < (part.n * kPer + 31) / 32; i += kDThreads) bits[i] = 0;
        if (tid == 0) sh->twice = 0;
        __syncthreads();
        for (int k = tid; k < a.K; k += kDThreads) {
            const int x = sh->id[k];
            if (x < 0) continue;
            const int o = part.offset(x);
            if (atomicOr(&bits[o >> 5], 1u << (o & 31)) >> (o & 31) & 1u) sh->twice = 1;
        }
        // read after the next block barrier
    }

    // g: the row's gradient scale (w times the upstream gradient, over T).
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
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int x = part.index(i, q);
                if (x >= 0 && x < a.V) store_one(x, v[q]);
            }
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
    __device__ void fill(float v) const {
        float g[kPer];
#pragma unroll
        for (int q = 0; q < kPer; ++q) g[q] = v;
        const bool same = alike();
        for (int i = tid; i < part.n; i += kDThreads) store(i, g, same);
    }
    // P q_v / T for every column of the part (logits from `get`), then the teacher's columns.
    template <class G, class S>
    __device__ void gradient(float g, float m, float S_, G get, S logit_at) {
        const float A = g * sum_p / S_;
        const bool same = alike();
        float own[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int k = tid + j * kDThreads;
            own[j] = k < a.K && sh->id[k] >= 0 ? logit_at(sh->id[k]) : 0.f;  // before anything is written: grad may be student
        }
        __syncthreads();
        const bool twice = sh->twice != 0;
#pragma unroll 4
        for (int i = tid; i < part.n; i += kDThreads) {
            float l[kPer];
            P::unpack(get(i), l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) l[q] = A * ptx::ex2((l[q] - m) * c);
            store(i, l, same);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const int k = tid + j * kDThreads;
            const int x = k < a.K ? sh->id[k] : -1;
            if (x < 0) continue;
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

// Running maximum and exp-sum of a thread's logits.
template <int EB>
__device__ __forceinline__ void running(const uint4 &v, float c, float &m, float &s) {
    constexpr int kPer = 16 / EB;
    float l[kPer];
    Part<EB>::unpack(v, l);
    float top = l[0];
#pragma unroll
    for (int q = 1; q < kPer; ++q) top = fmaxf(top, l[q]);
    if (top > m) {
        s *= ptx::ex2((m - top) * c);  // m = -inf: s is 0
        m = top;
    }
    if (m == -INFINITY) {  // nothing but masked logits, or NaN, so far
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            if (l[q] != l[q]) s = NAN;
        return;
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q) s += ptx::ex2((l[q] - m) * c);
}

// Loss and row statistics, and with GRAD the gradient: a cluster per row.
template <int EB, bool GRAD>
__global__ void __launch_bounds__(kDThreads) distill_kernel(const DistillArgs a) {
    extern __shared__ uint4 dyn[];
    DistillShared *sh = reinterpret_cast<DistillShared *>(dyn);
    uint4 *buf = dyn + sizeof(DistillShared) / 16;
    const uint32_t rank = cluster_rank();
    const int b = blockIdx.x / a.cluster;
    Distill<EB> d(a, sh, b, rank);
    const int tid = d.tid;
    const float w = a.weight ? a.weight[b] : 1.f;
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
    const int n = d.part.n;
    if (GRAD) {
        for (int i = tid; i < n; i += kDThreads) d.part.copy(buf, i);
        copies_commit();
    }
    float logp[kSlots];
    d.teacher(logp);
    if (GRAD) {
        d.mark(reinterpret_cast<uint32_t *>(buf + a.part));
        copies_wait<0>();
    }
    float m = -INFINITY, s = 0.f;
    if (GRAD) {
        for (int i = tid; i < n; i += kDThreads) {
            d.part.mend(buf, i);
            running<EB>(buf[i], d.c, m, s);
        }
    } else {
        int i = tid;
        for (; i + 3 * kDThreads < n; i += 4 * kDThreads) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = d.part.fetch(i + j * kDThreads);
#pragma unroll
            for (int j = 0; j < 4; ++j) running<EB>(v[j], d.c, m, s);
        }
        for (; i < n; i += kDThreads) running<EB>(d.part.fetch(i), d.c, m, s);
    }
    // the block's, then the cluster's
    const float bm = d.block_max(m, 0);
    s = s == s && m == -INFINITY ? 0.f : s * ptx::ex2((m - bm) * d.c);
    s = d.block_add(s, 1);  // after this barrier the part is in shared memory for every thread
    auto logit_at = [&](int x) {
        return GRAD ? Part<EB>::logit(buf, d.part.offset(x)) : Part<EB>::logit(a.student, static_cast<size_t>(b) * a.V + x);
    };
    const float invT = 1.f / a.T;
    float dot = 0.f, ps = 0.f;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
        const int k = tid + j * kDThreads;
        if (k >= a.K || sh->id[k] < 0) continue;
        const float p = sh->p[k];
        if (p == 0.f) continue;
        const float l = logit_at(sh->id[k]);
        dot += p * (logp[j] - (l == -INFINITY ? l : (l - bm) * invT));  // a masked token the teacher wants: +inf
        ps += p;
    }
    dot = d.block_add(dot, 2);
    ps = d.block_add(ps, 3);
    cluster_wait();
    if (tid < a.cluster) {
        const uint32_t to = peer(&sh->slot[rank], tid);
        st_peer(to, __float_as_uint(bm));
        st_peer(to + 4, __float_as_uint(s));
        st_peer(to + 8, __float_as_uint(dot));
        st_peer(to + 12, __float_as_uint(ps));
    }
    cluster_sync();
    m = -INFINITY;
    for (int r = 0; r < a.cluster; ++r) m = fmaxf(m, sh->slot[r].x);
    s = 0.f;
    dot = 0.f;
    for (int r = 0; r < a.cluster; ++r) {
        const float4 v = sh->slot[r];
        s += v.x == -INFINITY ? v.y : v.y * ptx::ex2((v.x - m) * d.c);  // a part of masked logits has sum 0 (or NaN)
        if (v.w != 0.f) dot += v.z + v.w * ((m - v.x) * invT);
    }
    const bool bad = d.bad || !(m < INFINITY && s > 0.f && s < INFINITY);  // NaN, +inf, or nothing but -inf
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
        d.gradient(w * invT, m, s, [&](int i) { return buf[i]; }, logit_at);
}

// The gradient alone, from the logits and a forward call's statistics: a CTA per part of a row.
template <int EB>
__global__ void __launch_bounds__(kDThreads) distill_backward_kernel(const DistillArgs a) {
    extern __shared__ uint4 dyn[];
    DistillShared *sh = reinterpret_cast<DistillShared *>(dyn);
    const int b = blockIdx.x / a.cluster;
    Distill<EB> d(a, sh, b, blockIdx.x % a.cluster);
    const float up = (a.weight ? a.weight[b] : 1.f) * a.grad_loss[b];
    if (up == 0.f) {
        d.fill(0.f);
        return;
    }
    float logp[kSlots];
    d.teacher(logp);
    d.mark(reinterpret_cast<uint32_t *>(dyn + sizeof(DistillShared) / 16));
    const float m = a.stats[2 * static_cast<size_t>(b)], s = a.stats[2 * static_cast<size_t>(b) + 1];
    if (d.bad || !(fabsf(m) < INFINITY && s > 0.f && s < INFINITY)) {
        if (d.tid == 0) atomicOr(a.status, SPEC_DEV_NONFINITE);
        d.fill(NAN);
        return;
    }
    d.gradient(up / a.T, m, s, [&](int i) { return d.part.fetch(i); },
               [&](int x) { return Part<EB>::logit(a.student + (static_cast<size_t>(b) * a.V + x) * EB, 0); });
}

}  // namespace vocab
}  // namespace spec
