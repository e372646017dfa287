// distill.cuh -- distillation from a teacher's largest logits: the loss of each
// row and its gradient.
//
//   q = softmax(s / T),  p_k = exp(t_k / T - lse)  (or the softmax of the K entries),  P = sum_k p_k
//   loss = w sum_k p_k (log p_k - log q_{id_k}),   d loss / d s_v = (w / T) (P q_v - sum_{k: id_k = v} p_k)
//
// HBM bounds all three forms.  Loss and gradient in one call read each logit once:
// a cluster keeps the row in its CTAs' shared memory (64 KB each, three CTAs an SM)
// between the exp-sum and the gradient, and goes on to another row: as a thread
// takes a vector for the gradient, it sends for the next row's into its place, so
// that memory is read while the gradient is written and the next teacher weighed.
// A row has one cluster barrier.  2048 rows of 128256 bf16 take 214 us (4.7 TB/s of
// reads and writes; 147 at the copy rate).  What holds it back is the row's own chain
// (exp-sum 2.8 us, barrier and merging 4, gradient 3.6: 11 us a row, in which an SM
// moves 384 KB) and steady write-back.  Tried and slower: no prefetch (223 us), one
// CTA a row with the second read from L2 (253), 44 KB or 37 KB parts (225 to 260), 128
// or 512 threads.
//
// The loss alone (one CTA a row where rows are many: 100 us there, 5.3 TB/s) and the
// gradient alone (shares of 96 KB: 162 us, 6.5 TB/s, 95 % of the copy rate) stream;
// their first loads are under way while the teacher is weighed.
//
// A CTA writes its share of P q_v densely and then, after a block barrier, the
// columns of its own teacher entries over it; an entry's column is written by one
// thread (the first slot that names it), which adds the slots that name it too in
// their order, so the gradient does not depend on timing.
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
    float2 part[kDWarps];           // each warp's share of the teacher's normaliser: a maximum and a sum
    float2 slot[2][kMaxCluster * kDWarps];  // of each warp of the row: its maximum and exp-sum
    float loss[2][kMaxCluster * kDWarps];   // and (rank 0) its share of the loss
    int twice[2];                   // some column is named by two entries
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

// Exponents (l - m) c are formed as l c - q, q the rounded m c, in one operation a pair, where |q| is below
// this: q is then off by 2^-13 at most, which is made up for to the first order (the second: 2^-28).
// Beyond it (finite masks, small temperatures) they are computed as they stand: q could be off by
// many octaves, and a row's weights or their sum would overflow or vanish.
constexpr float kPlainLimit = 4096.f;
__device__ __forceinline__ bool plain(float q) { return fabsf(q) < kPlainLimit; }
// 2^((l - m) c) of two logits: as l c - q (PLAIN), or as it stands.
template <bool PLAIN>
__device__ __forceinline__ unsigned long long exp2_pair(float l0, float l1, float c, float m, float q) {
    float x, y;
    split(PLAIN ? fma2(pair(l0, l1), pair(c, c), pair(-q, -q)) : mul2(add2(pair(l0, l1), pair(-m, -m)), pair(c, c)), x, y);
    return pair(ptx::ex2(x), ptx::ex2(y));
}

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
        tid = threadIdx.x;
        lane = tid & 31;
        warp = tid >> 5;
        c = kLog2ef / a.T;
        invT = 1.f / a.T;
        place(row, rank);
    }
    __device__ __forceinline__ void place(int row, uint32_t rank) {
        b = row;
        part.place(a.student, a.student_end, a.V, b, rank, a.part);
    }
    // The teacher's entries, on their way while the copies of the logits are issued.
    __device__ __forceinline__ void ask_teacher(int row, int32_t (&ids)[SLOTS], float (&logits)[SLOTS]) const {
        const size_t at = static_cast<size_t>(row) * a.K;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const int k = tid + j * kDThreads;
            ids[j] = -1;
            logits[j] = -INFINITY;
            if (k < a.K) {
                ids[j] = __ldg(a.ids + at + k);
                logits[j] = __ldg(a.top + at + k);
            }
        }
    }
    // Every CTA of a row weighs all K entries (P has to be the same everywhere).  First each warp's share
    // of the normaliser, then, after a block barrier, log p and p, which it keeps for the entries in its
    // part.  Their columns are marked in a bitmap, one bit a logit, cleared before; sh->twice[turn]: a
    // column was marked before.
    __device__ __forceinline__ void teacher_share() {
        float top = -INFINITY, s = 0.f;
        bool wrong = false, off = false;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            if (id[j] >= a.V || id[j] < -1) off = true, id[j] = -1;
            if (id[j] < 0) t[j] = -INFINITY;
            if (!(t[j] < INFINITY)) wrong = true;
            top = fmaxf(top, t[j]);
        }
        if (off) atomicOr(a.status, SPEC_DEV_BAD_TOKEN);
        if (a.lse) {
            top = 0.f;  // log p = t / T - lse
            const float z = __ldg(a.lse + b);
            if (!(z < INFINITY)) wrong = true;
            const float rest = fmaf(-invT, a.T, 1.f) * invT;  // 1 / T - invT
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const bool any = t[j] > -INFINITY;
                if (any && z == -INFINITY) wrong = true;  // (a masked row's teacher has no entries)
                // t / T as a pair: it may be far larger than its difference from lse
                const float h = __fmul_rn(t[j], invT), l = fabsf(h) < 1e30f ? fmaf(t[j], rest, fmaf(t[j], invT, -h)) : 0.f;
                t[j] = any ? (h - z) + l : -INFINITY;
                s += any ? expf(t[j]) : 0.f;
            }
        } else if (__any_sync(kAllLanes, top > -INFINITY)) {
            top = warp_max(top);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) s += t[j] > -INFINITY ? expf((t[j] - top) * invT) : 0.f;
        }
        if (wrong) s = NAN;
        if (__any_sync(kAllLanes, s != 0.f)) s = warp_add(s);
        if (lane == 0) sh->part[warp] = make_float2(top, s);
    }
    __device__ __forceinline__ void teacher_finish(uint32_t *bits, int turn) {
        float top = -INFINITY, s = 0.f;
#pragma unroll
        for (int i = 0; i < kDWarps; ++i) top = fmaxf(top, sh->part[i].x);
#pragma unroll
        for (int i = 0; i < kDWarps; ++i) {
            const float2 v = sh->part[i];
            s += a.lse ? v.y : v.y == 0.f ? 0.f : v.y * expf((v.x - top) * invT);
        }
        sum_p = a.lse || !(s > 0.f) ? s : 1.f;  // (NaN stays)
        const float norm = !a.lse && s > 0.f ? logf(s) : 0.f;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const bool any = t[j] > -INFINITY;
            if (!a.lse) t[j] = any ? (t[j] - top) * invT - norm : 0.f;
            const float p = any ? expf(t[j]) : 0.f;
            const int k = tid + j * kDThreads;
            const int o = id[j] >= 0 ? part.offset(id[j]) : -1;
            if (o < 0 || o >= part.n * kPer) id[j] = -1;
            sh->id[k] = id[j];
            sh->p[k] = p;
            if (bits && id[j] >= 0 && (atomicOr(&bits[o >> 5], 1u << (o & 31)) >> (o & 31) & 1u)) sh->twice[turn] = 1;
        }
    }
    __device__ __forceinline__ void clear(uint32_t *bits) {
        for (int i = tid; i < (a.part * kPer + 31) / 32; i += kDThreads) bits[i] = 0;
    }

    // The vectors of the part that lie in the row alone: [first, end).  The others, at most the row's
    // first and last, are written by logit, as all are where the tensors' vectors do not lie alike.
    __device__ __forceinline__ int whole_from() const { return part.n > 0 && part.edge(0) ? 1 : 0; }
    __device__ __forceinline__ int whole_upto() const { return part.n > 0 && part.edge(part.n - 1) ? part.n - 1 : part.n; }
    static __device__ __forceinline__ uint4 packed(const float (&v)[kPer]) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (EB == 4)
                w[q] = __float_as_uint(v[q]);
            else
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[q]) : "f"(v[(2 * q + 1) % kPer]), "f"(v[(2 * q) % kPer]));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The gradients make(load(i), floats) of every vector i, into whole vectors' places or by logit.  A
    // batch of loads goes before its stores: grad may be student, so the compiler would keep their order
    // and wait for each load alone.
    static constexpr int kBatch = 4;
    // The whole vectors' first batch for write(), loaded ahead of what it waits for.
    template <class L>
    __device__ __forceinline__ void ask_first(L load, uint4 (&v)[kBatch]) const {
        const int upto = whole_upto(), i = tid < whole_from() ? tid + kDThreads : tid;
        if (i + (kBatch - 1) * kDThreads < upto) {
            load(i, v);
            return;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            uint4 one[1] = {make_uint4(0, 0, 0, 0)};
            if (i + j * kDThreads < upto) load(i + j * kDThreads, one);
            v[j] = one[0];
        }
    }
    template <class L, class F>
    __device__ __forceinline__ void write(L load, F make, const uint4 (*ahead)[kBatch] = nullptr) const {
        const bool alike = ((reinterpret_cast<uintptr_t>(a.grad) ^ reinterpret_cast<uintptr_t>(a.student)) & 15) == 0;
        const int from = alike ? whole_from() : 0, upto = alike ? whole_upto() : 0;
        int i = tid < from ? tid + kDThreads : tid;
        unsigned char *dst = a.grad + (part.at(0) - a.student) + static_cast<size_t>(i) * 16;
        auto put = [](unsigned char *at, const uint4 &v) {
            asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(__cvta_generic_to_global(at)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w));
        };
        if (ahead && alike) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (i + j * kDThreads >= upto) break;
                float l[kPer];
                make((*ahead)[j], l);
                put(dst + 16 * j * kDThreads, packed(l));
            }
            i += kBatch * kDThreads;
            dst += 16 * kBatch * kDThreads;
        }
        for (; i + (kBatch - 1) * kDThreads < upto; i += kBatch * kDThreads, dst += 16 * kBatch * kDThreads) {
            uint4 v[kBatch];
            load(i, v);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                float l[kPer];
                make(v[j], l);
                put(dst + 16 * j * kDThreads, packed(l));
            }
        }
        uint4 v[1];
        for (; i < upto; i += kDThreads, dst += 16 * kDThreads) {
            float l[kPer];
            load(i, v);
            make(v[0], l);
            put(dst, packed(l));
        }
        // the rest: vector 0 before `from`, and those from `upto` on
        for (int j = tid < from || upto == 0 ? tid : upto + (tid + kDThreads - upto % kDThreads) % kDThreads; j < part.n;
             j = j < from && upto > 0 ? upto + (tid + kDThreads - upto % kDThreads) % kDThreads : j + kDThreads) {
            float l[kPer];
            load(j, v);
            make(v[0], l);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const int x = part.index(j, q);
                if (x >= 0 && x < a.V) store_one(x, l[q]);
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
    __device__ __forceinline__ void fill(float g) const {
        write([](int, auto &v) { v[0] = make_uint4(0, 0, 0, 0); },
              [&](const uint4 &, float(&v)[kPer]) {
#pragma unroll
                  for (int q = 0; q < kPer; ++q) v[q] = g;
              });
    }
    template <bool PLAIN, class G>
    __device__ __forceinline__ void dense(float m, float q, float A, G get, const uint4 (*ahead)[kBatch]) const {
        write(
            get,
            [&](const uint4 &v, float(&l)[kPer]) {
                P::unpack(v, l);
#pragma unroll
                for (int e = 0; e < kPer; e += 2) split(mul2(exp2_pair<PLAIN>(l[e], l[e + 1], c, m, q), pair(A, A)), l[e], l[e + 1]);
            },
            ahead);
    }
    // The logits of this thread's entries.
    template <class L>
    __device__ __forceinline__ void own_logits(L logit_at, float (&own)[SLOTS]) const {
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) own[j] = id[j] >= 0 ? logit_at(id[j]) : 0.f;
    }
    // (w / T) P q_v for every column of the part (logits from `get`), then, after a block barrier, the
    // teacher's columns over it.  g: w / T; m, S: the row's maximum and exp-sum; own: read before
    // anything is written, as grad may be student.
    template <class G>
    __device__ __forceinline__ void gradient(float g, float m, float S, const float (&own)[SLOTS], int turn, G get,
                                             const uint4 (*ahead)[kBatch] = nullptr) {
        // where exponents are l c - q, q's rounding goes into the factor
        const float q = __fmul_rn(m, c), A = g * sum_p / S;
        if (plain(q))
            dense<true>(m, q, A * (1.f + 0.6931471805599453f * fmaf(-m, c, q)), get, ahead);
        else
            dense<false>(m, q, A, get, ahead);
        __syncthreads();
        const bool twice = sh->twice[turn] != 0;
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

// A thread's running maximum m and sum of 2^((l - m) c), or, where plain(q), of 2^(l c - q); at the end
// the rounding of q goes into the sum.
template <int EB>
struct Running {
    using P = Part<EB>;
    float m = -INFINITY, q = -INFINITY;
    unsigned long long s = 0;  // a pair

    template <int N>
    __device__ __forceinline__ void add(const uint4 (&v)[N], float c) {
        const float top = P::vectors_max(v);  // NaN if there is one
        if (!(top <= m) && m == m) {      // (a NaN stays)
            const float to = __fmul_rn(top, c);  // (rounded, as weigh() subtracts it: not to be fused into q - to)
            // from the old maximum's form to the new one's
            const float x = plain(q) ? (plain(to) ? q - to : fmaf(-top, c, q)) : plain(to) ? fmaf(m, c, -to) : (m - top) * c;
            const float f = m > -INFINITY ? ptx::ex2(x) : 0.f;
            s = mul2(s, pair(f, f));
            m = top;
            q = to;
        }
        if (m == -INFINITY) return;  // masked so far
        if (plain(q))
            weigh<true>(v, c);
        else
            weigh<false>(v, c);
    }
    template <bool PLAIN, int N>
    __device__ __forceinline__ void weigh(const uint4 (&v)[N], float c) {
        unsigned long long sum = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float l[P::kPer];
            P::unpack(v[j], l);
            unsigned long long e[P::kPer / 2];
#pragma unroll
            for (int i = 0; i < P::kPer / 2; ++i) e[i] = exp2_pair<PLAIN>(l[2 * i], l[2 * i + 1], c, m, q);
#pragma unroll
            for (int h = P::kPer / 4; h; h >>= 1)
#pragma unroll
                for (int i = 0; i < h; ++i) e[i] = add2(e[i], e[i + h]);
            sum = j ? add2(sum, e[0]) : e[0];
        }
        s = add2(s, sum);
    }
    // A thread's vectors of the part, from global memory; meanwhile() runs while the first are on their way.
    template <class F>
    __device__ __forceinline__ void stream(const P &part, int tid, float c, F meanwhile) {
        constexpr int kBatch = 4;
        const int n = part.n;
        uint4 v[kBatch];
        auto load = [&](int i) {
            if (i > 0 && i + (kBatch - 1) * kDThreads < n - 1) {
                const uint4 *src = reinterpret_cast<const uint4 *>(part.at(i));
#pragma unroll
                for (int j = 0; j < kBatch; ++j) v[j] = src[j * kDThreads];
            } else {  // (-inf beyond the end)
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    v[j] = P::nothing();
                    if (i + j * kDThreads < n) v[j] = part.fetch(i + j * kDThreads);
                }
            }
        };
        load(tid);
        meanwhile();
        for (int i = tid; i < n;) {
            add(v, c);
            i += kBatch * kDThreads;
            if (i < n) load(i);
        }
    }
    __device__ __forceinline__ float sum(float c) const {
        float x, y;
        split(s, x, y);
        return (x + y) * (plain(q) ? 1.f + 0.6931471805599453f * fmaf(-m, c, q) : 1.f);
    }
};

// A warp's maximum and exp-sum, to every CTA of the row; row_sums() after the row's barrier.
template <int EB, int SLOTS>
__device__ __forceinline__ void post_sums(Distill<EB, SLOTS> &d, const Running<EB> &r, uint32_t rank, int turn) {
    const float m = warp_max(r.m);  // (NaN passes through the sums)
    const float s = warp_add(r.m == -INFINITY ? 0.f : r.sum(d.c) * ptx::ex2((r.m - m) * d.c));
    if (d.lane < d.a.cluster) st_peer(peer(&d.sh->slot[turn][rank * kDWarps + d.warp], d.lane), pair(m, s));
}
template <int EB, int SLOTS>
__device__ __forceinline__ void row_sums(const Distill<EB, SLOTS> &d, int turn, float *row_m, float *row_s) {
    constexpr int kEach = (kMaxCluster * kDWarps + 31) / 32;
    float2 v[kEach];
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int g = i * 32 + d.lane;
        v[i] = g < d.a.cluster * kDWarps ? d.sh->slot[turn][g] : make_float2(-INFINITY, 0.f);
        m = fmaxf(m, v[i].x);
    }
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < kEach; ++i) s += v[i].x == -INFINITY ? v[i].y : v[i].y * ptx::ex2((v[i].x - m) * d.c);  // (masked: 0, or NaN)
    *row_m = m;
    *row_s = warp_add(s);
}
// This warp's share of the row's loss, to the CTA of rank 0: sum of p (log p - log q).
template <int EB, int SLOTS>
__device__ __forceinline__ void post_loss(Distill<EB, SLOTS> &d, const float (&own)[SLOTS], float m, float s, uint32_t rank, int turn) {
    const float log_s = logf(s);
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < SLOTS; ++j) {
        const float p = d.id[j] >= 0 ? d.sh->p[d.tid + j * kDThreads] : 0.f;
        // a masked token that the teacher wants: +inf
        if (p != 0.f) v += p * (d.t[j] - (own[j] == -INFINITY ? own[j] : (own[j] - m) * d.invT) + log_s);
    }
    if (__any_sync(kAllLanes, v != 0.f)) v = warp_add(v);
    if (d.lane == 0) st_peer(peer(&d.sh->loss[turn][rank * kDWarps + d.warp], 0), __float_as_uint(v));
}
// A row's loss and statistics, by a warp of rank 0 after the barrier that follows post_loss.
template <int EB, int SLOTS>
__device__ __forceinline__ void write_row(const Distill<EB, SLOTS> &d, int row, float w, bool sound, float m, float s, int turn) {
    float v = 0.f;
    for (int g = d.lane; g < d.a.cluster * kDWarps; g += 32) v += d.sh->loss[turn][g];
    v = warp_add(v);
    if (d.lane == 0) {
        d.a.loss[row] = sound ? w * v : NAN;
        reinterpret_cast<float2 *>(d.a.stats)[row] = sound ? make_float2(m, s) : make_float2(NAN, NAN);
        if (!sound) atomicOr(d.a.status, SPEC_DEV_NONFINITE);
    }
}
template <int EB, int SLOTS>
__device__ __forceinline__ bool row_sound(const Distill<EB, SLOTS> &d, float m, float s) {  // not: NaN, +inf, or nothing but -inf
    return d.sum_p == d.sum_p && m < INFINITY && s > 0.f && s < INFINITY;
}
template <int EB, int SLOTS>
__device__ __forceinline__ void ignored(const Distill<EB, SLOTS> &d, uint32_t rank) {
    if (rank == 0 && d.tid == 0) {
        d.a.loss[d.b] = 0.f;
        reinterpret_cast<float2 *>(d.a.stats)[d.b] = make_float2(0.f, 0.f);
    }
}

// Loss and row statistics: a cluster per row.
template <int EB, int SLOTS>
__global__ void __launch_bounds__(kDThreads, 4) distill_loss_kernel(const DistillArgs a) {
    extern __shared__ uint4 dyn[];
    const uint32_t rank = cluster_rank();
    Distill<EB, SLOTS> d(a, reinterpret_cast<DistillShared<SLOTS> *>(dyn), blockIdx.x / a.cluster, rank);
    const float w = a.weight ? __ldg(a.weight + d.b) : 1.f;
    if (w == 0.f) {  // its logits are not read
        ignored(d, rank);
        return;
    }
    cluster_arrive();
    d.ask_teacher(d.b, d.id, d.t);
    Running<EB> r;
    r.stream(d.part, d.tid, d.c, [&]() { d.teacher_share(); });
    cluster_wait();  // the peers have started
    post_sums(d, r, rank, 0);
    cluster_sync();
    float m, s, own[SLOTS];
    row_sums(d, 0, &m, &s);
    d.teacher_finish(nullptr, 0);
    d.own_logits([&](int x) { return Part<EB>::logit(a.student + (static_cast<size_t>(d.b) * a.V + x) * EB, 0); }, own);
    post_loss(d, own, m, s, rank, 0);
    cluster_sync();
    if (rank == 0 && d.warp == 0) write_row(d, d.b, w, row_sound(d, m, s), m, s, 0);
}

// Loss, statistics and gradient: a cluster takes every gridDim-th row.  A row has one cluster barrier,
// between its sums and its gradient, which also carries the loss of the row before.
template <int EB, int SLOTS>
__global__ void __launch_bounds__(kDThreads, kTrainCtas) distill_kernel(const DistillArgs a) {
    extern __shared__ uint4 dyn[];
    DistillShared<SLOTS> *sh = reinterpret_cast<DistillShared<SLOTS> *>(dyn);
    uint4 *buf = dyn + sizeof(DistillShared<SLOTS>) / 16;
    uint32_t *bits = reinterpret_cast<uint32_t *>(buf + a.part);
    const uint32_t rank = cluster_rank();
    const int step = static_cast<int>(gridDim.x) / a.cluster;
    Distill<EB, SLOTS> d(a, sh, static_cast<int>(blockIdx.x) / a.cluster, rank);
    const int tid = d.tid;
    cluster_arrive();
    auto weight = [&](int row) { return row < a.N && a.weight ? __ldg(a.weight + row) : 1.f; };
    // the first row of weight other than 0 from `row` on; those before it get their zeros
    auto live = [&](int row, float &w) {
        while (row < a.N && w == 0.f) {
            Distill<EB, SLOTS> z(a, sh, row, rank);
            z.fill(0.f);
            ignored(z, rank);
            row += step;
            w = weight(row);
        }
        return row;
    };
    float w = weight(d.b);
    int row = live(d.b, w);
    if (row >= a.N) {
        cluster_wait();
        return;
    }
    d.place(row, rank);
    d.ask_teacher(row, d.id, d.t);
    d.part.copy_all(buf, tid, kDThreads);
    copies_commit();
    d.clear(bits);
    if (tid < 2) sh->twice[tid] = 0;
    struct {
        int row = -1;
        float w, m, s;
        bool sound;
    } last;  // the row before, whose loss is on its way
    for (int turn = 0, first = 1;; turn ^= 1, first = 0) {
        float next_w = weight(row + step);
        d.teacher_share();
        copies_wait<0>();
        d.part.mend_all(buf, tid, kDThreads);
        Running<EB> r;
        int i = tid;
        const int n = d.part.n;
        for (; i + 3 * kDThreads < n; i += 4 * kDThreads) {
            const uint4 v[4] = {buf[i], buf[i + kDThreads], buf[i + 2 * kDThreads], buf[i + 3 * kDThreads]};
            r.add(v, d.c);
        }
        for (; i < n; i += kDThreads) {
            const uint4 v[1] = {buf[i]};
            r.add(v, d.c);
        }
        if (first) cluster_wait();  // the peers have started
        post_sums(d, r, rank, turn);
        cluster_sync();
        if (last.row >= 0 && rank == 0 && d.warp == 0) write_row(d, last.row, last.w, last.sound, last.m, last.s, turn ^ 1);
        float m, s, own[SLOTS];
        row_sums(d, turn, &m, &s);
        d.teacher_finish(bits, turn);
        d.own_logits([&](int x) { return Part<EB>::logit(buf, d.part.offset(x)); }, own);
        const bool sound = row_sound(d, m, s);
        post_loss(d, own, m, s, rank, turn);
        const int next = live(row + step, next_w);
        // the next row's vectors into the places of those taken
        Part<EB> ahead;
        int from = 0, upto = 0;
        int32_t ids[SLOTS];
        float logits[SLOTS];
        if (next < a.N) {
            d.ask_teacher(next, ids, logits);
            ahead.place(a.student, a.student_end, a.V, next, rank, a.part);
            from = ahead.copy_from();
            upto = ahead.copy_upto();
        }
        auto take = [&](int j, auto &v) {
            constexpr int N = static_cast<int>(sizeof(v) / sizeof(uint4));
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = buf[j + e * kDThreads];
            // (an address that waits for v: the copy must not overtake the read)
            const uint32_t dst = smem_u32(buf + j);
            const unsigned char *src = ahead.at(j);
            if (j >= from && j + (N - 1) * kDThreads < upto) {
#pragma unroll
                for (int e = 0; e < N; ++e) copy16(dst + 16 * e * kDThreads + (v[e].w & a.zero), src + 16 * e * kDThreads);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (j + e * kDThreads >= from && j + e * kDThreads < upto)
                        copy16(dst + 16 * e * kDThreads + (v[e].w & a.zero), src + 16 * e * kDThreads);
            }
        };
        __syncthreads();  // the entries' logits have been read, the bitmap is complete
        if (sound) {
            d.gradient(w * d.invT, m, s, own, turn, take);
        } else {
            d.fill(NAN);
            uint4 v[1];
            for (int j = tid; j < n; j += kDThreads) take(j, v);
            __syncthreads();
        }
        last.row = row;
        last.w = w;
        last.m = m;
        last.s = s;
        last.sound = sound;
        if (next >= a.N) {
            cluster_sync();
            if (rank == 0 && d.warp == 0) write_row(d, last.row, last.w, last.sound, last.m, last.s, turn);
            return;
        }
        for (int j = tid; j < upto; j += kDThreads)
            if (j >= n) copy16(smem_u32(buf + j), ahead.at(j));
        copies_commit();
        d.clear(bits);  // (marked after the next barrier)
        if (tid == 0) sh->twice[turn ^ 1] = 0;
        row = next;
        w = next_w;
        d.b = next;
        d.part = ahead;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            d.id[j] = ids[j];
            d.t[j] = logits[j];
        }
    }
}

// The gradient alone, from the logits and a forward call's statistics: a CTA per part of a row.
template <int EB, int SLOTS>
__global__ void __launch_bounds__(kDThreads, 4) distill_backward_kernel(const DistillArgs a) {
    extern __shared__ uint4 dyn[];
    DistillShared<SLOTS> *sh = reinterpret_cast<DistillShared<SLOTS> *>(dyn);
    uint32_t *bits = reinterpret_cast<uint32_t *>(dyn + sizeof(DistillShared<SLOTS>) / 16);
    const int b = blockIdx.x / a.cluster;
    Distill<EB, SLOTS> d(a, sh, b, blockIdx.x % a.cluster);
    const float w = a.weight ? __ldg(a.weight + b) : 1.f, grad_loss = __ldg(a.grad_loss + b), up = w * grad_loss;
    if (w == 0.f || grad_loss == 0.f || up == 0.f) {  // (0 times an infinite factor is not 0)
        d.fill(0.f);
        return;
    }
    auto fetch = [&](int i, auto &v) {
        const uint4 *src = reinterpret_cast<const uint4 *>(d.part.at(i));
        if (sizeof(v) > sizeof(uint4) || !d.part.edge(i)) {  // (a batch is of whole vectors)
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(v) / sizeof(uint4)); ++j) v[j] = src[j * kDThreads];
        } else {
            v[0] = d.part.fetch(i);
        }
    };
    uint4 first[Distill<EB, SLOTS>::kBatch];
    d.ask_teacher(b, d.id, d.t);
    d.ask_first(fetch, first);
    const float2 ms = __ldg(reinterpret_cast<const float2 *>(a.stats) + b);
    d.clear(bits);
    if (d.tid == 0) sh->twice[0] = 0;
    d.teacher_share();
    __syncthreads();
    d.teacher_finish(bits, 0);
    if (!row_sound(d, fabsf(ms.x) < INFINITY ? ms.x : INFINITY, ms.y)) {
        if (d.tid == 0) atomicOr(a.status, SPEC_DEV_NONFINITE);
        d.fill(NAN);
        return;
    }
    float own[SLOTS];
    d.own_logits([&](int x) { return Part<EB>::logit(a.student + (static_cast<size_t>(b) * a.V + x) * EB, 0); }, own);
    __syncthreads();
    d.gradient(up * d.invT, ms.x, ms.y, own, 0, fetch, &first);
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
    const long long most = form == kLossGrad ? kPartBytes : form == kLoss ? kLossBytes : kBackwardBytes;
    const long long limit = form == kBackward ? 1 << 20 : kMaxCluster;
    long long cs = std::min(limit, (vecs * 16 + most - 1) / most);
    while (2 * cs <= kMaxCluster && a.N * cs < kWaves * di.sms && vecs / cs > 2 * kDThreads) cs *= 2;
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
    if (form == kLossGrad) {  // as many rows under way as there are clusters at a time
        const int most_rows = resident_clusters(dev, reinterpret_cast<const void *>(kernel), cfg);
        if (most_rows > 0 && most_rows < a.N) cfg.gridDim = dim3(static_cast<unsigned>(most_rows * cs));
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(SPEC_ERR_CUDA, "distillation launch (N=%d, cluster=%lld, smem=%zu): %s", a.N, cs, smem, cudaGetErrorString(e));
    return SPEC_OK;
}

template <int EB>
spec_status launch_distill(const DistillArgs &a, int form, cudaStream_t stream) {
    if (a.K <= kDThreads) {
        if (form == kLoss) return go(distill_loss_kernel<EB, 1>, a, EB, 1, form, stream);
        if (form == kLossGrad) return go(distill_kernel<EB, 1>, a, EB, 1, form, stream);
        return go(distill_backward_kernel<EB, 1>, a, EB, 1, form, stream);
    }
    if (form == kLoss) return go(distill_loss_kernel<EB, 4>, a, EB, 4, form, stream);
    if (form == kLossGrad) return go(distill_kernel<EB, 4>, a, EB, 4, form, stream);
    return go(distill_backward_kernel<EB, 4>, a, EB, 4, form, stream);
}

}  // namespace vocab
}  // namespace spec
