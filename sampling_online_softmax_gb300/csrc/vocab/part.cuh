// part.cuh -- one CTA's share of a row: the row's 16-byte vectors, on the 16-byte
// grid of global memory, are dealt out to the CTAs in contiguous runs, so every
// vector belongs to one CTA and only the row's first and last can hold logits
// of a neighbouring row (read as -inf).  Bytes outside the tensor are never read.
#pragma once

#include "../ptx.cuh"
#include "cluster.cuh"

namespace spec {
namespace vocab {

// Pairs of floats in one instruction each.
__device__ __forceinline__ unsigned long long pair(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(unsigned long long p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int EB>
struct Part {
    static constexpr int kPer = 16 / EB;  // logits per vector
    const unsigned char *win;             // the row's first vector (the row starts `lead` logits into it)
    const unsigned char *base, *end;      // the tensor
    int lead, first, n, total, V;         // this CTA's vectors: first .. first + n - 1 of the row's total

    __device__ __forceinline__ void place(const unsigned char *tensor, const unsigned char *tensor_end, int V_, int row, int rank, int part) {
        base = tensor;
        end = tensor_end;
        V = V_;
        const size_t bytes = static_cast<size_t>(V) * EB;
        const unsigned char *p = base + static_cast<size_t>(row) * bytes;
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
        win = p - off;
        lead = off / EB;
        total = static_cast<int>((off + bytes + 15) >> 4);
        first = rank * part;
        n = max(0, min(part, total - first));
    }
    // The logit's index in its row of element q of vector i (of this CTA's).
    __device__ __forceinline__ int index(int i, int q) const { return (first + i) * kPer + q - lead; }
    // Where logit x of the row is, in elements from the CTA's first vector.
    __device__ __forceinline__ int offset(int x) const { return x + lead - first * kPer; }
    __device__ __forceinline__ const unsigned char *at(int i) const { return win + (static_cast<size_t>(first + i) << 4); }
    __device__ __forceinline__ bool edge(int i) const { return first + i == 0 || first + i == total - 1; }
    __device__ __forceinline__ bool inside(int i) const { return at(i) >= base && at(i) + 16 <= end; }

    // The vectors that can be read whole: all but one that lies across the tensor's first or last byte.
    __device__ __forceinline__ int copy_from() const { return n > 0 && !inside(0) ? 1 : 0; }
    __device__ __forceinline__ int copy_upto() const { return n > 0 && !inside(n - 1) ? n - 1 : n; }
    // This thread's vectors (i = tid, tid + step, ...) to shared memory, asynchronously.
    __device__ __forceinline__ void copy_all(uint4 *buf, int tid, int step) const {
        const int from = copy_from(), upto = copy_upto();
        const unsigned char *src = at(tid);
        uint32_t dst = smem_u32(buf + tid);
        for (int i = tid; i < upto; i += step, src += 16 * step, dst += 16 * step)
            if (i >= from) copy16(dst, src);
    }
    // After the copies: the row's first and last vector, which may hold a neighbour's logits or lie
    // across the tensor's end, by the threads that own them.
    __device__ __forceinline__ void mend_all(uint4 *buf, int tid, int step) const {
        if (n <= 0) return;
        if (tid == 0 && edge(0)) buf[0] = by_logit(at(0), index(0, 0), V);
        if (tid == (n - 1) % step && edge(n - 1)) buf[n - 1] = by_logit(at(n - 1), index(n - 1, 0), V);
    }
    // Vector `at`, whose first element is logit x0 of the row, element by element.
    static __device__ __noinline__ uint4 by_logit(const unsigned char *at, int x0, int V) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (EB == 4) {
                const int x = x0 + q;
                w[q] = x >= 0 && x < V ? *reinterpret_cast<const uint32_t *>(at + 4 * q) : 0xff800000u;
            } else {
                uint32_t h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int x = x0 + 2 * q + j;
                    h[j] = x >= 0 && x < V ? *reinterpret_cast<const uint16_t *>(at + 4 * q + 2 * j) : 0xff80u;
                }
                w[q] = h[0] | h[1] << 16;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 fetch(int i) const {
        return edge(i) ? by_logit(at(i), index(i, 0), V) : *reinterpret_cast<const uint4 *>(at(i));
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
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // The largest logit of a vector, NaN if it holds one.
    static __device__ __forceinline__ float vector_max(const uint4 &v) {
        if (EB == 2) {
            const uint32_t m = max2(max2(v.x, v.y), max2(v.z, v.w));
            return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
        }
        return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    // The largest logit of N vectors.
    template <int N>
    static __device__ __forceinline__ float vectors_max(const uint4 (&v)[N]) {
        if (EB == 2) {
            uint32_t m[N];
#pragma unroll
            for (int j = 0; j < N; ++j) m[j] = max2(max2(v[j].x, v[j].y), max2(v[j].z, v[j].w));
#pragma unroll
            for (int h = N / 2; h; h >>= 1)
#pragma unroll
                for (int j = 0; j < h; ++j) m[j] = max2(m[j], m[j + h]);
            return max_nan(__uint_as_float(m[0] << 16), __uint_as_float(m[0] & 0xffff0000u));
        }
        float m = vector_max(v[0]);
#pragma unroll
        for (int j = 1; j < N; ++j) m = max_nan(m, vector_max(v[j]));
        return m;
    }
    // A vector of -inf.
    static __device__ __forceinline__ uint4 nothing() {
        const uint32_t w = EB == 2 ? 0xff80ff80u : 0xff800000u;
        return make_uint4(w, w, w, w);
    }
    static __device__ __forceinline__ float logit(const void *p, int i) {
        return EB == 4 ? reinterpret_cast<const float *>(p)[i]
                       : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << 16);
    }
};

}  // namespace vocab
}  // namespace spec
