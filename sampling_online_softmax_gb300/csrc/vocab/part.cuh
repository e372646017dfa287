// part.cuh -- one CTA's share of a row: the row's 16-byte vectors, on the 16-byte
// grid of global memory, are dealt out to the CTAs in contiguous runs, so every
// vector belongs to one CTA and only the row's first and last can hold logits
// of a neighbouring row (read as -inf).  Bytes outside the tensor are never read.
#pragma once

#include "cluster.cuh"

namespace spec {
namespace vocab {

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

    __device__ __forceinline__ void copy(uint4 *buf, int i) const {
        if (inside(i)) copy16(smem_u32(buf + i), at(i));
    }
    // After the copy: an edge vector's logits outside the row become -inf.
    __device__ __forceinline__ void mend(uint4 *buf, int i) const {
        if (edge(i)) buf[i] = by_logit(at(i), index(i, 0), V);
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
    static __device__ __forceinline__ float logit(const void *p, int i) {
        return EB == 4 ? reinterpret_cast<const float *>(p)[i]
                       : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << 16);
    }
};

}  // namespace vocab
}  // namespace spec
