// attention.cuh -- attention of drafted tokens over the paged cache and their own tree, on the
// fifth-generation tensor cores.
//
// The rows of a block are (node, query head) pairs that share a key head, so a tile of keys is read
// once for all of them.  Scores S = Q K^T and weighted sums O += P V are tcgen05 products of 128 rows:
//   Q, K, V   shared memory, in swizzled rows of 128 bytes (K and V as TMA lays them)
//   S, O      tensor memory, a row a lane; P, the weights in the element type, over S's columns
// Two products are under way at once, each with a warpgroup of its own for the softmax: blocks of more
// than 128 rows have two halves, which share each tile; smaller ones take their tiles in turn, and the
// two sums are joined at the end.  While one warpgroup computes weights, the other's products run.
//
//   warps 0-3, 4-7   softmax of product 0, 1: a thread a row
//   four warps       values whose other rows must be 0 (what lies behind a sequence's end, nodes that are
//                    not finite: 0 * NaN is NaN); eight of them where 8-bit tiles are widened too
//   one warp each    TMA of tiles; tcgen05.mma; TMA of queries; TMA of 8-bit tiles
//
// The softmax keeps a row's running maximum as it was until a tile's exceeds it by 2^8: weights up to 2^8
// lose nothing in a float format, and O is rescaled almost never.
#pragma once

#include <type_traits>

#include "attention.h"
#include "cache.cuh"
#include "tensor.cuh"

namespace spec {
namespace context {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, bool Q8>
struct Layout {
    static constexpr int kQ = kTile * D * 2;     // bytes of 128 rows of queries, keys or values
    static constexpr int kRing = Q8 ? (D == 128 ? 4 : 6) : (D == 128 ? 5 : 8);
    static constexpr int kStage = Q8 ? kTile * D : 0;
    static constexpr int kStages = Q8 ? (D == 128 ? 2 : 8) : 0;
    static constexpr int kWorkers = Q8 ? 8 : 4;              // warps that clear and widen
    static constexpr int kThreads = (8 + kWorkers + 4) * 32;
    // Registers of a thread after the start: the sum over the warps is what the launch has (65536 at 512
    // threads, 640 * 96 at 640).
    static constexpr int kSoftmaxRegs = Q8 ? 152 : 192, kOtherRegs = Q8 ? 56 : 64;
    static constexpr int kBytes = 2 * kQ + kRing * kQ + kStages * kStage;
};

struct Control {  // behind the tiles in shared memory
    uint64_t full[8], empty[8];    // ring of tiles
    uint64_t copied[8];            // a slot's values are there, to be cleared in part
    uint64_t staged[8], free_[8];  // ring of 8-bit tiles
    uint64_t q_full[2], q_empty[2];
    uint64_t scores[2], weights[2], sums[2];  // of the two products
    uint64_t joined[2];            // both warpgroups: statistics there, sums read
    uint64_t drained;
    uint32_t tmem;
    int gave_up;
    int odd[8];                    // a value of the piece's nodes is not finite (by piece, in turn)
    int scan[20];
    int total, b, before;          // tiles in all; the sequence a CTA begins in and the tiles before it
    float2 stats[2][kTile];
};

// A CTA's pieces of the list, in order.
struct Piece {
    bool shared, two;    // of the prefix; two products a tile
    int b, g, first, rows;
    int t0, t1, tiles;   // the piece's tiles, of the block's
    int len, context;    // own: the sequence's length, its context's tiles
};

struct Walk {
    const AttentionArgs &a;
    int left, item, t, b, tiles, context, len, per_seq, shared_items, shared_tiles;
    bool shared;

    __device__ Walk(const AttentionArgs &a_, const Control *c) : a(a_) {
        const int lo = static_cast<int>(static_cast<long long>(blockIdx.x) * c->total / a.ctas);
        left = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * c->total / a.ctas) - lo;
        shared_tiles = tiles_of(a.shared_len);
        shared_items = shared_tiles ? a.cache.kv_heads * a.shared_blocks : 0;
        per_seq = a.cache.kv_heads * a.blocks;
        b = -1;
        shared = lo < shared_items * shared_tiles;
        if (shared) {
            item = lo / shared_tiles;
            t = lo % shared_tiles;
        } else if (left > 0) {
            sequence(c->b);
            item = (lo - c->before) / tiles;
            t = (lo - c->before) % tiles;
        }
    }
    __device__ void sequence(int to) {
        b = to;
        const int room = a.cache.table_width << a.cache.page_bits;
        len = __ldg(a.lens + b);
        if (len >= 0) len = min(max(len, a.shared_len), room);
        context = len > a.shared_len ? tiles_of(len) - a.shared_len / kTile : 0;
        tiles = len < 0 ? 0 : context + tiles_of(a.N);
        item = 0;
    }
    __device__ bool next(Piece *p) {
        if (left <= 0) return false;
        if (shared && item == shared_items) shared = false;
        if (!shared)
            while (b < 0 || tiles == 0 || item == per_seq) sequence(b + 1);
        const int blocks = shared ? a.shared_blocks : a.blocks, rows = shared ? a.shared_rows : a.block_rows;
        const int all = shared ? a.B * a.N * a.group : a.N * a.group;
        const int block = item % blocks;
        p->shared = shared;
        p->two = rows > a.half_nodes * a.group;
        p->b = shared ? 0 : b;
        p->g = item / blocks;
        p->first = block * rows;
        p->rows = min(rows, all - p->first);
        p->tiles = shared ? shared_tiles : tiles;
        p->t0 = t;
        p->t1 = min(p->tiles, t + left);
        p->len = shared ? a.shared_len : len;
        p->context = shared ? shared_tiles : context;
        left -= p->t1 - p->t0;
        t = p->t1;
        if (t == p->tiles) {
            t = 0;
            ++item;
        }
        return true;
    }
};

// A ring's next slot, and the parity of its round.
struct Cursor {
    int slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step(int n) {
        if (++slot == n) {
            slot = 0;
            round ^= 1;
        }
    }
};

// The row of the batch that row `r` (of all the rows of piece p's kind) is.
struct RowId {
    int b, n, h;
};
__device__ __forceinline__ RowId row_id(const AttentionArgs &a, const Piece &p, int r) {
    const int i = (p.first + r) / a.group, h = (p.first + r) % a.group;
    return RowId{p.shared ? i / a.N : p.b, p.shared ? i % a.N : i, p.g * a.group + h};
}

// Sixteen e4m3 values, times 2^(byte - 127), as 16 elements.
template <typename T>
struct Widen;
template <>
struct Widen<__nv_bfloat16> {
    uint32_t m1, m2;
    bool twice;
    // An e4m3 value's bits, moved into bf16's places, read as 2^-120 of it (subnormal ones too), so
    // it is a product with 2^(120 + e), in two steps where that is past bf16.
    __device__ __forceinline__ void scale(uint32_t byte) {
        const int e = static_cast<int>(byte) - 127, e1 = min(e + 120, 127);
        uint32_t s1 = static_cast<uint32_t>(max(e1 + 127, 1)) << 7;
        const uint32_t s2 = static_cast<uint32_t>(127 + e + 120 - e1) << 7;
        if (byte == 255) s1 = 0x7fff;
        m1 = s1 | s1 << 16;
        m2 = s2 | s2 << 16;
        twice = e > 7;
    }
    __device__ __forceinline__ void zero() { m1 = m2 = 0, twice = false; }
    static __device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    template <bool TWICE>
    __device__ __forceinline__ uint2 four(uint32_t w) const {
        const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
        uint32_t x = times((a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), m1), y = times((b & 0x80008000u) | ((b >> 4) & 0x07f007f0u), m1);
        if (TWICE) x = times(x, m2), y = times(y, m2);
        return make_uint2(x, y);
    }
};
template <>
struct Widen<__half> {
    static constexpr bool twice = false;
    uint32_t m;
    __device__ __forceinline__ void scale(uint32_t byte) {
        const int e = min(max(static_cast<int>(byte) - 127, -24), 15);
        uint32_t s = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : 1u << (e + 24);
        if (byte == 255) s = 0x7fff;
        m = s | s << 16;
    }
    __device__ __forceinline__ void zero() { m = 0; }
    static __device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    template <bool>
    __device__ __forceinline__ uint2 four(uint32_t w) const {
        const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffff), __NV_E4M3);
        const __half2_raw y = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
        return make_uint2(times(*reinterpret_cast<const uint32_t *>(&x), m), times(*reinterpret_cast<const uint32_t *>(&y), m));
    }
};

// Where a tile's 16-byte chunk c of row r lies: 64 columns (8 chunks) a sub-tile of 128 rows, swizzled.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * (kTile * 128) + r * 128 + ((c & 7) ^ (r & 7)) * 16);
}
__device__ __forceinline__ void store16(uint32_t at, const uint4 &x) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
__device__ __forceinline__ uint4 load16(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
    return x;
}

// Packed fp32 arithmetic.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)), "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&r);
}

// Where a piece leaves its rows' sums, column by column (a warp's rows lie next to each other), and (maximum, sum).
struct Part {
    float *sums;    // [D][rows]
    float2 *stats;  // [rows]
    int rows;
};
// A block that a CTA does not hold whole: at the CTA's begin (its block began in an earlier one) or its end.
template <int D>
__device__ __forceinline__ Part cut_part(const AttentionArgs &a, int cta, bool at_end) {
    const size_t i = static_cast<size_t>(cta) * 2 + (at_end ? 1 : 0);
    return Part{a.cut_sums + i * kBlockRows * D, a.cut_stats + i * kBlockRows, kBlockRows};
}
// A whole block, beside a prefix: of sequence b's rows, or of the batch's (`first`: its first row of them).
template <int D>
__device__ __forceinline__ Part whole_part(const AttentionArgs &a, bool shared, int b, int g, int first) {
    const size_t per_seq = static_cast<size_t>(a.N) * a.group, all = per_seq * a.B;
    const size_t row = shared ? (a.cache.kv_heads + g) * all + first : g * all + b * per_seq + first;
    const int rows = shared ? min(static_cast<int>(all) - first, a.shared_rows) : min(static_cast<int>(per_seq) - first, a.block_rows);
    return Part{a.row_sums + row * D, a.row_stats + row, rows};
}

// ------------------------------------------------------------------ the four kinds of warps
template <typename T, int D, bool Q8>
struct Attention {
    using L = Layout<D, Q8>;
    static constexpr bool kHalf = std::is_same<T, __half>::value;
    static constexpr uint32_t kType = kHalf ? 0 : 1;
    static constexpr uint32_t kScoresInstr = instruction(kType, kTile, false), kSumsInstr = instruction(kType, D, true);
    static constexpr uint32_t kScores = 0, kSums = 256;  // columns of tensor memory; 128 a product
    // fp16 weights: up to 2^15 instead of 2^8, since they stop at 2^-25
    static constexpr float kShift = kHalf ? 7.0f : 0.0f;

    const AttentionArgs &a;
    Control *c;
    uint32_t tiles, stages;  // shared-memory addresses: queries, then the ring; 8-bit tiles
    uint32_t tmem;
    int lane, warp;

    __device__ __forceinline__ bool wait(const uint64_t *bar, uint32_t parity) {
        return wait_phase(ptx::smem_addr(bar), parity, &c->gave_up, a.status);
    }
    __device__ __forceinline__ uint32_t ring(int slot) const { return tiles + 2 * L::kQ + slot * L::kQ; }
    // Whether a piece's tile t of the context ends behind the sequence, or begins before what is its own.
    __device__ __forceinline__ bool ragged(const Piece &p, int t) const {
        const int at = (first_tile(p) + t) * kTile;
        return at + kTile > p.len || at < begin(p);
    }
    __device__ __forceinline__ int first_tile(const Piece &p) const { return p.shared ? 0 : a.shared_len / kTile; }
    __device__ __forceinline__ int begin(const Piece &p) const { return p.shared ? 0 : a.shared_len; }  // the piece's first position

    // ---- TMA
    // The keys and values of one tile of the context, in boxes of at most a page: lane i the i-th.
    struct Boxes {
        int page, y;
    };
    __device__ __forceinline__ Boxes boxes_of(const Piece &p, int t, int box, bool &bad) const {
        const long long pos = static_cast<long long>(first_tile(p) + t) * kTile + lane * box;
        Boxes b{a.cache.pages, (p.g << a.cache.page_bits) + static_cast<int>(pos & ((1 << a.cache.page_bits) - 1))};  // outside: zeros
        if (lane < kTile / box && pos < p.len && pos + box > begin(p)) {
            const int entry = __ldg(a.cache.table + static_cast<size_t>(p.b) * a.cache.table_width + (pos >> a.cache.page_bits));
            if (entry < 0 || entry >= a.cache.pages) bad = true;
            else b.page = entry;
        }
        return b;
    }
    __device__ __forceinline__ int box_rows() const { return min(1 << a.cache.page_bits, kTile); }
    // No copy is in flight when the CTA ends: where a wait gave up, the last one into each of the n slots is waited for
    // (`rounds`: the parities of their barriers' phases).
    __device__ void drain(const uint64_t *bars, int n, uint32_t issued, uint32_t rounds) {
        for (int i = 0; i < n; ++i) {
            bool done = !(issued >> i & 1);
            for (int k = 0; !done && k < kWaitTries; ++k) done = ptx::mbar_try_wait(ptx::smem_addr(bars + i), rounds >> i & 1);
        }
    }
    // Tiles into the ring: of a 16-bit cache, and of the nodes.  Each round of each slot is waited for and
    // arrived at by this warp and by the workers, whichever fills it: a parity tells a round from its
    // neighbours alone, so none may run ahead of the ring by more than a round, or fall behind it.
    __device__ void load_tiles(const Maps &maps) {
        Walk walk(a, c);
        Piece p;
        Cursor at;
        // tiles that one block takes are read once; where several blocks take them, L2 may keep them
        const uint64_t once = ptx::policy_evict_first(), normal = policy_evict_normal();
        const int box = box_rows();
        bool bad = false, ok = true;
        uint32_t issued = 0, rounds = 0, copied = 0, copies = 0;  // a bit a slot: loaded; its last phase's parity; the same of `copied`
        while (ok && walk.next(&p)) {
            const uint64_t policy = (p.shared ? a.shared_blocks : a.blocks) == 1 ? once : normal;
            for (int t = p.t0; ok && t < p.t1; ++t) {
                Boxes boxes;
                if (!Q8 && t < p.context) boxes = boxes_of(p, t, box, bad);
                for (int w = 0; w < 2; ++w, at.step(L::kRing)) {
                    if (!(ok = wait(&c->empty[at.slot], at.round ^ 1))) break;
                    const uint32_t full = ptx::smem_addr(&c->full[at.slot]), to = ring(at.slot), bit = 1u << at.slot;
                    if (Q8 && t < p.context) {
                        if (lane == 0) arrive(full);
                        __syncwarp();
                        continue;
                    }
                    // Values that the workers look through first: their copy is waited for there.
                    const bool checked = w && (t >= p.context || ragged(p, t));
                    const uint32_t bar = checked ? ptx::smem_addr(&c->copied[at.slot]) : full;
                    if (lane == 0) {
                        if (checked) arrive(full);
                        ptx::mbar_arrive_expect_tx(bar, L::kQ);
                    }
                    __syncwarp();
                    if (t >= p.context) {
                        if (lane < D / 64) tma_load4(to + lane * (kTile * 128), w ? &maps.v_nodes : &maps.k_nodes, lane * 64, p.g, (t - p.context) * kTile, p.b, bar, normal);
                    } else if (lane < kTile / box) {
                        for (int x = 0; x < D; x += 64) tma_load3(to + (x / 64) * (kTile * 128) + lane * box * 128, w ? &maps.v : &maps.k, x, boxes.y, boxes.page, bar, policy);
                    }
                    if (checked) copied |= bit, copies ^= bit;
                    else issued |= bit, rounds = (rounds & ~bit) | at.round << at.slot;
                }
            }
        }
        if (bad) atomicOr(a.status, SPEC_DEV_BAD_PAGE);
        if (!ok) {
            drain(c->full, L::kRing, issued, rounds);
            drain(c->copied, L::kRing, copied, ~copies);
        }
    }
    // 8-bit tiles, to be widened.
    __device__ void load_stages(const Maps &maps) {
        Walk walk(a, c);
        Piece p;
        Cursor at;
        const uint64_t once = ptx::policy_evict_first(), normal = policy_evict_normal();
        const int box = box_rows();
        bool bad = false, ok = true;
        uint32_t issued = 0, rounds = 0;
        while (ok && walk.next(&p)) {
            const uint64_t policy = (p.shared ? a.shared_blocks : a.blocks) == 1 ? once : normal;
            for (int t = p.t0; ok && t < min(p.t1, p.context); ++t) {
                const Boxes boxes = boxes_of(p, t, box, bad);
                for (int w = 0; w < 2; ++w) {
                    if (!(ok = wait(&c->free_[at.slot], at.round ^ 1))) break;
                    const uint32_t bar = ptx::smem_addr(&c->staged[at.slot]);
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, L::kStage);
                    __syncwarp();
                    if (lane < kTile / box) tma_load3(stages + at.slot * L::kStage + lane * box * D, w ? &maps.v : &maps.k, 0, boxes.y, boxes.page, bar, policy);
                    issued |= 1u << at.slot;
                    rounds = (rounds & ~(1u << at.slot)) | at.round << at.slot;
                    at.step(L::kStages > 0 ? L::kStages : 1);
                }
            }
        }
        if (bad) atomicOr(a.status, SPEC_DEV_BAD_PAGE);
        if (!ok) drain(c->staged, L::kStages, issued, rounds);
    }
    // Queries: a half holds a.half_nodes nodes, whose heads of the group lie next to each other.
    __device__ void load_queries(const Maps &maps) {
        Walk walk(a, c);
        Piece p;
        const uint64_t normal = policy_evict_normal();
        uint32_t round = 0, issued = 0;  // a bit a half
        int half = 0, count = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            if (p.two) half = 0;
            for (int h = 0; ok && h < 2; ++h) {
                if (!p.two && h != half) continue;
                if (!(ok = wait(&c->q_empty[h], (round >> h & 1) ^ 1))) break;
                round ^= 1u << h;
                issued |= 1u << h;
                // (the piece four on: none is read that far back, nor loaded that far ahead)
                if (lane == 0) *const_cast<volatile int *>(&c->odd[(count + 4) & 7]) = 0;
                const uint32_t bar = ptx::smem_addr(&c->q_full[h]);
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar, a.q_nodes * a.group * D * 2);
                __syncwarp();
                const int node = p.first / a.group + (p.two ? h * a.half_nodes : 0);
                const int z = a.q_merged && !p.shared ? p.b * a.N + node : node, b = a.q_merged ? 0 : p.b;
                if (lane < D / 64) tma_load4(tiles + h * L::kQ + lane * (kTile * 128), &maps.q, lane * 64, p.g * a.group, z, b, bar, normal);
            }
            ++count;
            if (!p.two) half ^= 1;
        }
        if (!ok) drain(c->q_full, 2, issued, ~round);
    }

    // ---- tcgen05.mma
    struct Pending {
        bool any, add, release, final;
        int slot;
        uint32_t round;
    };
    // The same in every lane, said so that the compiler keeps it in a uniform register, as the mma wants it.
    static __device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
    __device__ bool add_values(Pending &w, int s, uint32_t &weights_round) {
        w.any = false;
        if (!wait(&c->full[w.slot], w.round) || !wait(&c->weights[s], weights_round)) return false;
        weights_round ^= 1;
        fence_after();
        const uint32_t v = uniform(operand(ring(w.slot), kTile * 128)), d = uniform(tmem + kSums + s * 128), p = uniform(tmem + kScores + s * 128);
        if (elect()) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) mma_tmem(d, p + k * 8, descriptor(v + k * 16 * 128 / 16), kSumsInstr, w.add || k > 0);
            if (w.release) mma_commit(ptx::smem_addr(&c->empty[w.slot]));
            if (w.final) mma_commit(ptx::smem_addr(&c->sums[s]));
        }
        __syncwarp();
        return true;
    }
    __device__ void multiply() {
        Walk walk(a, c);
        Piece p;
        Cursor at;
        Pending pending[2] = {};
        uint32_t weights_round[2] = {0, 0}, q_round[2] = {0, 0};
        int half = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            const int n = p.t1 - p.t0;
            if (p.two) half = 0;
            for (int h = 0; ok && h < 2; ++h)
                if (p.two || h == half) {
                    ok = wait(&c->q_full[h], q_round[h]);
                    q_round[h] ^= 1;
                }
            for (int i = 0; ok && i < n; ++i) {
                const Cursor keys = at;
                at.step(L::kRing);
                const Cursor values = at;
                at.step(L::kRing);
                for (int x = 0; ok && x < (p.two ? 2 : 1); ++x) {
                    const int s = p.two ? x : i & 1;
                    if (pending[s].any && !(ok = add_values(pending[s], s, weights_round[s]))) break;
                    if (x == 0 && !(ok = wait(&c->full[keys.slot], keys.round))) break;
                    fence_after();
                    const uint32_t q = uniform(operand(tiles + (p.two ? x : half) * L::kQ, 16)), k = uniform(operand(ring(keys.slot), 16));
                    const uint32_t d = uniform(tmem + kScores + s * 128);
                    if (elect()) {
#pragma unroll
                        for (int e = 0; e < D / 16; ++e) {
                            const uint32_t off = ((e / 4) * (kTile * 128) + (e % 4) * 32) / 16;
                            mma(d, descriptor(q + off), descriptor(k + off), kScoresInstr, e > 0);
                        }
                        mma_commit(ptx::smem_addr(&c->scores[s]));
                        if (x == (p.two ? 1 : 0)) mma_commit(ptx::smem_addr(&c->empty[keys.slot]));
                        if (i == n - 1) {
                            if (p.two) mma_commit(ptx::smem_addr(&c->q_empty[x]));
                            else mma_commit(ptx::smem_addr(&c->q_empty[half]));
                        }
                    }
                    __syncwarp();
                    pending[s] = Pending{true, p.two ? i > 0 : i > 1, !p.two || x == 1, p.two ? i == n - 1 : i >= n - 2, values.slot, values.round};
                }
            }
            // the piece's last weights: the earlier product's first
            for (int x = 0; ok && x < 2; ++x) {
                const int s = p.two ? x : (n + x) & 1;
                if (pending[s].any) ok = add_values(pending[s], s, weights_round[s]);
            }
            if (!p.two) half ^= 1;
        }
        // Every product done before tensor memory is freed, also where a wait gave up.
        if (elect()) mma_commit(ptx::smem_addr(&c->drained));
        __syncwarp();
        bool done = false;
        for (int n = 0; !done && n < kWaitTries; ++n) done = ptx::mbar_try_wait(ptx::smem_addr(&c->drained), 0);
    }

    // ---- workers: a thread a row, or two threads where there are eight warps
    static constexpr int kLanes = D / 8, kSplit = L::kWorkers / 4, kShare = kLanes / kSplit;  // 16-byte chunks of a row; of a thread
    __device__ __forceinline__ static bool odd_pair(uint32_t x) {  // an infinity or NaN among two elements
        constexpr uint32_t e = kHalf ? 0x7c00u : 0x7f80u;
        return (x & e) == e || (x >> 16 & e) == e;
    }
    // The rows of a tile of values outside [from, to) become 0.
    __device__ __forceinline__ void clear_rows(uint32_t at, int tid, int from, int to) const {
        const int r = tid & 127;
        if (r >= from && r < to) return;
#pragma unroll 4
        for (int x = 0; x < kShare; ++x) store16(at + chunk_at(r, (tid >> 7) * kShare + x), make_uint4(0, 0, 0, 0));
    }
    // Values of nodes that are not finite become 0 (true: there were some): a row that does not see them would
    // get 0 * NaN.  The rows that do are given them at the end.
    __device__ __forceinline__ bool take_odd(uint32_t at, int tid) const {
        bool odd = false;
#pragma unroll 4
        for (int i = 0; i < kShare; ++i) {
            const uint32_t to = at + chunk_at(tid & 127, (tid >> 7) * kShare + i);
            uint4 v = load16(to);
            if (odd_pair(v.x) || odd_pair(v.y) || odd_pair(v.z) || odd_pair(v.w)) {
                constexpr uint32_t e = kHalf ? 0x7c00u : 0x7f80u;
                uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if ((w[k] & e) == e) w[k] &= 0xffff0000u;
                    if ((w[k] >> 16 & e) == e) w[k] &= 0xffffu;
                }
                store16(to, v);
                odd = true;
            }
        }
        return odd;
    }
    // The page of this thread's row of a piece's tile t, -1 where there is none; the scales of its keys and values.
    __device__ __forceinline__ int row_page(const Piece &p, int t, int r) const {
        const int pos = (first_tile(p) + t) * kTile + r;
        if (t >= min(p.t1, p.context) || pos >= p.len || pos < begin(p)) return -1;
        const int page = __ldg(a.cache.table + static_cast<size_t>(p.b) * a.cache.table_width + (pos >> a.cache.page_bits));
        return page < a.cache.pages ? page : -1;
    }
    __device__ __forceinline__ int row_scales(const Piece &p, int t, int r, int page) const {  // keys', values' << 8; -1: no row
        if (page < 0) return -1;
        const int pos = (first_tile(p) + t) * kTile + r;
        const size_t row = cache_row(a.cache, (static_cast<long long>(page) << a.cache.page_bits) + (pos & ((1 << a.cache.page_bits) - 1)), p.g);
        return __ldg(a.cache.scale[0] + row) | __ldg(a.cache.scale[1] + row) << 8;
    }
    // An 8-bit tile, widened: half a row a thread; the chunks in turned order, so that eight rows' meet different banks.
    template <bool TWICE>
    __device__ __forceinline__ void widen(uint32_t from, uint32_t to, int tid, const Widen<T> &w) const {
        constexpr int kChunks = D / 32;
        const int r = tid & 127;
        uint4 v[kChunks];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) v[j] = load16(from + r * D + turned(j, tid) * 16);
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            const int x = turned(j, tid);
            const uint2 b0 = w.template four<TWICE>(v[j].x), b1 = w.template four<TWICE>(v[j].y);
            store16(to + chunk_at(r, 2 * x), make_uint4(b0.x, b0.y, b1.x, b1.y));
            const uint2 b2 = w.template four<TWICE>(v[j].z), b3 = w.template four<TWICE>(v[j].w);
            store16(to + chunk_at(r, 2 * x + 1), make_uint4(b2.x, b2.y, b3.x, b3.y));
        }
    }
    // The j-th chunk of thread tid's half row: of 16 bytes, eight rows' in one step lie in eight places modulo 128 bytes.
    static __device__ __forceinline__ int turned(int j, int tid) {
        const int k = j + (tid >> 7) * (D / 32);
        return D == 128 ? (k + tid) & 7 : (k + (tid >> 1)) & 3;
    }
    __device__ void work(int tid) {
        Walk walk(a, c);
        Piece p;
        Cursor at, staged;
        uint32_t copies = 0;  // the parity of each slot's next copy to look through
        int count = 0;
        bool ok = true;
        const int r = tid & 127;
        while (ok && walk.next(&p)) {
            int scales = -1, next_page = -1;  // of the tile at hand; of the one after it
            if (Q8) {
                scales = row_scales(p, p.t0, r, row_page(p, p.t0, r));
                next_page = row_page(p, p.t0 + 1, r);
            }
            for (int t = p.t0; ok && t < p.t1; ++t) {
                int next_scales = -1;
                if (Q8) {  // two dependent loads, each issued a tile ahead of its use
                    next_scales = row_scales(p, t + 1, r, next_page);
                    next_page = row_page(p, t + 2, r);
                }
                for (int w = 0; ok && w < 2; ++w, at.step(L::kRing)) {
                    const uint32_t to = ring(at.slot);
                    if (!(ok = wait(&c->empty[at.slot], at.round ^ 1))) break;
                    if (Q8 && t < p.context) {
                        if (!(ok = wait(&c->staged[staged.slot], staged.round))) break;
                        Widen<T> x;
                        if (scales >= 0) x.scale(scales >> (8 * w) & 255);
                        else x.zero();
                        const uint32_t from = stages + staged.slot * L::kStage;
                        if (__any_sync(0xffffffffu, x.twice)) widen<true>(from, to, tid, x);
                        else widen<false>(from, to, tid, x);
                        __syncwarp();
                        if (lane == 0) arrive(ptx::smem_addr(&c->free_[staged.slot]));
                        staged.step(L::kStages > 0 ? L::kStages : 1);
                        fence_async();
                    } else if (w && (t >= p.context || ragged(p, t))) {
                        if (!(ok = wait(&c->copied[at.slot], copies >> at.slot & 1))) break;
                        copies ^= 1u << at.slot;
                        if (t < p.context) {
                            const int base = (first_tile(p) + t) * kTile;
                            clear_rows(to, tid, begin(p) - base, p.len - base);
                        } else if (take_odd(to, tid)) {
                            *const_cast<volatile int *>(&c->odd[count & 7]) = 1;
                        }
                        fence_async();
                    }
                    __syncwarp();
                    if (lane == 0) arrive(ptx::smem_addr(&c->full[at.slot]));
                }
                scales = next_scales;
            }
            ++count;
        }
    }

    // ---- softmax
    // Which of a tile's columns 32 k .. 32 k + 31 a row of node n sees: a bit a column.
    __device__ __forceinline__ uint32_t seen(const Piece &p, int t, int n, int k) const {
        if (t < p.context) {
            const int at = (first_tile(p) + t) * kTile + 32 * k;
            const int from = min(max(begin(p) - at, 0), 32), to = min(max(p.len - at, 0), 32);
            return static_cast<uint32_t>((1ull << to) - 1) & ~static_cast<uint32_t>((1ull << from) - 1);
        }
        const int m = (t - p.context) * kTile + 32 * k;
        if (m >= a.N) return 0;
        uint32_t w = a.N - m < 32 ? (1u << (a.N - m)) - 1 : ~0u;
        if (a.mask) w &= __ldg(a.mask + static_cast<size_t>(n) * ((a.N + 31) / 32) + m / 32);
        else w &= static_cast<uint32_t>((1ull << min(max(n - m + 1, 0), 32)) - 1);
        return w;
    }
    template <bool MASKED>
    static __device__ __forceinline__ float largest(const uint32_t (&x)[32], uint32_t w) {
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], MASKED && !((w >> j) & 1) ? -INFINITY : __uint_as_float(x[j]));
        return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    }
    // Weights of 32 columns into tensor memory; their sum is added to `sum`.
    template <bool MASKED>
    static __device__ __forceinline__ void weigh(const uint32_t (&x)[32], uint32_t w, float2 scale, float2 sub, float2 (&sum)[2], uint32_t to) {
        uint32_t y[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float2 e = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), scale, sub);
            e.x = ptx::ex2(e.x);
            e.y = ptx::ex2(e.y);
            if (MASKED) {
                if (!((w >> j) & 1)) e.x = 0.0f;
                if (!((w >> (j + 1)) & 1)) e.y = 0.0f;
            }
            sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], e);
            y[j / 2] = Elt<T>::from_float2(e.x, e.y);
        }
        tmem_store16(to, y);
    }
    // A tile's scores into weights, in two passes over tensor memory (the row's maximum, then the weights), 32 columns
    // at a time, the next ones under way.  The loops stay loops: every unrolled copy is fetched cold in each launch.
    template <bool MASKED>
    __device__ __forceinline__ void tile_weights(const Piece &p, int t, int n, uint32_t s_at, uint32_t o_at, float scale, bool first, float &m, float &l) {
        uint32_t x[32], y[32];
        float top = -INFINITY;
        __syncwarp();  // tensor memory's loads and stores take the warp as one: here and below, behind what parts it
        tmem_load32(x, s_at);
#pragma unroll 1
        for (int k = 0; k < 4; k += 2) {
            const uint32_t w0 = MASKED ? seen(p, t, n, k) : 0, w1 = MASKED ? seen(p, t, n, k + 1) : 0;
            if (MASKED) __syncwarp();
            wait_loads(x);
            tmem_load32(y, s_at + 32 * k + 32);
            top = fmaxf(top, largest<MASKED>(x, w0));
            wait_loads(y);
            tmem_load32(x, s_at + ((32 * k + 64) & 127));  // (the last: the first columns again, for the second pass)
            top = fmaxf(top, largest<MASKED>(y, w1));
        }
        top = top * scale;
        // `m` is what the exponents subtract; -inf while the row has seen nothing
        const float want = top - kShift;
        const bool moves = m == -INFINITY ? want > -INFINITY : want > m + 8.0f;
        if (__any_sync(0xffffffffu, moves)) {
            const float f = moves ? (m == -INFINITY ? 0.0f : ptx::ex2(m - want)) : 1.0f;
            l *= f;
            if (moves) m = want;
            __syncwarp();
            if (!first) {
                wait_loads(x);
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    tmem_load32(y, o_at + k);
                    wait_loads(y);
#pragma unroll
                    for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                    tmem_store32(o_at + k, y);
                }
            }
        }
        const float sub = m == -INFINITY ? 0.0f : -m;
        const float2 c2 = make_float2(scale, scale), s2 = make_float2(sub, sub);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        __syncwarp();
#pragma unroll 1
        for (int k = 0; k < 4; k += 2) {
            const uint32_t w0 = MASKED ? seen(p, t, n, k) : 0, w1 = MASKED ? seen(p, t, n, k + 1) : 0;
            if (MASKED) __syncwarp();
            wait_loads(x);
            tmem_load32(y, s_at + 32 * k + 32);
            weigh<MASKED>(x, w0, c2, s2, sum, s_at + 16 * k);
            wait_loads(y);
            if (k == 0) tmem_load32(x, s_at + 64);
            weigh<MASKED>(y, w1, c2, s2, sum, s_at + 16 * k + 16);
        }
        const float2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
        wait_stores();
    }
    // Rows of a piece that see a value of a node which is not finite get it: 32 columns from column d0.
    __device__ void add_odd(const Piece &p, const RowId &id, int d0, uint32_t (&x)[32]) const {
        for (int t = max(p.t0, p.context); t < p.t1; ++t) {
            for (int k = 0; k < 4; ++k)
                for (uint32_t w = seen(p, t, id.n, k); w; w &= w - 1) {
                    const int node = (t - p.context) * kTile + 32 * k + __ffs(w) - 1;
                    const T *v = reinterpret_cast<const T *>(a.v) + p.b * a.stride[4] + node * a.stride[5] + p.g * D + d0;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float y = static_cast<float>(v[j]);
                        if (!isfinite(y)) x[j] = __float_as_uint(__uint_as_float(x[j]) + y);
                    }
                }
        }
    }
    // Columns [d0, d1) of the block's row r: f0 * product 0's sums + f1 * product 1's, to where the piece's go.
    __device__ void write_sums(const Piece &p, int r, int d0, int d1, bool use0, bool use1, float f0, float f1, float m, float l, bool odd) {
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21) + kSums;
        const bool live = r < p.rows;
        const RowId id = row_id(a, p, live ? r : 0);
        const size_t row = (static_cast<size_t>(id.b) * a.N + id.n) * a.heads + id.h;
        const bool whole = p.t0 == 0 && p.t1 == p.tiles;
        const bool final = whole && a.shared_len == 0;
        const Part to = whole ? whole_part<D>(a, p.shared, p.b, p.g, p.first) : cut_part<D>(a, blockIdx.x, p.t0 == 0);
        if (live && d0 == 0) {
            if (!final) to.stats[r] = make_float2(m, l);
            else if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
        }
        const float inv = final ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
#pragma unroll 1
        for (int d = d0; d < d1; d += 32) {
            uint32_t x[32];
            __syncwarp();
            if (use0) {
                tmem_load32(x, lanes + d);
                wait_loads(x);
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f0);
            }
            if (use1) {
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                    uint32_t y[16];
                    tmem_load16(y, lanes + 128 + d + h);
                    wait_loads(y);
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[h + j] = __float_as_uint(use0 ? fmaf(__uint_as_float(y[j]), f1, __uint_as_float(x[h + j])) : __uint_as_float(y[j]) * f1);
                }
            }
            if (live && odd) add_odd(p, id, d, x);
            if (live && final) {
                uint4 *out = reinterpret_cast<uint4 *>(a.out + (row * D + d) * 2);
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(x[j + e]) * inv;
                    out[j / 8] = pack8<T>(v);
                }
            } else if (live) {
#pragma unroll
                for (int j = 0; j < 32; ++j) to.sums[static_cast<size_t>(d + j) * to.rows + r] = __uint_as_float(x[j]);
            }
        }
    }
    __device__ void softmax(int s, int tid) {
        Walk walk(a, c);
        Piece p;
        uint32_t scores_round = 0, sums_round = 0, joined_round = 0;
        int count = 0;
        bool ok = true;
        const float scale = a.scale * kLog2e;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, at bit 16
        while (ok && walk.next(&p)) {
            const uint32_t s_at = tmem + lanes + kScores + s * 128, o_at = tmem + lanes + kSums + s * 128;
            const int own = tid < a.half_nodes * a.group ? tid : kBlockRows, r = own + (p.two ? s * a.half_nodes * a.group : 0);  // this thread's row of the block
            const bool idle = __all_sync(0xffffffffu, r >= p.rows);  // the warp has none
            const int n = row_id(a, p, min(r, p.rows - 1)).n;
            float m = -INFINITY, l = 0.0f;
            bool first = true;
            for (int t = p.t0 + (p.two ? 0 : s); t < p.t1; t += p.two ? 1 : 2) {
                if (!(ok = wait(&c->scores[s], scores_round))) break;
                scores_round ^= 1;
                fence_after();
                if (!idle) {
                    const bool masked = t >= p.context || ragged(p, t);
                    if (masked) tile_weights<true>(p, t, n, s_at, o_at, scale, first, m, l);
                    else tile_weights<false>(p, t, n, s_at, o_at, scale, first, m, l);
                }
                first = false;
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(ptx::smem_addr(&c->weights[s]));
            }
            if (!ok) break;
            const int any = p.two ? 2 : min(2, p.t1 - p.t0);  // products with sums
            if (p.two || s < any) {
                if (!(ok = wait(&c->sums[s], sums_round))) break;
                sums_round ^= 1;
                fence_after();
            }
            const bool odd = *const_cast<volatile int *>(&c->odd[count & 7]) != 0 && !p.shared && p.t1 > p.context;
            if (p.two) {
                if (!idle) write_sums(p, r, 0, D, s == 0, s == 1, 1.0f, 1.0f, m, l, odd);
                fence_before();
            } else {
                // Both products' sums: each warpgroup writes half the columns.
                c->stats[s][tid] = make_float2(m, l);
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(ptx::smem_addr(&c->joined[0]));
                if (!(ok = wait(&c->joined[0], joined_round))) break;
                fence_after();
                const float2 x = c->stats[0][tid], y = any == 2 ? c->stats[1][tid] : make_float2(-INFINITY, 0.0f);
                const float top = fmaxf(x.x, y.x);
                const float f0 = x.x == -INFINITY ? 0.0f : ptx::ex2(x.x - top), f1 = y.x == -INFINITY ? 0.0f : ptx::ex2(y.x - top);
                if (!idle) write_sums(p, r, s * (D / 2), (s + 1) * (D / 2), true, any == 2, f0, f1, top, x.y * f0 + y.y * f1, odd);
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(ptx::smem_addr(&c->joined[1]));
                if (!(ok = wait(&c->joined[1], joined_round))) break;
                joined_round ^= 1;
                fence_after();
            }
            ++count;
        }
    }
};

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(Layout<D, Q8>::kThreads, 1) attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Maps maps) {
    using L = Layout<D, Q8>;
    constexpr int kThreads = L::kThreads;
    extern __shared__ __align__(1024) unsigned char smem[];
    Control *c = reinterpret_cast<Control *>(smem + L::kBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // Every CTA counts the tiles before each sequence: a thread some sequences, then a scan over threads.
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    const int room = a.cache.table_width << a.cache.page_bits, nodes = tiles_of(a.N), per_seq = a.cache.kv_heads * a.blocks;
    const int shared_tiles = tiles_of(a.shared_len) * a.cache.kv_heads * a.shared_blocks;
    int mine = 0;
    bool bad = false;
    const auto tiles = [&](int b) {
        int len = __ldg(a.lens + b);
        if (len < 0) return 0;
        bad |= len < a.shared_len || len > room;
        len = min(max(len, a.shared_len), room);
        return ((len > a.shared_len ? tiles_of(len) - a.shared_len / kTile : 0) + nodes) * per_seq;
    };
    for (int b = b0; b < b1; ++b) mine += tiles(b);
    if (bad && blockIdx.x == 0) atomicOr(a.status, SPEC_DEV_BAD_LENGTH);
    int sum = mine;
    for (int x = 1; x < 32; x *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, sum, x);
        if (lane >= x) sum += y;
    }
    if (lane == 31) c->scan[warp] = sum;
    if (tid == 0) {
        c->gave_up = 0;
        for (int i = 0; i < 8; ++i) c->odd[i] = 0;
        for (int i = 0; i < 8; ++i) {
            ptx::mbar_init(ptx::smem_addr(&c->full[i]), L::kWorkers + 1);
            ptx::mbar_init(ptx::smem_addr(&c->empty[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->copied[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->staged[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->free_[i]), L::kWorkers);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&c->q_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->q_empty[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->scores[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->weights[i]), 4);
            ptx::mbar_init(ptx::smem_addr(&c->sums[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->joined[i]), 8);
        }
        ptx::mbar_init(ptx::smem_addr(&c->drained), 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    int before = shared_tiles + sum - mine;
    for (int i = 0; i < warp; ++i) before += c->scan[i];
    if (tid == kThreads - 1) c->total = before + mine;
    __syncthreads();
    const int total = c->total;
    const int lo = static_cast<int>(static_cast<long long>(blockIdx.x) * total / a.ctas);
    const int hi = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * total / a.ctas);
    for (int b = b0; b < b1; ++b) {
        if (blockIdx.x == 0) a.starts[b] = before;
        const int n = tiles(b);
        if (lo >= before && lo < before + n) c->b = b, c->before = before;
        before += n;
    }
    if (blockIdx.x == 0 && tid == kThreads - 1) a.starts[a.B] = total;
    if (lo >= hi) return;  // the whole CTA
    constexpr int kFirst = 8 + L::kWorkers;  // of the four single warps
    if (warp == kFirst + 1) tmem_alloc(ptx::smem_addr(&c->tmem), 512);
    __syncthreads();
    fence_after();

    Attention<T, D, Q8> x{a, c, ptx::smem_addr(smem), ptx::smem_addr(smem) + 2 * L::kQ + L::kRing * L::kQ, c->tmem, lane, warp};
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftmaxRegs));
        x.softmax(warp >> 2, tid & 127);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kOtherRegs));
        if (warp < kFirst) x.work(tid - 256);
        else if (warp == kFirst) x.load_tiles(maps);
        else if (warp == kFirst + 1) x.multiply();
        else if (warp == kFirst + 2) x.load_queries(maps);
        else if (Q8) x.load_stages(maps);
    }

    fence_before();
    __syncthreads();
    if (warp == kFirst + 1) tmem_free(c->tmem, 512);
}

// ------------------------------------------------------------------ joining
// 32 rows of a block, a lane each, D / 8 columns a warp: the partial sums of the pieces that hold them, in the order
// of their keys, and the result through shared memory, so that it is written in whole lines.
template <typename T, int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ AttentionArgs a) {
    constexpr int E = D / 8;
    __shared__ uint32_t result[32][D / 2 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = (a.block_rows + 31) / 32;
    const int first = blockIdx.x % chunks * 32, item = blockIdx.x / chunks;
    const int block = item % a.blocks, g = item / a.blocks % a.cache.kv_heads, b = item / a.blocks / a.cache.kv_heads;
    const int total = a.starts[a.B], start = a.starts[b], tiles = (a.starts[b + 1] - start) / (a.cache.kv_heads * a.blocks);
    if (tiles == 0) return;  // left out
    const auto owner = [&](int t) { return static_cast<int>(((t + 1ll) * a.ctas - 1) / total); };
    const int own0 = start + (g * a.blocks + block) * tiles, c0 = owner(own0), c1 = owner(own0 + tiles - 1);
    if (c0 == c1 && !a.shared_len) return;  // written already
    const int rows = min(a.block_rows, a.N * a.group - block * a.block_rows);  // of the block
    const int r = min(first + lane, rows - 1), in_seq = block * a.block_rows + r;
    const bool live = first + lane < rows;

    float m = -INFINITY, l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    const auto take = [&](const Part &p, int at) {
        const float2 s = p.stats[at];
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = p.sums[static_cast<size_t>(warp * E + e) * p.rows + at];
        const float top = fmaxf(m, s.x), was = m == -INFINITY ? 0.0f : ptx::ex2(m - top), now = s.x == -INFINITY ? 0.0f : ptx::ex2(s.x - top);
        l = l * was + s.y * now;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * was + x[e] * now;
        m = top;
    };
    const auto pieces = [&](int t0, int from, int to, int at) {  // of a block whose tiles begin at t0
        for (int c = from; c <= to; ++c) {
            const int lo = static_cast<int>(static_cast<long long>(c) * total / a.ctas);
            if (lo == static_cast<int>((c + 1ll) * total / a.ctas)) continue;  // a CTA without tiles
            take(cut_part<D>(a, c, t0 >= lo), at);
        }
    };
    if (a.shared_len) {  // the prefix comes first; the rows of a block may lie in two of its blocks
        const int all = b * a.N * a.group + in_seq, at = all % a.shared_rows, part = all / a.shared_rows, n = tiles_of(a.shared_len);
        const int t0 = (g * a.shared_blocks + part) * n, s0 = owner(t0), s1 = owner(t0 + n - 1);
        if (s0 == s1) take(whole_part<D>(a, true, 0, g, part * a.shared_rows), at);
        else pieces(t0, s0, s1, at);
    }
    if (c0 == c1) take(whole_part<D>(a, false, b, g, block * a.block_rows), r);
    else pieces(own0, c0, c1, r);

    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < E; e += 2) result[lane][(warp * E + e) / 2] = Elt<T>::from_float2(o[e] * inv, o[e + 1] * inv);
    const size_t row = (static_cast<size_t>(b) * a.N + in_seq / a.group) * a.heads + g * a.group + in_seq % a.group;
    if (a.lse && warp == 0 && live) a.lse[row] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * (D / 2); i += 256) {
        const int k = i / (D / 2), x = i % (D / 2), s = block * a.block_rows + first + k;
        if (first + k >= rows) break;
        const size_t to = (static_cast<size_t>(b) * a.N + s / a.group) * a.heads + g * a.group + s % a.group;
        reinterpret_cast<uint32_t *>(a.out)[to * (D / 2) + x] = result[k][x];
    }
}

}  // namespace context
}  // namespace spec
