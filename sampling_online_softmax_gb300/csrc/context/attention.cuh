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
//                    not finite: 0 * NaN is NaN); 8-bit tiles, widened: four for keys, four for values
//   a lane each      tcgen05.mma of product 0, of product 1
//   one or two warps the list of work, TMA of queries and of tiles; with 8-bit tiles one more for their TMA
//
// The softmax keeps a row's running maximum as it was until a tile's exceeds it by 2^8: weights up to 2^8
// lose nothing in a float format, and O is rescaled almost never.
//
// What bounds it, by rows a block and the cache's type (128-wide heads, one CTA an SM):
//   long contexts, few rows   HBM: 3 contexts of up to 131072, 9 nodes x 4 heads: 190 us, 6.6 TB/s, 97 % of a copy
//   two full halves           the chain scores -> weights -> sums of two products, about 3 us a tile, of which its four products are
//                             1.35 us and the exponentials of both halves 0.5 (32 a clock and SM, measured); a row's weights
//                             come from eight loads of tensor memory, each waited for before what is computed from it: 48 sequences
//                             of 9 nodes behind 16384 shared tokens 158 us (0.75 PFLOP/s; over an 8-bit cache 194), 64 nodes of 16
//                             sequences over 4096 74 us, 15 of them the second kernel's (8 bits: 82)
//   8-bit tiles               widening, 1.6 thousand clocks a tile of two times four warps, and shared memory, which it and the
//                             products share: 64 sequences of 5 nodes over 8192 234 us, 3.1 TB/s (16 bits: 222 us, 6.5 TB/s)
//   small calls               launches and the chain from the list to the first sums: one token over 700 16 us
// With four warps for keys and values of 8 bits, in turn, the last took 280 us; with two halves of rows the eight are slower (64
// query heads, 32 nodes: 436 us against 421), since the softmax has fewer registers and shares more.  All 8-bit calls take eight: a form
// with four for two halves alone would be four more kernels, for those 3 %.
// The softmaxes in turn, and the second kernel launched early, were each measured slower.
#pragma once

#include <algorithm>
#include <type_traits>

#include "attention.h"
#include "cache.cuh"
#include "tensor.cuh"

namespace spec {
namespace context {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, bool Q8>
struct Layout {
    static constexpr int kTileBytes = kTile * D * 2;         // of 128 rows of keys or values
    static constexpr int kStageBytes = Q8 ? kTile * D : 0;   // of an 8-bit tile
    static constexpr int kWorkers = Q8 ? 8 : 4;              // warps that clear and widen: 8 bits, four for keys and four for values
    static constexpr int kThreads = (8 + kWorkers + 4) * 32;
    // Registers of a thread after the start, by role: over the warpgroups they sum to what the launch has, 4 * 128 or 5 * 96.
    static constexpr int kLaunchRegs = Q8 ? 96 : 128, kSoftmaxRegs = Q8 ? 128 : 176, kWorkerRegs = 64, kSingleRegs = 96;
};

// How shared memory is shared out: two halves of queries, as many rows of each as a launch has (a product reads 128 rows
// all the same; what the others hold goes nowhere), then the ring of tiles and 8-bit tiles.  Four tiles of the ring
// keep both products fed where 8-bit ones are widened into it; the rest holds copies under way.
template <int D, bool Q8>
inline void share_out(AttentionArgs *a, int room) {
    using L = Layout<D, Q8>;
    a->q_sub = (a->q_nodes * a->group + 7) / 8 * 1024;
    int left = room - 2 * a->q_sub * (D / 64);
    a->ring = Q8 ? (D == 128 ? 4 : 8) : std::min(8, left / L::kTileBytes);
    left -= a->ring * L::kTileBytes;
    a->stages = Q8 ? std::min(8, left / L::kStageBytes) / 2 * 2 : 0;  // (even: keys and values have slots of their own)
}

// A CTA's run of the list, cut at the blocks' borders.
struct Piece {
    int shared, two;     // of the prefix; two products a tile
    int b, g, first, rows;
    int t0, t1, tiles;   // the piece's tiles, of the block's
    int context;         // own: the context's tiles; the nodes' follow
    int plain0, plain1;  // tiles of the context that begin and end inside it: every row sees every key
    int at, from, to;    // tile 0's first position; the positions that are the piece's
    int turn;            // one product a tile: tile t0 is product `turn`'s, and so on in turn
    int last;            // no piece: the run is over
    int odd;             // a value of its nodes is not finite
};
constexpr int kPieces = 4;

struct Control {  // behind the tiles in shared memory
    Piece pieces[kPieces];
    uint64_t piece_there[kPieces], piece_done[kPieces];
    uint64_t full[8], empty[8];    // ring of tiles
    uint64_t copied[8];            // a slot's values are there, to be cleared in part
    uint64_t staged[8], free_[8];  // ring of 8-bit tiles
    uint64_t q_full[2], q_empty[2];
    uint64_t scores[2], weights[2][2], sums[2];  // of the two products; weights of a tile's first and second 64 keys
    uint64_t joined[2];            // both warpgroups: statistics there, sums read
    uint64_t drained;
    uint32_t tmem;
    int gave_up;
    int scan[20];
    int total, b, before;          // tiles in all; the sequence a CTA begins in and the tiles before it
    float2 stats[2][kTile];
};

// The pieces of a CTA, in order.
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
        p->last = 0;
        p->shared = shared;
        p->two = rows > a.half_nodes * a.group;
        p->b = shared ? 0 : b;
        p->g = item / blocks;
        p->first = block * rows;
        p->rows = min(rows, all - p->first);
        p->tiles = shared ? shared_tiles : tiles;
        p->t0 = t;
        p->t1 = min(p->tiles, t + left);
        p->context = shared ? shared_tiles : context;
        p->at = shared ? 0 : a.shared_len / kTile * kTile;
        p->from = shared ? 0 : a.shared_len;
        p->to = shared ? a.shared_len : len;
        p->plain0 = (p->from - p->at + kTile - 1) / kTile;
        p->plain1 = (p->to - p->at) / kTile;
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

// The row of the batch that row r of a piece is.
struct RowId {
    int b, n, h;
};
__device__ __forceinline__ RowId row_id(const AttentionArgs &a, const Piece &p, int r) {
    const int i = (p.first + r) / a.group, h = (p.first + r) % a.group;
    return RowId{p.shared ? i / a.N : p.b, p.shared ? i % a.N : i, p.g * a.group + h};
}

// e4m3 values times 2^(byte - 127), four at a time: exact steps, by the conversions that there are (of which each
// takes less than moving the bits by shifts and masks, or by multiplications).
template <typename T>
struct Widen;
template <>
struct Widen<__nv_bfloat16> {
    static constexpr uint32_t again = 0;
    float m;
    __device__ __forceinline__ void scale(uint32_t byte) { m = scale_of(byte); }
    __device__ __forceinline__ uint2 four(uint32_t w) const {
        const float2 a = e4m3x2(w), b = e4m3x2(w >> 16);
        return make_uint2(Elt<__nv_bfloat16>::from_float2(a.x * m, a.y * m), Elt<__nv_bfloat16>::from_float2(b.x * m, b.y * m));
    }
};
template <>
struct Widen<__half> {
    // fp16 has the powers 2^-24 .. 2^15.  A row written from bf16 may have others: the row is multiplied by one of them,
    // which is exact or overflows as the whole would, and then again by what is left (0: nothing).
    uint32_t m, again;
    static __device__ __forceinline__ uint32_t power(int e) {
        const uint32_t s = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : 1u << (e + 24);
        return s | s << 16;
    }
    __device__ __forceinline__ void scale(uint32_t byte) {
        const int e = static_cast<int>(byte) - 127;
        again = 0;
        if (e > 15) m = power(15), again = power(min(e - 15, 15));
        else if (e < -24) m = power(-15), again = power(max(e + 15, -24));  // (448 * 2^-39 rounds to 0, as any less does)
        else m = power(e);
        if (byte == 255) m = 0x7fff7fffu;
    }
    static __device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
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

// Where a piece leaves its rows' sums, four columns at a time (a warp's rows lie next to each other), and (maximum, sum).
struct Part {
    float *sums;    // [D / 4][rows][4]
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

// Values of nodes m0 .. m1 - 1 that are not finite, to a row of node n that sees them: its columns [d0, d1), already
// written, four next to each other and `step` from there to the next four.  Out of line: it is hardly ever called, and inlined it would keep registers from what is.
template <typename T, typename X>
__device__ __noinline__ void add_odd(const AttentionArgs &a, int b, int g, int n, int m0, int m1, int d0, int d1, int D, X *to, int step) {
    for (int m = m0; m < m1; ++m) {
        const bool on = a.mask ? a.mask[static_cast<size_t>(n) * ((a.N + 31) / 32) + m / 32] >> (m & 31) & 1 : m <= n;
        if (!on) continue;
        const T *v = reinterpret_cast<const T *>(a.v) + b * a.stride[4] + m * a.stride[5] + g * D;
        for (int d = d0; d < d1; ++d) {
            const float y = static_cast<float>(v[d]);
            X &x = to[static_cast<size_t>(d / 4) * step + d % 4];
            if (!isfinite(y)) x = static_cast<X>(static_cast<float>(x) + y);
        }
    }
}

// ------------------------------------------------------------------ the kinds of warps
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
    uint32_t queries, tiles, stages;  // shared-memory addresses: of queries, of the ring, of 8-bit tiles
    uint32_t tmem;
    int lane, warp;
    int piece_at = 0;
    uint32_t piece_round = 0;

    __device__ __forceinline__ bool wait(const uint64_t *bar, uint32_t parity) {
        return wait_phase<false>(ptx::smem_addr(bar), parity, &c->gave_up, a.status);
    }
    __device__ __forceinline__ bool hurry(const uint64_t *bar, uint32_t parity) {
        return wait_phase<true>(ptx::smem_addr(bar), parity, &c->gave_up, a.status);
    }
    __device__ __forceinline__ bool wait1(const uint64_t *bar, uint32_t parity) {
        return wait_alone(ptx::smem_addr(bar), parity, &c->gave_up, a.status);
    }
    __device__ __forceinline__ uint32_t ring(int slot) const { return tiles + slot * L::kTileBytes; }
    __device__ __forceinline__ uint32_t query_half(int h) const { return queries + h * (D / 64) * a.q_sub; }

    // Test builds only: whether this CTA leaves out a worker's arrivals (0), the first softmax warp's (1), the list's (2).
#ifdef SPEC_TEST_HOOKS
    __device__ __forceinline__ bool withheld(int what) const { return a.withhold == static_cast<int>(blockIdx.x) * 4 + what; }
#else
    static __device__ __forceinline__ constexpr bool withheld(int) { return false; }
#endif
    // ---- pieces: one warp walks the list; the others take them in turn, and say when they are done with one
    __device__ __forceinline__ const Piece *piece() const { return c->pieces[piece_at].last ? nullptr : &c->pieces[piece_at]; }
    __device__ __forceinline__ const Piece *next_piece() { return wait(&c->piece_there[piece_at], piece_round) ? piece() : nullptr; }
    __device__ __forceinline__ const Piece *next_piece1() { return wait1(&c->piece_there[piece_at], piece_round) ? piece() : nullptr; }
    __device__ __forceinline__ void done_piece1() {
        arrive(ptx::smem_addr(&c->piece_done[piece_at]));
        if (++piece_at == kPieces) piece_at = 0, piece_round ^= 1;
    }
    __device__ __forceinline__ void done_piece() {
        __syncwarp();
        if (lane == 0) arrive(ptx::smem_addr(&c->piece_done[piece_at]));
        if (++piece_at == kPieces) piece_at = 0, piece_round ^= 1;
    }
    // Whether values of a tile are to be looked through: the context's ends, and the nodes.
    static __device__ __forceinline__ bool plain(const Piece &p, int t) { return t >= p.plain0 && t < p.plain1; }

    __device__ __forceinline__ bool announce(const Piece &p) {
        if (!wait(&c->piece_done[piece_at], piece_round ^ 1)) return false;
        if (lane == 0) {
            c->pieces[piece_at] = p;
            if (!withheld(2)) arrive(ptx::smem_addr(&c->piece_there[piece_at]));
        }
        __syncwarp();
        if (++piece_at == kPieces) piece_at = 0, piece_round ^= 1;
        return true;
    }
    // 8 bits: the products take the ring's tiles in turn across pieces, so that each has slots of its own there (the
    // ring's are a multiple of four) and need not see the other's, which the workers may be late with.
    static __device__ __forceinline__ bool next_of(Walk &walk, Piece *p, int &tiles) {
        const bool more = walk.next(p);
        p->last = !more;
        p->odd = 0;
        p->turn = Q8 ? tiles & 1 : 0;
        tiles += p->t1 - p->t0;
        return more;
    }
    // The queries of a piece: a half holds a.half_nodes nodes, whose heads of the group lie next to each other.
    struct Queries {
        uint32_t round = 0, issued = 0;  // a bit a half
        int half = 0;
    };
    __device__ __forceinline__ bool load_queries(const Piece &p, const Maps &maps, Queries &q) {
        if (p.two) q.half = 0;
        for (int h = 0; h < 2; ++h) {
            if (!p.two && h != q.half) continue;
            if (!wait(&c->q_empty[h], (q.round >> h & 1) ^ 1)) return false;
            q.round ^= 1u << h;
            q.issued |= 1u << h;
            const uint32_t bar = ptx::smem_addr(&c->q_full[h]);
            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, a.q_nodes * a.group * D * 2);
            __syncwarp();
            const int node = p.first / a.group + (p.two ? h * a.half_nodes : 0);
            const int z = a.q_merged && !p.shared ? p.b * a.N + node : node, b = a.q_merged ? 0 : p.b;
            if (lane < D / 64) tma_load4(query_half(h) + lane * a.q_sub, &maps.q, lane * 64, p.g * a.group, z, b, bar, policy_evict_normal());
        }
        if (!p.two) q.half ^= 1;
        return true;
    }
    __device__ void lead(const Maps &maps) {
        Walk walk(a, c);
        Piece p;
        Queries q;
        int tiles = 0;
        while (true) {
            const bool more = next_of(walk, &p, tiles);
            if (!announce(p) || !more || !load_queries(p, maps, q)) break;
        }
        if (c->gave_up) drain(c->q_full, 2, q.issued, ~q.round);
    }

    // ---- TMA
    // The keys and values of one tile of the context, in boxes of at most a page: lane i the i-th.
    struct Boxes {
        int page, y;
    };
    __device__ __forceinline__ Boxes boxes_of(const Piece &p, int t, int box, bool &bad) const {
        const long long pos = static_cast<long long>(p.at) + t * kTile + lane * box;
        Boxes b{a.cache.pages, (p.g << a.cache.page_bits) + static_cast<int>(pos & ((1 << a.cache.page_bits) - 1))};  // outside: zeros
        if (lane < kTile / box && pos < p.to && pos + box > p.from) {
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
    struct Tiles {
        Cursor at;
        bool bad = false;
        uint32_t issued = 0, rounds = 0, copied = 0, copies = 0;  // a bit a slot: loaded; its last phase's parity; the same of `copied`
    };
    __device__ __forceinline__ bool load_tiles(const Piece &p, const Maps &maps, Tiles &s) {
        const int box = box_rows();
        const uint64_t normal = policy_evict_normal();
        // tiles that one block takes are read once; where several blocks take them, L2 may keep them
        const uint64_t policy = (p.shared ? a.shared_blocks : a.blocks) == 1 ? ptx::policy_evict_first() : normal;
        for (int t = p.t0; t < p.t1; ++t) {
            Boxes boxes;
            if (!Q8 && t < p.context) boxes = boxes_of(p, t, box, s.bad);
            for (int w = 0; w < 2; ++w, s.at.step(a.ring)) {
                if (!wait(&c->empty[s.at.slot], s.at.round ^ 1)) return false;
                const uint32_t full = ptx::smem_addr(&c->full[s.at.slot]), to = ring(s.at.slot), bit = 1u << s.at.slot;
                if (Q8 && t < p.context) {
                    if (lane == 0) arrive(full);
                    __syncwarp();
                    continue;
                }
                // Values that the workers look through first: their copy is waited for there.
                const bool checked = w && !plain(p, t);
                const uint32_t bar = checked ? ptx::smem_addr(&c->copied[s.at.slot]) : full;
                if (lane == 0) {
                    if (checked) arrive(full);
                    ptx::mbar_arrive_expect_tx(bar, L::kTileBytes);
                }
                __syncwarp();
                if (t >= p.context) {
                    if (lane < D / 64) tma_load4(to + lane * (kTile * 128), w ? &maps.v_nodes : &maps.k_nodes, lane * 64, p.g, (t - p.context) * kTile, p.b, bar, normal);
                } else if (lane < kTile / box) {
                    for (int x = 0; x < D; x += 64) tma_load3(to + (x / 64) * (kTile * 128) + lane * box * 128, w ? &maps.v : &maps.k, x, boxes.y, boxes.page, bar, policy);
                }
                if (checked) s.copied |= bit, s.copies ^= bit;
                else s.issued |= bit, s.rounds = (s.rounds & ~bit) | s.at.round << s.at.slot;
            }
        }
        return true;
    }
    __device__ __forceinline__ void end_tiles(const Tiles &s) {
        if (s.bad) atomicOr(a.status, SPEC_DEV_BAD_PAGE);
        if (!c->gave_up) return;
        drain(c->full, a.ring, s.issued, s.rounds);
        drain(c->copied, a.ring, s.copied, ~s.copies);
    }
    __device__ void load_tiles(const Maps &maps) {
        Tiles s;
        for (const Piece *p; (p = next_piece()) && load_tiles(*p, maps, s);) done_piece();
        end_tiles(s);
    }
    // The list, the queries and the ring by one warp, which has the next piece announced before a piece's tiles.
    __device__ void lead_tiles(const Maps &maps) {
        Walk walk(a, c);
        Piece p, next;
        Queries q;
        Tiles s;
        int tiles = 0;
        bool more = next_of(walk, &p, tiles), ok = announce(p);
        while (ok && more) {
            more = next_of(walk, &next, tiles);
            ok = announce(next) && load_queries(p, maps, q) && load_tiles(p, maps, s);
            p = next;
        }
        end_tiles(s);
        if (c->gave_up) drain(c->q_full, 2, q.issued, ~q.round);
    }
    // 8-bit tiles, to be widened.
    __device__ void load_stages(const Maps &maps) {
        Cursor at;
        const uint64_t once = ptx::policy_evict_first(), normal = policy_evict_normal();
        const int box = box_rows();
        bool bad = false, ok = true;
        uint32_t issued = 0, rounds = 0;
        for (const Piece *pp; ok && (pp = next_piece()); done_piece()) {
            const Piece &p = *pp;
            const uint64_t policy = (p.shared ? a.shared_blocks : a.blocks) == 1 ? once : normal;
            const int t1 = min(p.t1, p.context);
            for (int t = p.t0; ok && t < t1; ++t) {
                const Boxes boxes = boxes_of(p, t, box, bad);
                for (int w = 0; w < 2; ++w) {
                    if (!(ok = wait(&c->free_[at.slot], at.round ^ 1))) break;
                    const uint32_t bar = ptx::smem_addr(&c->staged[at.slot]);
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, L::kStageBytes);
                    __syncwarp();
                    if (lane < kTile / box) tma_load3(stages + at.slot * L::kStageBytes + lane * box * D, w ? &maps.v : &maps.k, 0, boxes.y, boxes.page, bar, policy);
                    issued |= 1u << at.slot;
                    rounds = (rounds & ~(1u << at.slot)) | at.round << at.slot;
                    at.step(a.stages);
                }
            }
        }
        if (bad) atomicOr(a.status, SPEC_DEV_BAD_PAGE);
        if (c->gave_up) drain(c->staged, a.stages, issued, rounds);
    }

    // ---- tcgen05.mma: a lane a product.  The tensor cores hold few products ahead, so what a lane does between
    // its own is hidden behind the other's.  A slot of the ring is free after two arrivals: one of each lane, used or
    // not; 8 bits, one product a tile: both of the lane that uses it.
    __device__ __forceinline__ bool add_values(int s, const Cursor &values, uint32_t round, bool add, bool last, bool alone) {
        const uint32_t d = tmem + kSums + s * 128, x = tmem + kScores + s * 128, v = operand(ring(values.slot), kTile * 128);
        if (!wait1(&c->full[values.slot], values.round) || !wait1(&c->weights[s][0], round)) return false;
        fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k) mma_tmem(d, x + k * 8, descriptor(v + k * 128), kSumsInstr, add || k > 0);
        if (!wait1(&c->weights[s][1], round)) return false;
        fence_after();
#pragma unroll
        for (int k = kTile / 32; k < kTile / 16; ++k) mma_tmem(d, x + k * 8, descriptor(v + k * 128), kSumsInstr, true);
        mma_commit(ptx::smem_addr(&c->empty[values.slot]));
        if (alone) mma_commit(ptx::smem_addr(&c->empty[values.slot]));
        if (last) mma_commit(ptx::smem_addr(&c->sums[s]));
        return true;
    }
    __device__ void multiply(int s) {
        Cursor at;
        uint32_t round = 0, q_round = 0;  // of the weights; a bit a half
        const uint32_t sub = a.q_sub / 16, x = tmem + kScores + s * 128;
        int half = 0;
        bool ok = true;
        for (const Piece *p; ok && (p = next_piece1()); done_piece1()) {
            const int n = p->t1 - p->t0;
            const bool two = p->two;
            if (two) half = 0;
            for (int h = 0; ok && h < 2; ++h) {
                if (!two && h != half) continue;
                ok = wait1(&c->q_full[h], q_round >> h & 1);
                q_round ^= 1u << h;
            }
            if (!ok) break;
            const int own = two ? s : half, turn = p->turn ^ s, used = two ? n : (n - turn + 1) / 2;
            const bool alone = Q8 && !two;
            if (two) arrive(ptx::smem_addr(&c->q_empty[1 - s]));
            else if (used == 0) arrive(ptx::smem_addr(&c->q_empty[half]));
            const uint32_t q = operand(query_half(own), 16);
            Cursor values;
            int done = 0;  // own tiles whose scores are under way
            for (int i = 0; ok && i < n; ++i) {
                const Cursor keys = at;
                at.step(a.ring);
                const Cursor next = at;
                at.step(a.ring);
                if (!two && (i & 1) != turn) {
                    if (alone) continue;
                    if (!(ok = wait1(&c->full[keys.slot], keys.round))) break;
                    arrive(ptx::smem_addr(&c->empty[keys.slot]));
                    if (!(ok = wait1(&c->full[next.slot], next.round))) break;
                    arrive(ptx::smem_addr(&c->empty[next.slot]));
                    continue;
                }
                if (done) {
                    if (!(ok = add_values(s, values, round, done > 1, false, alone))) break;
                    round ^= 1;
                }
                if (!(ok = wait1(&c->full[keys.slot], keys.round))) break;
                fence_after();
                const uint32_t k = operand(ring(keys.slot), 16);
#pragma unroll
                for (int e = 0; e < D / 16; ++e) mma(x, descriptor(q + (e / 4) * sub + (e % 4) * 2), descriptor(k + (e / 4) * (kTile * 128 / 16) + (e % 4) * 2), kScoresInstr, e > 0);
                mma_commit(ptx::smem_addr(&c->scores[s]));
                mma_commit(ptx::smem_addr(&c->empty[keys.slot]));
                if (alone) mma_commit(ptx::smem_addr(&c->empty[keys.slot]));
                if (++done == used) mma_commit(ptx::smem_addr(&c->q_empty[own]));
                values = next;
            }
            if (ok && used) {
                ok = add_values(s, values, round, done > 1, true, alone);
                round ^= 1;
            }
            if (!two) half ^= 1;
        }
        // Every product done before tensor memory is freed, also where a wait gave up.
        mma_commit(ptx::smem_addr(&c->drained));
        bool done = false;
        for (int n = 0; !done && n < kWaitTries; ++n) done = ptx::mbar_try_wait(ptx::smem_addr(&c->drained), 0);
    }

    // ---- workers: a thread a row
    static constexpr int kLanes = D / 8;  // 16-byte chunks of a row
    __device__ __forceinline__ static bool odd_pair(uint32_t x) {  // an infinity or NaN among two elements
        constexpr uint32_t e = kHalf ? 0x7c00u : 0x7f80u;
        return (x & e) == e || (x >> 16 & e) == e;
    }
    // The rows of a tile of values outside [from, to) become 0.
    __device__ __forceinline__ void clear_rows(uint32_t at, int r, int from, int to) const {
        if (r >= from && r < to) return;
#pragma unroll 4
        for (int x = 0; x < kLanes; ++x) store16(at + chunk_at(r, x), make_uint4(0, 0, 0, 0));
    }
    // Values of nodes that are not finite become 0 (true: there were some): a row that does not see them would
    // get 0 * NaN.  The rows that do are given them at the end.
    __device__ __forceinline__ bool take_odd(uint32_t at, int r) const {
        bool odd = false;
#pragma unroll 4
        for (int i = 0; i < kLanes; ++i) {
            const uint32_t to = at + chunk_at(r, i);
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
    // The row of a thread at position `pos` of a piece: its page as the table has it (-1: no such row), and the scale of its
    // keys (which = 0) or values, from a page.
    __device__ __forceinline__ int row_page(const int32_t *table, int pos, int from, int to) const {
        return pos >= from && pos < to ? __ldg(table + (pos >> a.cache.page_bits)) : -1;
    }
    __device__ __forceinline__ uint32_t row_scale(int page, int pos, int g, int which) const {
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.cache.pages)) return kNoRow;
        const int in_page = (g << a.cache.page_bits) + (pos & ((1 << a.cache.page_bits) - 1));
        const size_t row = static_cast<size_t>(static_cast<uint32_t>(page)) * static_cast<uint32_t>(a.cache.kv_heads << a.cache.page_bits) + in_page;
        return __ldg(a.cache.scale[which] + row);
    }
    static constexpr uint32_t kNoRow = 256;
    // An 8-bit tile, widened: the chunks of 16 in turned order, so that eight rows' meet different banks.
    __device__ __forceinline__ void widen(uint32_t from, uint32_t to, int r, const Widen<T> &w) const {
        constexpr int kChunks = D / 16, kAhead = 2;
#pragma unroll 1
        for (int j0 = 0; j0 < kChunks; j0 += kAhead) {
            uint4 v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) v[j] = load16(from + r * D + turned(j0 + j, r) * 16);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int x = turned(j0 + j, r);
                const uint2 b0 = w.four(v[j].x), b1 = w.four(v[j].y);
                store16(to + chunk_at(r, 2 * x), make_uint4(b0.x, b0.y, b1.x, b1.y));
                const uint2 b2 = w.four(v[j].z), b3 = w.four(v[j].w);
                store16(to + chunk_at(r, 2 * x + 1), make_uint4(b2.x, b2.y, b3.x, b3.y));
            }
        }
    }
    // A widened row times w.again, where its power of two takes two steps.
    __device__ __forceinline__ void widen_again(uint32_t to, int r, uint32_t m) const {
#pragma unroll 1
        for (int i = 0; i < kLanes; ++i) {
            uint4 v = load16(to + chunk_at(r, i));
            v.x = Widen<__half>::times(v.x, m), v.y = Widen<__half>::times(v.y, m), v.z = Widen<__half>::times(v.z, m), v.w = Widen<__half>::times(v.w, m);
            store16(to + chunk_at(r, i), v);
        }
    }
    static __device__ __forceinline__ int turned(int j, int r) { return D == 128 ? (j + r) & 7 : (j + (r >> 1)) & 3; }
    // 8 bits: keys (which = 0) or values (1) widened, values of nodes looked through.  Both rings have an even number of
    // slots, so keys and values have slots of their own and neither's warps wait for the other's.
    __device__ void work8(int r, int which) {
        Cursor at, staged;
        at.slot = staged.slot = which;
        uint32_t copies = 0;
        bool ok = true;
        for (const Piece *pp; ok && (pp = next_piece()); done_piece()) {
            const Piece &p = *pp;
            // Two dependent loads, each issued a tile ahead of its use.
            const int32_t *table = a.cache.table + static_cast<size_t>(p.b) * a.cache.table_width;
            const int from = p.from, end = min(p.to, p.at + p.t1 * kTile), context = p.context, t1 = p.t1, g = p.g;
            int pos = p.at + p.t0 * kTile + r;
            uint32_t next_byte = row_scale(row_page(table, pos, from, end), pos, g, which);
            int next_page = row_page(table, pos + kTile, from, end);
            for (int t = p.t0; ok && t < t1; ++t, pos += kTile) {
                const uint32_t byte = next_byte, to = ring(at.slot);
                next_byte = row_scale(next_page, pos + kTile, g, which);
                next_page = row_page(table, pos + 2 * kTile, from, end);
                if (!(ok = hurry(&c->empty[at.slot], at.round ^ 1))) break;
                if (t < context) {
                    if (!(ok = hurry(&c->staged[staged.slot], staged.round))) break;
                    if (byte != kNoRow) {
                        Widen<T> x;
                        x.scale(byte);
                        widen(stages + staged.slot * L::kStageBytes, to, r, x);
                        if (kHalf && x.again) widen_again(to, r, x.again);
                    } else {
                        clear_rows(to, r, 0, 0);
                    }
                    __syncwarp();
                    if (lane == 0) arrive(ptx::smem_addr(&c->free_[staged.slot]));
                    staged.step(a.stages);
                    staged.step(a.stages);
                    fence_async();
                } else if (which) {
                    if (!(ok = look_through(p, at.slot, to, r, copies))) break;
                }
                __syncwarp();
                if (lane == 0 && !(warp == 8 && withheld(0))) arrive(ptx::smem_addr(&c->full[at.slot]));
                at.step(a.ring);
                at.step(a.ring);
            }
        }
    }
    __device__ __forceinline__ bool look_through(const Piece &p, int slot, uint32_t to, int r, uint32_t &copies) {
        if (!wait(&c->copied[slot], copies >> slot & 1)) return false;
        copies ^= 1u << slot;
        if (take_odd(to, r)) *const_cast<volatile int *>(&c->pieces[piece_at].odd) = 1;
        fence_async();
        return true;
    }
    __device__ void work(int r) {
        Cursor at;
        uint32_t copies = 0;  // the parity of each slot's next copy to look through
        bool ok = true;
        for (const Piece *pp; ok && (pp = next_piece()); done_piece()) {
            const Piece &p = *pp;
            for (int t = p.t0; ok && t < p.t1; ++t)
                for (int w = 0; ok && w < 2; ++w, at.step(a.ring)) {
                    const uint32_t to = ring(at.slot);
                    if (!(ok = wait(&c->empty[at.slot], at.round ^ 1))) break;
                    if (w && t >= p.context) {
                        if (!(ok = look_through(p, at.slot, to, r, copies))) break;
                    } else if (w && !plain(p, t)) {
                        if (!(ok = wait(&c->copied[at.slot], copies >> at.slot & 1))) break;
                        copies ^= 1u << at.slot;
                        const int base = p.at + t * kTile;
                        clear_rows(to, r, p.from - base, p.to - base);
                        fence_async();
                    }
                    __syncwarp();
                    if (lane == 0 && !(warp == 8 && withheld(0))) arrive(ptx::smem_addr(&c->full[at.slot]));
                }
        }
    }

    // ---- softmax
    // Which of a tile's columns 32 k .. 32 k + 31 a row of node n sees: a bit a column.
    __device__ __forceinline__ uint32_t seen(const Piece &p, int t, int n, int k) const {
        if (t < p.context) {
            const int at = p.at + t * kTile + 32 * k;
            const int from = min(max(p.from - at, 0), 32), to = min(max(p.to - at, 0), 32);
            return static_cast<uint32_t>((1ull << to) - 1) & ~static_cast<uint32_t>((1ull << from) - 1);
        }
        const int m = (t - p.context) * kTile + 32 * k;
        if (m >= a.N) return 0;
        uint32_t w = a.N - m < 32 ? (1u << (a.N - m)) - 1 : ~0u;
        if (a.mask) w &= __ldg(a.mask + static_cast<size_t>(n) * ((a.N + 31) / 32) + m / 32);
        else w &= static_cast<uint32_t>((1ull << min(max(n - m + 1, 0), 32)) - 1);
        return w;
    }
    static __device__ __forceinline__ float largest(const uint32_t (&x)[32], uint32_t w) {
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], !((w >> j) & 1) ? -INFINITY : __uint_as_float(x[j]));
        return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    }
    // Weights of 32 columns; their sum is added to `sum`.
    static __device__ __forceinline__ void weigh(const uint32_t (&x)[32], uint32_t w, float2 scale, float2 sub, float2 (&sum)[2], uint32_t (&y)[16]) {
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            float2 e = fma2(make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), scale, sub);
            e.x = ptx::ex2(e.x);
            e.y = ptx::ex2(e.y);
            if (!((w >> j) & 1)) e.x = 0.0f;
            if (!((w >> (j + 1)) & 1)) e.y = 0.0f;
            sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], e);
            y[j / 2] = Elt<T>::from_float2(e.x, e.y);
        }
    }
    // A row's maximum and sum move on to what `top`, the largest score of a tile, asks for; the sums are scaled along.
    // `m` is what the exponents subtract, in units of log 2; -inf while the row has seen nothing.
    __device__ __forceinline__ void move_on(float top, bool live, uint32_t o_at, bool first, float &m, float &l) const {
        const float want = top - kShift;
        const bool moves = live && (m == -INFINITY ? want > -INFINITY : want > m + 8.0f);
        if (!__any_sync(0xffffffffu, moves)) return;
        const float f = moves ? (m == -INFINITY ? 0.0f : ptx::ex2(m - want)) : 1.0f;
        l *= f;
        if (moves) m = want;
        __syncwarp();  // tensor memory's loads and stores take the warp as one: here and below, behind what parts it
        if (first) return;
#pragma unroll 1
        for (int k = 0; k < D; k += 16) {
            uint32_t y[16];
            tmem_load16(y, o_at + k);
            wait_loads(y);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
            tmem_store16(o_at + k, y);
        }
    }
    __device__ __forceinline__ void weights_there(int s, int h, uint32_t arrivals) {
        wait_stores();
        fence_before();
        __syncwarp();
        if (lane == 0 && !(warp == 0 && withheld(1))) arrive(ptx::smem_addr(&c->weights[s][h]), arrivals);
    }
    // A tile's scores into weights, whose halves the products may take one after the other: the row's maximum, then the
    // weights, 32 columns at a time, in loops that read tensor memory twice.  Code counts here, since the kinds of warps share
    // the instruction caches: with one reading, all 128 columns unrolled and their weights held until the maximum is known
    // to stand, 48 x 9 nodes behind 16384 shared tokens take 172 us, in loops of 64 columns 162, in these 158.
    // MASKED: a row sees some of the columns; those that no row sees (behind a context's end, beyond few nodes) are skipped.
    template <bool MASKED>
    __device__ __forceinline__ void tile_weights(int s, uint32_t arrivals, bool live, uint32_t (&w)[4], uint32_t s_at, uint32_t o_at, float scale, bool first, float &m, float &l) {
        const auto next = [&] {
            const uint32_t x = w[0];
            w[0] = w[1], w[1] = w[2], w[2] = w[3], w[3] = x;
            return x;
        };
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        const float2 c2 = make_float2(scale, scale);
        float top = -INFINITY;
        __syncwarp();
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            const uint32_t seen = MASKED ? next() : ~0u;
            if (MASKED && !__any_sync(0xffffffffu, seen != 0)) continue;
            uint32_t x[32];
            tmem_load32(x, s_at + 32 * k);
            wait_loads(x);
            top = fmaxf(top, largest(x, seen));
        }
        move_on(top * scale, live, o_at, first, m, l);
        const float sub = m == -INFINITY ? 0.0f : -m;
        const float2 s2 = make_float2(sub, sub);
        __syncwarp();
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            const uint32_t seen = MASKED ? next() : ~0u;
            uint32_t p[16];
            if (MASKED && !__any_sync(0xffffffffu, seen != 0)) {
#pragma unroll
                for (int j = 0; j < 16; ++j) p[j] = 0;
            } else {
                uint32_t x[32];
                tmem_load32(x, s_at + 32 * k);
                wait_loads(x);
                weigh(x, seen, c2, s2, sum, p);
            }
            tmem_store16(s_at + 16 * k, p);
            if (k & 1) weights_there(s, k >> 1, arrivals);
        }
        const float2 both = add2(sum[0], sum[1]);
        l += both.x + both.y;
    }

    // Columns [d0, d1) of the block's row r: f0 * product 0's sums + f1 * product 1's, to where the piece's go.
    __device__ void write_sums(const Piece &p, int r, int d0, int d1, bool use0, bool use1, float f0, float f1, float m, float l) {
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
        f0 *= inv;
        f1 *= inv;
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
            if (live && final) {
                uint4 *out = reinterpret_cast<uint4 *>(a.out + (row * D + d) * 2);
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(x[j + e]);
                    out[j / 8] = pack8<T>(v);
                }
            } else if (live) {
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    reinterpret_cast<float4 *>(to.sums)[(d + j) / 4 * to.rows + r] =
                        make_float4(__uint_as_float(x[j]), __uint_as_float(x[j + 1]), __uint_as_float(x[j + 2]), __uint_as_float(x[j + 3]));
            }
        }
        if (*const_cast<volatile const int *>(&p.odd) && live) {
            const int m0 = max(p.t0 - p.context, 0) * kTile, m1 = min((p.t1 - p.context) * kTile, a.N);
            if (final) add_odd<T>(a, p.b, p.g, id.n, m0, m1, d0, d1, D, reinterpret_cast<T *>(a.out) + row * D, 4);
            else add_odd<T>(a, p.b, p.g, id.n, m0, m1, d0, d1, D, to.sums + 4 * r, 4 * to.rows);
        }
    }
    __device__ void softmax(int s, int tid) {
        uint32_t scores_round = 0, sums_round = 0, joined_round = 0;
        bool ok = true, after_two = false;  // the piece before had two products a tile
        const float scale = a.scale * kLog2e;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, at bit 16
        const uint32_t s_at = tmem + lanes + kScores + s * 128, o_at = tmem + lanes + kSums + s * 128;
        const int half_rows = a.half_nodes * a.group;
        for (const Piece *p; ok && (p = next_piece()); done_piece()) {
            const bool two = p->two;
            const int r = (tid < half_rows ? tid : kBlockRows) + (two ? s * half_rows : 0);  // this thread's row of the block
            const bool idle = (warp & 3) != 0 && __all_sync(0xffffffffu, r >= p->rows);  // the warp has none: it only counts
            // The first warp arrives for those that are idle.  (A last block may have no rows for product 1.)  But behind a piece of
            // two products, whose warps nothing else brings together, each arrives for itself at a product's first tile: a product must
            // not write over sums that a warp, idle now, still reads, nor leave it behind by more than a phase of `sums`.
            const bool has_row = r < p->rows;
            const int live = max(1, (min(half_rows, p->rows - (two ? s * half_rows : 0)) + 31) / 32);
            const uint32_t arrivals = (warp & 3) == 0 ? 5 - live : 1, first_arrivals = after_two ? 1 : arrivals;
            const int t0 = p->t0, t1 = p->t1, plain0 = p->plain0, plain1 = p->plain1, n = row_id(a, *p, min(r, p->rows - 1)).n;
            float m = -INFINITY, l = 0.0f;
            bool first = true;
            const int turn = p->turn ^ s;
            const bool has_sums = two || t0 + turn < t1;  // (a product may have no tile of a piece)
            if (idle && after_two && has_sums) {
                fence_before();
                __syncwarp();
                if (lane < 2) arrive(ptx::smem_addr(&c->weights[s][lane]));
            }
            after_two = two;
            for (int t = idle ? t1 : t0 + (two ? 0 : turn); t < t1; t += two ? 1 : 2) {
                const bool masked = t < plain0 || t >= plain1;
                uint32_t w[4] = {};
                if (masked)
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = seen(*p, t, n, k);
                if (!(ok = hurry(&c->scores[s], scores_round))) break;
                scores_round ^= 1;
                fence_after();
                if (masked) tile_weights<true>(s, first ? first_arrivals : arrivals, has_row, w, s_at, o_at, scale, first, m, l);
                else tile_weights<false>(s, first ? first_arrivals : arrivals, has_row, w, s_at, o_at, scale, first, m, l);
                first = false;
            }
            if (!ok) break;
            if (has_sums) {
                if (!(ok = idle ? wait(&c->sums[s], sums_round) : hurry(&c->sums[s], sums_round))) break;
                sums_round ^= 1;
                fence_after();
            }
            if (idle) {  // the rounds that went by
                const int n = two ? t1 - t0 : (t1 - t0 - turn + 1) / 2;
                scores_round ^= n & 1;
            }
            // Two products a tile: each warpgroup writes its rows.  One: both products' sums are joined, and each
            // warpgroup writes half the columns.
            bool use0 = s == 0, use1 = s == 1;
            float f0 = 1.0f, f1 = 1.0f;
            if (!two) {
                c->stats[s][tid] = make_float2(m, l);
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(ptx::smem_addr(&c->joined[0]));
                if (!idle && !(ok = hurry(&c->joined[0], joined_round))) break;
                fence_after();
                const float2 x = c->stats[0][tid], y = c->stats[1][tid];
                use0 = t1 - t0 > 1 || p->turn == 0, use1 = t1 - t0 > 1 || p->turn == 1;
                m = fmaxf(x.x, y.x);
                f0 = x.x == -INFINITY ? 0.0f : ptx::ex2(x.x - m), f1 = y.x == -INFINITY ? 0.0f : ptx::ex2(y.x - m);
                l = x.y * f0 + y.y * f1;
            }
            if (!idle) write_sums(*p, r, two ? 0 : s * (D / 2), two ? D : (s + 1) * (D / 2), use0, use1, f0, f1, m, l);
            fence_before();
            if (!two) {
                __syncwarp();
                if (lane == 0) arrive(ptx::smem_addr(&c->joined[1]));
                if (!(ok = wait(&c->joined[1], joined_round))) break;
                joined_round ^= 1;
                fence_after();
            }
        }
    }
};

template <typename T, int D, bool Q8>
__global__ void __launch_bounds__(Layout<D, Q8>::kThreads, 1) attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Maps maps) {
    using L = Layout<D, Q8>;
    constexpr int kThreads = L::kThreads;
    extern __shared__ __align__(1024) unsigned char smem[];
    Control *c = reinterpret_cast<Control *>(smem + a.control);
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
        for (int i = 0; i < kPieces; ++i) {
            ptx::mbar_init(ptx::smem_addr(&c->piece_there[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->piece_done[i]), 8 + L::kWorkers + 3);
        }
        for (int i = 0; i < 8; ++i) {
            ptx::mbar_init(ptx::smem_addr(&c->full[i]), 4 + 1);
            ptx::mbar_init(ptx::smem_addr(&c->empty[i]), 2);
            ptx::mbar_init(ptx::smem_addr(&c->copied[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->staged[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->free_[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_addr(&c->q_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->q_empty[i]), 2);
            ptx::mbar_init(ptx::smem_addr(&c->scores[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->weights[i][0]), 4);
            ptx::mbar_init(ptx::smem_addr(&c->weights[i][1]), 4);
            ptx::mbar_init(ptx::smem_addr(&c->sums[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&c->joined[i]), 8);
        }
        ptx::mbar_init(ptx::smem_addr(&c->drained), 2);
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

    const uint32_t queries = ptx::smem_addr(smem), tiles_at = queries + 2 * (D / 64) * a.q_sub;
    Attention<T, D, Q8> x{a, c, queries, tiles_at, tiles_at + a.ring * L::kTileBytes, c->tmem, lane, warp};
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftmaxRegs));
        x.softmax(warp >> 2, tid & 127);
    } else {
        if (warp < kFirst) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kWorkerRegs));
        else if (L::kSingleRegs < L::kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kSingleRegs));
        if (warp < kFirst) {
            if (Q8) x.work8(tid & 127, (warp - 8) >> 2);
            else x.work(tid & 127);
        } else if (warp == kFirst + 1 || warp == kFirst + 2) {
            if (lane == 0) x.multiply(warp - kFirst - 1);
            __syncwarp();
        } else if (warp == kFirst) {
            if (Q8) x.lead_tiles(maps);
            else x.load_tiles(maps);
        } else {
            if (Q8) x.load_stages(maps);
            else x.lead(maps);
        }
    }

    fence_before();
    __syncthreads();
    if (warp == kFirst + 1) tmem_free(c->tmem, 512);
}

// ------------------------------------------------------------------ joining
// x * y / z for y <= kMaxCtas, in 32 bits where these do (all but lists of millions of tiles).
__device__ __forceinline__ int share_of(int x, int y, int z) {
    if (x < 1 << 24) return static_cast<int>(static_cast<uint32_t>(x) * static_cast<uint32_t>(y) / static_cast<uint32_t>(z));
    return static_cast<int>(static_cast<long long>(x) * y / z);
}

// 32 rows of a block, a lane each, D / 8 columns a warp: the partial sums of the pieces that hold them, in the order
// of their keys, and the result through shared memory, so that it is written in whole lines.  kAtOnce: pieces whose loads
// are under way together.
template <typename T, int D, int kAtOnce>
__global__ void __launch_bounds__(256, kAtOnce == 1 ? 4 : 1) attention_join_kernel(const __grid_constant__ AttentionArgs a) {
    constexpr int E = D / 8;
    __shared__ uint32_t result[32][D / 2 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = (a.block_rows + 31) / 32;
    const int first = blockIdx.x % chunks * 32, item = blockIdx.x / chunks;
    const int block = item % a.blocks, g = item / a.blocks % a.cache.kv_heads, b = item / a.blocks / a.cache.kv_heads;
    const int total = a.starts[a.B], start = a.starts[b], tiles = (a.starts[b + 1] - start) / (a.cache.kv_heads * a.blocks);
    if (tiles == 0) return;  // left out
    // The CTA whose run holds tile t: the least c with t < (c + 1) total / ctas, rounded down.
    const auto owner = [&](int t) {
        if (t < 1 << 24) return static_cast<int>(((t + 1u) * static_cast<uint32_t>(a.ctas) - 1) / static_cast<uint32_t>(total));
        return static_cast<int>(((t + 1ll) * a.ctas - 1) / total);
    };
    const int own0 = start + (g * a.blocks + block) * tiles, c0 = owner(own0), c1 = owner(own0 + tiles - 1);
    if (c0 == c1 && !a.shared_len) return;  // written already
    const int rows = min(a.block_rows, a.N * a.group - block * a.block_rows);  // of the block
    const int r = min(first + lane, rows - 1), in_seq = block * a.block_rows + r;
    const bool live = first + lane < rows;

    float m = -INFINITY, l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    const auto load = [&](const Part &p, int at, float2 &stat, float (&x)[E]) {
        stat = p.stats[at];
#pragma unroll
        for (int e = 0; e < E; e += 4)
            *reinterpret_cast<float4 *>(x + e) = reinterpret_cast<const float4 *>(p.sums)[(warp * E + e) / 4 * p.rows + at];
    };
    const auto add = [&](const float2 &s, const float (&x)[E]) {
        const float top = fmaxf(m, s.x), was = m == -INFINITY ? 0.0f : ptx::ex2(m - top), now = s.x == -INFINITY ? 0.0f : ptx::ex2(s.x - top);
        l = l * was + s.y * now;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * was + x[e] * now;
        m = top;
    };
    const auto take = [&](const Part &p, int at) {
        alignas(16) float x[E];
        float2 stat;
        load(p, at, stat, x);
        add(stat, x);
    };
    // Of a block whose tiles begin at t0: kAtOnce pieces' loads under way together, and added in order.
    const auto pieces = [&](int t0, int from, int to, int at) {
        for (int c = from; c <= to; c += kAtOnce) {
            alignas(16) float x[kAtOnce][E];
            float2 stat[kAtOnce];
            bool there[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int lo = share_of(total, c + k, a.ctas);
                there[k] = c + k <= to && lo != share_of(total, c + k + 1, a.ctas);  // (not a CTA without tiles)
                if (there[k]) load(cut_part<D>(a, c + k, t0 >= lo), at, stat[k], x[k]);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (there[k]) add(stat[k], x[k]);
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
