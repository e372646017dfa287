// attention.h -- what the host and the kernels of the attention share: tiles, the split of the work, the
// parameter block.
//
// The work is a list of tiles of 128 keys.  First the shared prefix: for each key head and block of up to
// 256 rows of the whole batch, its tiles.  Then sequence by sequence, key head by key head, block by
// block of up to 256 of the sequence's rows, the tiles of its own context and of its nodes.  A CTA takes
// an equal run of the list, wherever that begins and ends, so the split balances to a tile whatever
// the lengths; a block that several CTAs share leaves partial sums, which a second kernel joins.
#pragma once

#include <cuda.h>

#include "context.h"

namespace spec {
namespace context {

constexpr int kTile = 128;       // keys of a tile, rows of a matrix product
constexpr int kBlockRows = 256;  // rows of a block: two products share a tile of keys
constexpr int kMaxCtas = 160;    // one an SM

struct AttentionArgs {
    CacheView cache;
    const unsigned char *q, *k, *v;
    long long stride[6];  // batch and token strides of q, k, v, in elements
    const int32_t *lens;
    const uint32_t *mask;
    unsigned char *out;
    float *lse;
    uint32_t *status;
    int B, N, heads, shared_len;
    float scale;
    // the split
    int group;                        // query heads a key head
    int half_nodes;                   // whole nodes of a product's 128 rows
    int blocks, block_rows;           // of a sequence's N * group rows: whole nodes, two halves at most
    int shared_blocks, shared_rows;   // of the batch's B * N * group rows
    int q_nodes;                      // nodes that a copy of queries brings
    int q_merged;                     // the batch's nodes are evenly spaced: one axis
    int ctas;
    // shared memory: bytes of 64 columns of a half's queries, tiles in the ring, 8-bit tiles, where Control begins
    int q_sub, ring, stages, control;
    // the workspace
    int32_t *starts;   // [B + 1] tiles before each sequence's
    float *cut_sums;   // [ctas][2][D][kBlockRows]: blocks cut at a CTA's begin and at its end
    float2 *cut_stats; // ... their rows' (maximum in units of log 2, sum)
    float *row_sums;   // [2][kv_heads][blocks' rows, D columns a block], with a prefix: whole blocks, the sequences' own and the prefix's
    float2 *row_stats;
#ifdef SPEC_TEST_HOOKS
    int withhold;  // 4 * CTA + what it leaves out, so that a wait runs out (below 0: nothing)
#endif
};

// The driver's encoder of tensor maps (null where the driver has none).
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled();

// Tensor maps: the cache's keys and values, the queries, the nodes' keys and values.
struct Maps {
    CUtensorMap k, v, q, k_nodes, v_nodes;
};

__host__ __device__ inline int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }

template <typename T, int D, bool Q8>
spec_status launch_attention(const AttentionArgs &a, cudaStream_t stream);

}  // namespace context
}  // namespace spec
