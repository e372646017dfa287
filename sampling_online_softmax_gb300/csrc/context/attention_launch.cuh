// attention_launch.cuh -- the launcher of the attention, instantiated one element type a unit.
#pragma once

#include <algorithm>
#include <climits>

#include "attention.cuh"

namespace spec {

#ifdef SPEC_TEST_HOOKS
int test_withhold_unit();  // test builds only
#endif

namespace context {

inline spec_status encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
                          const cuuint32_t *box, bool swizzled) {
    const EncodeTiled f = encode_tiled();
    if (!f) return fail(SPEC_ERR_CUDA, "the driver has no cuTensorMapEncodeTiled");
    const cuuint32_t each[4] = {1, 1, 1, 1};
    const CUresult r = f(map, type, rank, const_cast<void *>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPEC_OK : fail(SPEC_ERR_CUDA, "cuTensorMapEncodeTiled: error %d", (int)r);
}

// The cache's keys or values [pages][kv_heads * page_size][D] in boxes of up to 128 rows of a page: 16-bit ones in
// halves of 64 columns, swizzled as the products take them; 8-bit ones whole, to be widened.
template <int D, bool Q8>
spec_status cache_map(CUtensorMap *map, const AttentionArgs &a, int i, CUtensorMapDataType type) {
    const cuuint64_t rows = static_cast<cuuint64_t>(a.cache.kv_heads) << a.cache.page_bits, row = D * (Q8 ? 1 : 2);
    const cuuint64_t dims[3] = {D, rows, static_cast<cuuint64_t>(std::max(a.cache.pages, 1))}, strides[2] = {row, rows * row};
    const cuuint32_t box[3] = {Q8 ? D : 64, static_cast<cuuint32_t>(std::min(1 << a.cache.page_bits, kTile)), 1};
    // (a cache without pages is not read: any address does)
    return encode(map, Q8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type, 3, a.cache.pages ? a.cache.data[i] : a.out, dims, strides, box, !Q8);
}

// [batch][nodes][heads][D] in boxes of `heads` heads of `nodes` nodes, 64 columns, swizzled; the batch's nodes on one
// axis where `merged`.
inline spec_status nodes_map(CUtensorMap *map, const AttentionArgs &a, const void *base, int D, int heads, const long long *stride, bool merged, int box_heads,
                             int box_nodes, CUtensorMapDataType type) {
    const cuuint64_t B = a.B, N = a.N, token = stride[1] * 2, batch = merged ? token : stride[0] * 2;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), merged ? B * N : N, merged ? 1 : B};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, token, batch};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_nodes), 1};
    return encode(map, type, 4, base, dims, strides, box, true);
}

template <typename T, int D, bool Q8>
spec_status launch_attention(const AttentionArgs &a0, cudaStream_t stream) {
    DeviceInfo di;
    int dev = 0;
    spec_status st = device_info(&di, &dev);
    if (st != SPEC_OK) return st;
    auto kernel = attention_kernel<T, D, Q8>;
    st = allow_max_dyn_smem(dev, reinterpret_cast<const void *>(kernel), &di);
    if (st != SPEC_OK) return st;
    AttentionArgs a = a0;
    a.ctas = std::min(di.sms, kMaxCtas);
#ifdef SPEC_TEST_HOOKS
    a.withhold = test_withhold_unit();
#endif
    // All the shared memory there is, so that one CTA is on an SM: each takes all of its tensor memory.
    a.control = static_cast<int>((di.max_dyn - sizeof(Control)) / 1024 * 1024);
    share_out<D, Q8>(&a, a.control);
    const size_t smem = a.control + sizeof(Control);
    static_assert(sizeof(Control) <= 3 * 1024, "two full halves of queries, four tiles and two 8-bit ones leave no more of 227 KB");
    if (a.ring < 4 || (Q8 && a.stages < 2)) return fail(SPEC_ERR_UNSUPPORTED, "%zu bytes of shared memory a CTA do not do", di.max_dyn);
    const CUtensorMapDataType type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const int kv = a.cache.kv_heads;
    Maps maps;
    if ((st = cache_map<D, Q8>(&maps.k, a, 0, type)) != SPEC_OK || (st = cache_map<D, Q8>(&maps.v, a, 1, type)) != SPEC_OK ||
        (st = nodes_map(&maps.q, a, a.q, D, a.heads, a.stride, a.q_merged, a.group, a.q_nodes, type)) != SPEC_OK ||
        (st = nodes_map(&maps.k_nodes, a, a.k, D, kv, a.stride + 2, false, 1, kTile, type)) != SPEC_OK ||
        (st = nodes_map(&maps.v_nodes, a, a.v, D, kv, a.stride + 4, false, 1, kTile, type)) != SPEC_OK)
        return st;
    kernel<<<a.ctas, Layout<D, Q8>::kThreads, smem, stream>>>(a, maps);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(SPEC_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
    const long long join = static_cast<long long>(a.B) * a.cache.kv_heads * a.blocks * ((a.block_rows + 31) / 32);
    // Few CTAs wait for each piece's loads: 4 pieces at once.  Many hide them behind one another, and then registers count:
    // one at once, four CTAs an SM (3 contexts of 52105, 49 nodes x 4 heads of one key head, 21 CTAs: 68 us with one, 47 with
    // four, 45 with eight; 64 nodes of 16 sequences of 8 key heads, 1024 CTAs: 73 and 77 with one and four).
    if (join <= 2 * di.sms) attention_join_kernel<T, D, 4><<<static_cast<unsigned>(join), 256, 0, stream>>>(a);
    else attention_join_kernel<T, D, 1><<<static_cast<unsigned>(join), 256, 0, stream>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? SPEC_OK : fail(SPEC_ERR_CUDA, "join launch: %s", cudaGetErrorString(e));
}

}  // namespace context
}  // namespace spec
