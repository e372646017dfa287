// context.cu -- host side of the operators on the paged cache (spec_cache_append, spec_cache_read,
// spec_tree_attention): argument checks and dispatch.
#include <algorithm>
#include <climits>
#include <cmath>

#include "attention.h"
#include "cache.cuh"

namespace spec {

extern thread_local char g_last_error[512];

namespace context {

EncodeTiled encode_tiled() {
    static const EncodeTiled f = []() -> EncodeTiled {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

namespace {

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The checks that every call on a cache shares; `dtype` is the keys' and values' own.
spec_status cache_args(CacheView *v, const spec_cache *c, spec_dtype dtype, int B) {
    if (dtype != SPEC_BF16 && dtype != SPEC_F16) return fail(SPEC_ERR_INVALID_ARG, "keys and values of dtype %d", (int)dtype);
    if (!c) return fail(SPEC_ERR_INVALID_ARG, "cache is null");
    if (c->dtype != dtype && c->dtype != SPEC_E4M3) return fail(SPEC_ERR_INVALID_ARG, "a cache of dtype %d", (int)c->dtype);
    if (c->pages < 0 || c->kv_heads < 1 || c->table_width < 0) return fail(SPEC_ERR_INVALID_ARG, "need pages >= 0, kv_heads >= 1, table_width >= 0");
    if (c->head_dim != 64 && c->head_dim != 128) return fail(SPEC_ERR_UNSUPPORTED, "head_dim = %d: 64 or 128", c->head_dim);
    int bits = 4;
    while (bits < 8 && 1 << bits != c->page_size) ++bits;
    if (1 << bits != c->page_size) return fail(SPEC_ERR_UNSUPPORTED, "page_size = %d: 16, 32, 64, 128 or 256", c->page_size);
    if (c->table_width > 1 << (30 - bits)) return fail(SPEC_ERR_UNSUPPORTED, "table_width = %d: positions below 2^30", c->table_width);
    if (c->kv_heads > 1024) return fail(SPEC_ERR_UNSUPPORTED, "kv_heads = %d > 1024", c->kv_heads);
    if (B > 0 && c->pages && (!c->k || !c->v)) return fail(SPEC_ERR_INVALID_ARG, "the cache's k or v is null");
    if (B > 0 && c->table_width && !c->page_table) return fail(SPEC_ERR_INVALID_ARG, "page_table is null");
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4)) return fail(SPEC_ERR_INVALID_ARG, "the cache is misaligned");
    if (B > 0 && c->dtype == SPEC_E4M3 && c->pages && (!c->k_scale || !c->v_scale)) return fail(SPEC_ERR_INVALID_ARG, "an e4m3 cache needs k_scale and v_scale");
    *v = CacheView{{static_cast<unsigned char *>(c->k), static_cast<unsigned char *>(c->v)}, {c->k_scale, c->v_scale},
                   c->page_table, c->pages, bits, c->kv_heads, c->table_width};
    return SPEC_OK;
}

// Strides in elements of `n` tensors (batch, token), contiguous where `given` is null.  An axis of one entry takes the
// other's: its own says nothing (one token of each sequence is then evenly spaced, wherever the sequences lie).
spec_status strides_of(long long *to, const long long *given, int n, int B, long long N, const long long *token) {
    for (int i = 0; i < n; ++i) {
        to[2 * i] = given ? given[2 * i] : N * token[i];
        to[2 * i + 1] = given ? given[2 * i + 1] : token[i];
        if (N == 1) to[2 * i + 1] = B == 1 ? token[i] : to[2 * i];
        if (B == 1) to[2 * i] = to[2 * i + 1];
        if (to[2 * i] % 8 || to[2 * i + 1] % 8 || to[2 * i] < 0 || to[2 * i + 1] < 0)
            return fail(SPEC_ERR_INVALID_ARG, "strides must be multiples of 8 elements, and not negative");
    }
    return SPEC_OK;
}

enum CacheOp { kAppend, kRead };

template <typename T, int D, bool Q8>
spec_status launch_cache(CacheOp op, const CacheRowsArgs &a, cudaStream_t stream) {
    DeviceInfo di;
    int dev = 0;
    spec_status st = device_info(&di, &dev);
    if (st != SPEC_OK) return st;
    const int lanes = op == kRead && Q8 ? D / 16 : D / 8, tokens = std::max(1, kCacheThreads / (a.cache.kv_heads * lanes));
    const long long all = (static_cast<long long>(a.B) * a.S + tokens - 1) / tokens, resident = 8ll * di.sms;  // CTAs' worth; CTAs at once
    // One token under way a thread as long as the CTAs for that are all resident (384 accepted tokens of 8 heads of 128, append and
    // read: 6.3 us against 7.7 with two), two beyond (39950 tokens: 114 us against 118 with one).
    if (all <= resident) {
        if (op == kAppend) cache_append_kernel<T, D, Q8, 1><<<static_cast<unsigned>(all), kCacheThreads, 0, stream>>>(a);
        else cache_read_kernel<T, D, Q8, 1><<<static_cast<unsigned>(all), kCacheThreads, 0, stream>>>(a);
    } else {
        const unsigned grid = static_cast<unsigned>(std::min<long long>((all + 1) / 2, resident));
        if (op == kAppend) cache_append_kernel<T, D, Q8, 2><<<grid, kCacheThreads, 0, stream>>>(a);
        else cache_read_kernel<T, D, Q8, 2><<<grid, kCacheThreads, 0, stream>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPEC_OK : fail(SPEC_ERR_CUDA, "cache launch: %s", cudaGetErrorString(e));
}

template <typename T>
spec_status dispatch_cache(CacheOp op, const CacheRowsArgs &a, int D, bool q8, cudaStream_t s) {
    if (D == 64) return q8 ? launch_cache<T, 64, true>(op, a, s) : launch_cache<T, 64, false>(op, a, s);
    return q8 ? launch_cache<T, 128, true>(op, a, s) : launch_cache<T, 128, false>(op, a, s);
}

// The workspace: tiles before each sequence, then the partial sums (see AttentionArgs), each part on 16 bytes.
size_t attention_layout(AttentionArgs *a, int B, int N, int heads, int D, int shared_len, unsigned char *base) {
    size_t at = 0;
    const auto part = [&](size_t bytes) {
        unsigned char *p = base + at;
        at += (bytes + 15) / 16 * 16;
        return p;
    };
    const size_t cut = static_cast<size_t>(kMaxCtas) * 2 * kBlockRows, rows = shared_len ? 2 * static_cast<size_t>(B) * N * heads : 0;
    unsigned char *p[5] = {part(4 * (static_cast<size_t>(B) + 1)), part(cut * D * 4), part(cut * 8), part(rows * D * 4), part(rows * 8)};
    if (a) {
        a->starts = reinterpret_cast<int32_t *>(p[0]);
        a->cut_sums = reinterpret_cast<float *>(p[1]);
        a->cut_stats = reinterpret_cast<float2 *>(p[2]);
        a->row_sums = reinterpret_cast<float *>(p[3]);
        a->row_stats = reinterpret_cast<float2 *>(p[4]);
    }
    return at;
}

template <typename T>
spec_status dispatch_attention(const AttentionArgs &a, int D, bool q8, cudaStream_t s) {
    if (D == 64) return q8 ? launch_attention<T, 64, true>(a, s) : launch_attention<T, 64, false>(a, s);
    return q8 ? launch_attention<T, 128, true>(a, s) : launch_attention<T, 128, false>(a, s);
}

}  // namespace
}  // namespace context
}  // namespace spec

using namespace spec;
using namespace spec::context;

extern "C" spec_status spec_cache_append(const void *k, const void *v, spec_dtype dtype, int B, int N, const long long *strides,
                                         const int32_t *select, int S, const int32_t *start, const int32_t *count,
                                         const spec_cache *cache, uint32_t *dev_status, void *stream) try {
    g_last_error[0] = '\0';
    CacheRowsArgs a = {};
    spec_status st = cache_args(&a.cache, cache, dtype, B);
    if (st != SPEC_OK) return st;
    if (B < 0 || N < 0 || S < 0 || (!select && S != N)) return fail(SPEC_ERR_INVALID_ARG, "need B >= 0, N >= 0, S >= 0, and S == N without select");
    if (B == 0 || S == 0) return SPEC_OK;
    if (static_cast<long long>(B) * S > INT_MAX / 64) return fail(SPEC_ERR_UNSUPPORTED, "too many rows (B=%d, S=%d)", B, S);
    if ((N && (!k || !v)) || !start || !dev_status) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(SPEC_ERR_INVALID_ARG, "k or v misaligned (16 bytes)");
    if (!aligned(select, 4) || !aligned(start, 4) || !aligned(count, 4) || !aligned(dev_status, 4))
        return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    const long long token = static_cast<long long>(cache->kv_heads) * cache->head_dim, tokens[2] = {token, token};
    long long to[4];
    st = strides_of(to, strides, 2, B, N, tokens);
    if (st != SPEC_OK) return st;
    for (int i = 0; i < 2; ++i) a.batch_stride[i] = to[2 * i], a.token_stride[i] = to[2 * i + 1];
    a.src[0] = static_cast<const unsigned char *>(k);
    a.src[1] = static_cast<const unsigned char *>(v);
    a.select = select, a.start = start, a.count = count;
    a.B = B, a.N = N, a.S = S;
    a.status = dev_status;
    const bool q8 = cache->dtype == SPEC_E4M3;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_BF16 ? dispatch_cache<__nv_bfloat16>(kAppend, a, cache->head_dim, q8, s)
                              : dispatch_cache<__half>(kAppend, a, cache->head_dim, q8, s);
} catch (...) {  // (no exception leaves the C ABI)
    return fail(SPEC_ERR_CUDA, "spec_cache_append: a host allocation failed");
}

extern "C" spec_status spec_cache_read(const spec_cache *cache, int B, int S, const int32_t *start, const int32_t *count, void *k,
                                       void *v, spec_dtype dtype, uint32_t *dev_status, void *stream) try {
    g_last_error[0] = '\0';
    CacheRowsArgs a = {};
    spec_status st = cache_args(&a.cache, cache, dtype, B);
    if (st != SPEC_OK) return st;
    if (B < 0 || S < 0) return fail(SPEC_ERR_INVALID_ARG, "need B >= 0, S >= 0");
    if (B == 0 || S == 0) return SPEC_OK;
    if (static_cast<long long>(B) * S > INT_MAX / 64) return fail(SPEC_ERR_UNSUPPORTED, "too many rows (B=%d, S=%d)", B, S);
    if (!k || !v || !start || !dev_status) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(SPEC_ERR_INVALID_ARG, "k or v misaligned (16 bytes)");
    if (!aligned(start, 4) || !aligned(count, 4) || !aligned(dev_status, 4)) return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    a.dst[0] = static_cast<unsigned char *>(k);
    a.dst[1] = static_cast<unsigned char *>(v);
    a.start = start, a.count = count;
    a.B = B, a.S = S;
    a.status = dev_status;
    const bool q8 = cache->dtype == SPEC_E4M3;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_BF16 ? dispatch_cache<__nv_bfloat16>(kRead, a, cache->head_dim, q8, s)
                              : dispatch_cache<__half>(kRead, a, cache->head_dim, q8, s);
} catch (...) {
    return fail(SPEC_ERR_CUDA, "spec_cache_read: a host allocation failed");
}

extern "C" size_t spec_workspace_bytes_attention(int B, int N, int heads, int kv_heads, int head_dim, int shared_len) {
    if (B <= 0 || N < 1 || N > SPEC_MAX_NODES || kv_heads < 1 || heads < 1 || heads % kv_heads || (head_dim != 64 && head_dim != 128) || shared_len < 0)
        return 0;
    return attention_layout(nullptr, B, N, heads, head_dim, shared_len, nullptr);
}

extern "C" spec_status spec_tree_attention(const void *q, const void *k, const void *v, spec_dtype dtype, int B, int N, int heads,
                                           const long long *strides, const spec_cache *cache, const int32_t *context_lens,
                                           int shared_len, const uint32_t *mask, float scale, void *out, float *lse,
                                           uint32_t *dev_status, void *workspace, size_t workspace_bytes, void *stream) try {
    g_last_error[0] = '\0';
    AttentionArgs a = {};
    spec_status st = cache_args(&a.cache, cache, dtype, B);
    if (st != SPEC_OK) return st;
    const int kv = cache->kv_heads, D = cache->head_dim;
    if (B < 0 || N < 1 || heads < 1 || heads % kv) return fail(SPEC_ERR_INVALID_ARG, "need B >= 0, N >= 1, heads a multiple of kv_heads");
    if (N > SPEC_MAX_NODES) return fail(SPEC_ERR_UNSUPPORTED, "N = %d > %d", N, SPEC_MAX_NODES);
    if (heads / kv > kTile) return fail(SPEC_ERR_UNSUPPORTED, "%d query heads a key head: at most %d", heads / kv, kTile);
    if (shared_len < 0 || shared_len > cache->table_width * cache->page_size || (shared_len && !cache->pages))
        return fail(SPEC_ERR_INVALID_ARG, "shared_len = %d: within the page table", shared_len);
    if (!(scale > 0.0f && scale < INFINITY)) return fail(SPEC_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (B == 0) return SPEC_OK;
    if (static_cast<long long>(B) * N * heads > INT_MAX / 2) return fail(SPEC_ERR_UNSUPPORTED, "too many rows (B=%d, N=%d, heads=%d)", B, N, heads);
    if (!q || !k || !v || !context_lens || !out || !dev_status) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16))
        return fail(SPEC_ERR_INVALID_ARG, "q, k, v or out misaligned (16 bytes)");
    if (!aligned(context_lens, 4) || !aligned(mask, 4) || !aligned(lse, 4) || !aligned(dev_status, 4))
        return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    const size_t need = spec_workspace_bytes_attention(B, N, heads, kv, D, shared_len);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need)
        return fail(SPEC_ERR_WORKSPACE, "workspace of %zu bytes, 16-byte aligned, needed (got %zu)", need, workspace_bytes);
    const long long tokens[3] = {static_cast<long long>(heads) * D, static_cast<long long>(kv) * D, static_cast<long long>(kv) * D};
    st = strides_of(a.stride, strides, 3, B, N, tokens);
    if (st != SPEC_OK) return st;
    for (const long long x : a.stride)
        if (x == 0 || x >= 1ll << 38) return fail(SPEC_ERR_INVALID_ARG, "strides must be above 0 and below 2^38 elements");
    const void *in[3] = {q, k, v};
    for (int i = 0; i < 3; ++i) {  // the results go out while other CTAs still read
        const uintptr_t at = reinterpret_cast<uintptr_t>(in[i]), to = reinterpret_cast<uintptr_t>(out);
        const uintptr_t bytes = 2 * static_cast<uintptr_t>((B - 1) * a.stride[2 * i] + (N - 1) * a.stride[2 * i + 1] + tokens[i]);
        if (at < to + 2 * static_cast<uintptr_t>(B) * N * tokens[0] && to < at + bytes) return fail(SPEC_ERR_INVALID_ARG, "out overlaps q, k or v");
    }
    a.q = static_cast<const unsigned char *>(q);
    a.k = static_cast<const unsigned char *>(k);
    a.v = static_cast<const unsigned char *>(v);
    a.lens = context_lens;
    a.mask = mask;
    a.out = static_cast<unsigned char *>(out);
    a.lse = lse;
    a.status = dev_status;
    a.B = B, a.N = N, a.heads = heads, a.shared_len = shared_len;
    a.scale = scale;
    if (a.cache.pages == 0) a.cache.table_width = 0;  // no position is there
    attention_layout(&a, B, N, heads, D, shared_len, static_cast<unsigned char *>(workspace));
    // Blocks of two halves of up to 128 rows, whole nodes each, as equal as they can be.
    a.group = heads / kv;
    a.half_nodes = kTile / a.group;
    const auto split = [&](int nodes, int *blocks, int *block_rows) {
        *blocks = (nodes + 2 * a.half_nodes - 1) / (2 * a.half_nodes);
        const int each = (nodes + *blocks - 1) / *blocks;
        *block_rows = each * a.group;
        a.q_nodes = std::max(a.q_nodes, std::min(each, a.half_nodes));
    };
    split(N, &a.blocks, &a.block_rows);
    split(shared_len ? B * N : N, &a.shared_blocks, &a.shared_rows);
    a.q_merged = B == 1 || a.stride[0] == N * a.stride[1];
    if (shared_len && !a.q_merged) return fail(SPEC_ERR_UNSUPPORTED, "with shared_len, q's batch stride is N times its token stride");
    const long long tiles = static_cast<long long>(kv) * (static_cast<long long>(B) * a.blocks * (tiles_of(cache->table_width * cache->page_size) + tiles_of(N)) +
                                                          static_cast<long long>(a.shared_blocks) * tiles_of(shared_len));
    if (tiles > INT_MAX) return fail(SPEC_ERR_UNSUPPORTED, "too much work: %lld tiles of %d keys", tiles, kTile);
    const bool q8 = cache->dtype == SPEC_E4M3;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_BF16 ? dispatch_attention<__nv_bfloat16>(a, D, q8, s) : dispatch_attention<__half>(a, D, q8, s);
} catch (...) {
    return fail(SPEC_ERR_CUDA, "spec_tree_attention: a host allocation failed");
}
