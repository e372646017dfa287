// adjust.cu -- host side of spec_adjust_logits: argument checks, the split into CTAs, the launch.
#include <algorithm>
#include <climits>

#include "adjust.cuh"

namespace spec {

extern thread_local char g_last_error[512];

namespace vocab {
namespace {

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

template <int EB, bool VEC, bool INPLACE>
spec_status launch_adjust(AdjustArgs a, cudaStream_t stream) {
    DeviceInfo di;
    int dev = 0;
    spec_status st = device_info(&di, &dev);
    if (st != SPEC_OK) return st;
    auto kernel = adjust_kernel<EB, VEC, INPLACE>;
    st = allow_max_dyn_smem(dev, reinterpret_cast<const void *>(kernel), &di);
    if (st != SPEC_OK) return st;
    // Each CTA reads its sequence's whole history, so slices are long and a CTA takes all rows of its
    // sequence, unless that leaves CTAs fewer than are resident at once: then fewer rows, and then shorter slices.
    // The longest are halved also where there would be fewer than two rounds of CTAs (64 x 5 rows of 128256 bf16: 1024 CTAs
    // of 8192 tokens take 77 us, 2048 of 4096 71); shorter ones are not (16 x 5 rows: 1024 CTAs of 4096 tokens 21 us, 2048 of 2048 29).
    const long long resident = kAdjustResident * static_cast<long long>(di.sms);
    const auto slices = [&](int n) { return (a.V + n - 1) / n; };
    a.slice = kMaxSlice;
    a.slices = slices(a.slice);
    const int most = (a.N + kAdjustRows - 1) / kAdjustRows;  // groups of rows
    a.groups = static_cast<int>(std::min<long long>(most, std::max<long long>(1, resident / (static_cast<long long>(a.B) * a.slices))));
    a.rows = (a.N + a.groups - 1) / a.groups;
    a.groups = (a.N + a.rows - 1) / a.rows;
    while (a.slice > kMinSlice && static_cast<long long>(a.B) * a.groups * a.slices < (a.slice == kMaxSlice ? 2 : 1) * resident)
        a.slice /= 2, a.slices = slices(a.slice);
    const long long per_row = static_cast<long long>(a.B) * a.slices;
    if (per_row * a.groups > INT_MAX) return fail(SPEC_ERR_UNSUPPORTED, "too many rows (B=%d, N=%d, V=%d)", a.B, a.N, a.V);
    const size_t smem = 4 * static_cast<size_t>(AdjustShared(a).words);
    kernel<<<static_cast<unsigned>(per_row * a.groups), kAdjustThreads, smem, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPEC_OK : fail(SPEC_ERR_CUDA, "adjust launch: %s", cudaGetErrorString(e));
}

template <int EB>
spec_status dispatch(const AdjustArgs &a, cudaStream_t stream) {
    if (a.out == a.in) return launch_adjust<EB, true, true>(a, stream);
    // 16-byte vectors where logits and output lie alike on the 16-byte grid; tokens one by one elsewhere
    const bool alike = reinterpret_cast<uintptr_t>(a.in) % 16 == reinterpret_cast<uintptr_t>(a.out) % 16;
    return alike ? launch_adjust<EB, true, false>(a, stream) : launch_adjust<EB, false, false>(a, stream);
}

}  // namespace
}  // namespace vocab
}  // namespace spec

using namespace spec;
using namespace spec::vocab;

extern "C" spec_status spec_adjust_logits(const void *logits, spec_dtype dtype, int B, int N, int V, const int32_t *tokens, int L,
                                          const int32_t *prompt_len, const int32_t *total_len, const int32_t *node_tokens,
                                          const uint32_t *mask, const float *repetition, const float *frequency,
                                          const float *presence, const int32_t *bias_ids, const float *bias, int M,
                                          const uint32_t *allowed, void *out, uint32_t *dev_status, void *stream) try {
    g_last_error[0] = '\0';
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return fail(SPEC_ERR_INVALID_ARG, "logits of dtype %d", (int)dtype);
    if (B < 0 || N < 1 || V < 1 || L < 0 || M < 0) return fail(SPEC_ERR_INVALID_ARG, "need B >= 0, N >= 1, V >= 1, L >= 0, M >= 0");
    if (N > SPEC_MAX_NODES) return fail(SPEC_ERR_UNSUPPORTED, "N = %d > %d", N, SPEC_MAX_NODES);
    if (M > SPEC_MAX_BIASES) return fail(SPEC_ERR_UNSUPPORTED, "M = %d > %d", M, SPEC_MAX_BIASES);
    if (L >= 1 << 24) return fail(SPEC_ERR_UNSUPPORTED, "L = %d: histories shorter than 2^24", L);
    const int eb = dtype == SPEC_F32 ? 4 : 2;
    if (V > SPEC_MAX_ROW_BYTES / eb) return fail(SPEC_ERR_UNSUPPORTED, "V = %d: rows of at most %d bytes", V, SPEC_MAX_ROW_BYTES);
    if (B == 0) return SPEC_OK;
    if (!logits || !out || !dev_status || (L && !tokens) || (M && (!bias_ids || !bias)))
        return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(logits, eb) || !aligned(out, eb)) return fail(SPEC_ERR_INVALID_ARG, "logits or out misaligned");
    for (const void *p : {static_cast<const void *>(tokens), static_cast<const void *>(prompt_len), static_cast<const void *>(total_len),
                          static_cast<const void *>(node_tokens), static_cast<const void *>(mask), static_cast<const void *>(repetition),
                          static_cast<const void *>(frequency), static_cast<const void *>(presence), static_cast<const void *>(bias_ids),
                          static_cast<const void *>(bias), static_cast<const void *>(allowed), static_cast<const void *>(dev_status)})
        if (!aligned(p, 4)) return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    AdjustArgs a = {};
    a.in = static_cast<const unsigned char *>(logits);
    a.out = static_cast<unsigned char *>(out);
    const size_t bytes = static_cast<size_t>(B) * N * V * eb;
    const uintptr_t x = reinterpret_cast<uintptr_t>(logits), y = reinterpret_cast<uintptr_t>(out);
    if (x != y && (x > y ? x - y : y - x) < bytes) return fail(SPEC_ERR_INVALID_ARG, "out overlaps logits in part");
    a.B = B, a.N = N, a.V = V, a.L = L, a.M = M;
    a.tokens = tokens, a.prompt_len = prompt_len, a.total_len = total_len, a.nodes = node_tokens;
    a.mask = mask;
    a.repetition = repetition, a.frequency = frequency, a.presence = presence;
    a.bias_ids = bias_ids, a.bias = bias;
    a.allowed = allowed;
    a.status = dev_status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return eb == 4 ? dispatch<4>(a, s) : dispatch<2>(a, s);
} catch (...) {  // (no exception leaves the C ABI)
    return fail(SPEC_ERR_CUDA, "spec_adjust_logits: a host allocation failed");
}
