// vocab.cu -- host side of the operators on rows of logits (spec_sample_filtered,
// spec_top_logits, spec_distill, spec_distill_backward): argument checks and
// dispatch.
#include <climits>
#include <cmath>
#include <map>
#include <mutex>
#include <tuple>

#include "distill.h"

namespace spec {

extern thread_local char g_last_error[512];

namespace vocab {
namespace {

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool valid_dtype(spec_dtype d) { return d == SPEC_F32 || d == SPEC_BF16; }
int elt_bytes(spec_dtype d) { return d == SPEC_F32 ? 4 : 2; }

// The checks the distillation's calls share, and their fields of the parameter block.
spec_status distill_args(DistillArgs *a, const void *student, spec_dtype dtype, int N, int V, const int32_t *ids, const float *top,
                         int K, const float *lse, float T, const float *weight, uint32_t *dev_status) {
    if (!valid_dtype(dtype)) return fail(SPEC_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (N < 0 || V < 1 || K < 1) return fail(SPEC_ERR_INVALID_ARG, "need N >= 0, V >= 1, K >= 1");
    if (K > SPEC_MAX_TOP) return fail(SPEC_ERR_UNSUPPORTED, "K = %d > %d", K, SPEC_MAX_TOP);
    if (!(T >= kMinTemperature && T <= kMaxTemperature)) return fail(SPEC_ERR_INVALID_ARG, "temperature must be in [1e-6, 1e6]");
    a->N = N;
    if (N == 0) return SPEC_OK;
    const int eb = elt_bytes(dtype);
    if (!student || !aligned(student, eb)) return fail(SPEC_ERR_INVALID_ARG, "student logits null or misaligned");
    if (!ids || !top || !dev_status) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(ids, 4) || !aligned(top, 4) || !aligned(lse, 4) || !aligned(weight, 4) || !aligned(dev_status, 4))
        return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    if (V > SPEC_MAX_ROW_BYTES / eb) return fail(SPEC_ERR_UNSUPPORTED, "V = %d: rows of at most %d bytes", V, SPEC_MAX_ROW_BYTES);
    if (N > INT_MAX / 64) return fail(SPEC_ERR_UNSUPPORTED, "N too large");
    a->student = static_cast<const unsigned char *>(student);
    a->student_end = a->student + static_cast<size_t>(N) * static_cast<size_t>(V) * eb;
    a->ids = ids;
    a->top = top;
    a->lse = lse;
    a->weight = weight;
    a->V = V;
    a->K = K;
    a->T = T;
    a->status = dev_status;
    return SPEC_OK;
}

// The gradient lies over the logits each on its own, or beside them: shifted, it would overwrite others unread.
spec_status place_grad(DistillArgs *a, void *grad, spec_dtype dtype) {
    if (!aligned(grad, elt_bytes(dtype))) return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    a->grad = static_cast<unsigned char *>(grad);
    const uintptr_t g = reinterpret_cast<uintptr_t>(grad), s = reinterpret_cast<uintptr_t>(a->student);
    const size_t bytes = static_cast<size_t>(a->student_end - a->student);
    if (grad && g != s && (g > s ? g - s : s - g) < bytes)
        return fail(SPEC_ERR_INVALID_ARG, "grad overlaps student_logits in part");
    return SPEC_OK;
}

// The checks every operator on [B, V] logits shares, and their fields of the parameter block.
spec_status rows_args(RowArgs *a, const void *logits, spec_dtype dtype, int B, int V, uint32_t *dev_status) {
    const int eb = elt_bytes(dtype);
    if (!logits || !aligned(logits, eb)) return fail(SPEC_ERR_INVALID_ARG, "logits null or misaligned");
    if (!dev_status || !aligned(dev_status, 4)) return fail(SPEC_ERR_INVALID_ARG, "dev_status null or misaligned");
    if (V > SPEC_MAX_ROW_BYTES / eb) return fail(SPEC_ERR_UNSUPPORTED, "V = %d: rows of at most %d bytes", V, SPEC_MAX_ROW_BYTES);
    if (B > INT_MAX / kMaxCluster) return fail(SPEC_ERR_UNSUPPORTED, "B too large");
    a->base = static_cast<const unsigned char *>(logits);
    a->end = a->base + static_cast<size_t>(B) * static_cast<size_t>(V) * eb;
    a->B = B;
    a->V = V;
    a->status = dev_status;
    int bits = 1;
    while ((1ll << bits) < V) ++bits;
    a->U = 62 - bits < 48 ? 62 - bits : 48;
    return SPEC_OK;
}

std::mutex g_clusters_mutex;
std::map<std::tuple<int, const void *, size_t, unsigned>, int> g_clusters;

}  // namespace

int resident_clusters(int dev, const void *kernel, const cudaLaunchConfig_t &cfg) try {
    const auto key = std::make_tuple(dev, kernel, cfg.dynamicSmemBytes, cfg.attrs[0].val.clusterDim.x);
    std::lock_guard<std::mutex> lock(g_clusters_mutex);
    const auto it = g_clusters.find(key);
    if (it != g_clusters.end()) return it->second;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    g_clusters[key] = n;
    return n;
} catch (...) {  // (no exception leaves the C ABI)
    return 0;
}

}  // namespace vocab
}  // namespace spec

using namespace spec;
using namespace spec::vocab;

extern "C" spec_status spec_sample_filtered(const void *logits, spec_dtype dtype, int B, int V, const float *temperature,
                                            const int32_t *top_k, const float *top_p, const float *min_p, const float *u,
                                            int32_t *tokens, uint32_t *dev_status, void *stream) {
    g_last_error[0] = '\0';
    if (!valid_dtype(dtype)) return fail(SPEC_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (B < 0 || V < 1) return fail(SPEC_ERR_INVALID_ARG, "need B >= 0, V >= 1");
    if (B == 0) return SPEC_OK;
    RowArgs a = {};
    spec_status st = rows_args(&a, logits, dtype, B, V, dev_status);
    if (st != SPEC_OK) return st;
    if (!temperature || !u || !tokens) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(u, 4) ||
        !aligned(tokens, 4))
        return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.tokens = tokens;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_rows<4, kSampleRows>(a, s) : launch_rows<2, kSampleRows>(a, s);
}

extern "C" spec_status spec_top_logits(const void *logits, spec_dtype dtype, int B, int V, int K, float temperature,
                                       float *values, int32_t *ids, float *lse, uint32_t *dev_status, void *stream) {
    g_last_error[0] = '\0';
    if (!valid_dtype(dtype)) return fail(SPEC_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (B < 0 || V < 1 || K < 1) return fail(SPEC_ERR_INVALID_ARG, "need B >= 0, V >= 1, K >= 1");
    if (K > SPEC_MAX_TOP) return fail(SPEC_ERR_UNSUPPORTED, "K = %d > %d", K, SPEC_MAX_TOP);
    if (!(temperature >= kMinTemperature && temperature <= kMaxTemperature))
        return fail(SPEC_ERR_INVALID_ARG, "temperature must be in [1e-6, 1e6]");
    if (B == 0) return SPEC_OK;
    RowArgs a = {};
    spec_status st = rows_args(&a, logits, dtype, B, V, dev_status);
    if (st != SPEC_OK) return st;
    if (!values || !ids) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(values, 4) || !aligned(ids, 4) || !aligned(lse, 4)) return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    a.K = K;
    a.temp = temperature;
    a.values = values;
    a.ids = ids;
    a.lse = lse;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_rows<4, kTopRows>(a, s) : launch_rows<2, kTopRows>(a, s);
}

extern "C" spec_status spec_distill(const void *student_logits, spec_dtype dtype, int N, int V, const int32_t *top_ids,
                                    const float *top_logits, int K, const float *top_lse, float temperature,
                                    const float *row_weight, float *loss, float *stats, void *grad, uint32_t *dev_status,
                                    void *stream) {
    g_last_error[0] = '\0';
    DistillArgs a = {};
    spec_status st = distill_args(&a, student_logits, dtype, N, V, top_ids, top_logits, K, top_lse, temperature, row_weight, dev_status);
    if (st != SPEC_OK || N == 0) return st;
    if (!loss || !stats) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(loss, 4) || !aligned(stats, 8)) return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    st = place_grad(&a, grad, dtype);
    if (st != SPEC_OK) return st;
    a.loss = loss;
    a.stats = stats;
    const int form = grad ? kLossGrad : kLoss;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_distill<4>(a, form, s) : launch_distill<2>(a, form, s);
}

extern "C" spec_status spec_distill_backward(const void *student_logits, spec_dtype dtype, int N, int V, const int32_t *top_ids,
                                             const float *top_logits, int K, const float *top_lse, float temperature,
                                             const float *row_weight, const float *stats, const float *grad_loss, void *grad,
                                             uint32_t *dev_status, void *stream) {
    g_last_error[0] = '\0';
    DistillArgs a = {};
    spec_status st = distill_args(&a, student_logits, dtype, N, V, top_ids, top_logits, K, top_lse, temperature, row_weight, dev_status);
    if (st != SPEC_OK || N == 0) return st;
    if (!stats || !grad_loss || !grad) return fail(SPEC_ERR_INVALID_ARG, "a pointer is null");
    if (!aligned(stats, 8) || !aligned(grad_loss, 4)) return fail(SPEC_ERR_INVALID_ARG, "a pointer is misaligned");
    st = place_grad(&a, grad, dtype);
    if (st != SPEC_OK) return st;
    a.stats = const_cast<float *>(stats);
    a.grad_loss = grad_loss;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == SPEC_F32 ? launch_distill<4>(a, kBackward, s) : launch_distill<2>(a, kBackward, s);
}
