// distill.cu -- launches of the distillation kernels.
#include "distill.cuh"

namespace spec {
namespace vocab {
namespace {

template <class Kernel>
spec_status go(Kernel kernel, DistillArgs a, int eb, int form, cudaStream_t stream) {
    DeviceInfo di;
    int dev = 0;
    spec_status st = device_info(&di, &dev);
    if (st != SPEC_OK) return st;
    st = allow_max_dyn_smem(dev, reinterpret_cast<const void *>(kernel), &di);
    if (st != SPEC_OK) return st;
    const long long vecs = (static_cast<long long>(a.V) * eb + 14) / 16 + 1;  // at the worst alignment
    const long long most = 48 * 1024;
    long long cs = 1;
    const long long limit = form == kBackward ? 1 << 20 : kMaxCluster;
    while (cs < limit && (vecs + cs - 1) / cs * 16 > most) cs *= 2;
    while (cs < kMaxCluster && a.N * cs < 2 * di.sms && vecs / cs > 2 * kDThreads) cs *= 2;
    a.cluster = static_cast<int>(cs);
    a.part = static_cast<int>((vecs + cs - 1) / cs);
    const size_t row = form == kLossGrad ? static_cast<size_t>(a.part) * 16 : 0;
    const size_t bits = form == kLoss ? 0 : (static_cast<size_t>(a.part) * (16 / eb) + 31) / 32 * 4;
    const size_t smem = sizeof(DistillShared) + row + bits;
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail(SPEC_ERR_CUDA, "distillation launch (N=%d, cluster=%lld, smem=%zu): %s", a.N, cs, smem, cudaGetErrorString(e));
    return SPEC_OK;
}

}  // namespace

spec_status launch_distill(DistillArgs a, int eb, int form, cudaStream_t stream) {
    switch (form) {
        case kLoss: return eb == 4 ? go(distill_kernel<4, false>, a, eb, form, stream) : go(distill_kernel<2, false>, a, eb, form, stream);
        case kLossGrad: return eb == 4 ? go(distill_kernel<4, true>, a, eb, form, stream) : go(distill_kernel<2, true>, a, eb, form, stream);
        default: return eb == 4 ? go(distill_backward_kernel<4>, a, eb, form, stream) : go(distill_backward_kernel<2>, a, eb, form, stream);
    }
}

}  // namespace vocab
}  // namespace spec
