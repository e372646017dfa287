// attention_launch.cuh -- the launcher of the attention, instantiated one element type a unit.
#pragma once

#include <climits>

#include "attention.cuh"

namespace spec {
namespace context {

template <typename T, int D, bool Q8>
spec_status launch_attention(const AttentionArgs &a, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.B) * a.N * a.heads;
    attention_kernel<T, D, Q8><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SPEC_OK : fail(SPEC_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
}

}  // namespace context
}  // namespace spec
