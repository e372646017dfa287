// attention.h -- the parameter block of the attention and its launchers.
#pragma once

#include "context.h"

namespace spec {
namespace context {

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
};

template <typename T, int D, bool Q8>
spec_status launch_attention(const AttentionArgs &a, cudaStream_t stream);

}  // namespace context
}  // namespace spec
