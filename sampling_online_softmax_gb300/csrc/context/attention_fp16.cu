// attention_fp16.cu -- the attention of fp16 queries.
#include "attention_launch.cuh"

namespace spec {
namespace context {
template spec_status launch_attention<__half, 64, false>(const AttentionArgs &, cudaStream_t);
template spec_status launch_attention<__half, 64, true>(const AttentionArgs &, cudaStream_t);
template spec_status launch_attention<__half, 128, false>(const AttentionArgs &, cudaStream_t);
template spec_status launch_attention<__half, 128, true>(const AttentionArgs &, cudaStream_t);
}  // namespace context
}  // namespace spec
