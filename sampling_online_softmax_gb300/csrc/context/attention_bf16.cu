// attention_bf16.cu -- the attention of bf16 queries.
#include "attention_launch.cuh"

namespace spec {
namespace context {
template spec_status launch_attention<__nv_bfloat16, 64, false>(const AttentionArgs &, cudaStream_t);
template spec_status launch_attention<__nv_bfloat16, 64, true>(const AttentionArgs &, cudaStream_t);
template spec_status launch_attention<__nv_bfloat16, 128, false>(const AttentionArgs &, cudaStream_t);
template spec_status launch_attention<__nv_bfloat16, 128, true>(const AttentionArgs &, cudaStream_t);
}  // namespace context
}  // namespace spec
