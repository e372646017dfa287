// distill_bf16.cu -- the distillation kernels on bf16 logits.
#include "distill.cuh"

namespace spec {
namespace vocab {
template spec_status launch_distill<2>(const DistillArgs &, int, cudaStream_t);
}  // namespace vocab
}  // namespace spec
