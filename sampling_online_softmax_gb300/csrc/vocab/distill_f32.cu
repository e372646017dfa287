// distill_f32.cu -- the distillation kernels on f32 logits.
#include "distill.cuh"

namespace spec {
namespace vocab {
template spec_status launch_distill<4>(const DistillArgs &, int, cudaStream_t);
}  // namespace vocab
}  // namespace spec
