// rows_top_f32.cu -- row_kernel<4, kTopRows>.
#include "row_kernels.cuh"

namespace spec {
namespace vocab {
template spec_status launch_rows<4, kTopRows>(const RowArgs &, cudaStream_t);
}  // namespace vocab
}  // namespace spec
