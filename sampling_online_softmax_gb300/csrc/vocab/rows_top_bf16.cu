// rows_top_bf16.cu -- row_kernel<2, kTopRows>.
#include "row_kernels.cuh"

namespace spec {
namespace vocab {
template spec_status launch_rows<2, kTopRows>(const RowArgs &, cudaStream_t);
}  // namespace vocab
}  // namespace spec
