// rows_sample_f32.cu -- row_kernel<4, kSampleRows>.
#include "row_kernels.cuh"

namespace spec {
namespace vocab {
template spec_status launch_rows<4, kSampleRows>(const RowArgs &, cudaStream_t);
}  // namespace vocab
}  // namespace spec
