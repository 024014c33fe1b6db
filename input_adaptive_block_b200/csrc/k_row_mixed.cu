// The row passes on a float32 stream with bfloat16 branches.
#include "row_bwd.cuh"
#include "row_fwd.cuh"

namespace spade {
template cudaError_t row_fwd<float, rowio::bf16>(const RowArgs&, cudaStream_t);
template cudaError_t row_bwd<float, rowio::bf16>(const RowArgs&, int, bool, cudaStream_t);
}  // namespace spade
