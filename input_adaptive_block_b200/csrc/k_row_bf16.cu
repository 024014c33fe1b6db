// The row passes on a bfloat16 stream.
#include "row_bwd.cuh"
#include "row_fwd.cuh"

namespace spade {
template cudaError_t row_fwd<rowio::bf16, rowio::bf16>(const RowArgs&, cudaStream_t);
template cudaError_t row_bwd<rowio::bf16, rowio::bf16>(const RowArgs&, int, bool, cudaStream_t);
}  // namespace spade
