// The row passes on a float32 stream with float32 branches.
#include "row_bwd.cuh"
#include "row_fwd.cuh"

namespace spade {
template cudaError_t row_fwd<float, float>(const RowArgs&, cudaStream_t);
template cudaError_t row_bwd<float, float>(const RowArgs&, int, bool, cudaStream_t);
}  // namespace spade
