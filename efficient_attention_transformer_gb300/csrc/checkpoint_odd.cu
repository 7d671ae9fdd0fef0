// The kernels of checkpoint_rows.cuh over rows that are not on vectors' boundaries.
#include "checkpoint_rows.cuh"

namespace flashgau {

cudaError_t checkpoint_rows_odd(int what, const CheckpointArgs &a, int dtype,
                                unsigned most_blocks, cudaStream_t stream) {
  return rows<false>(what, a, dtype, most_blocks, stream);
}

}  // namespace flashgau
