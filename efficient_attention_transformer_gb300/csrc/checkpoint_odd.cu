// The kernels of checkpoint_rows.cuh over rows that are not whole vectors on their
// boundaries.
#include "checkpoint_rows.cuh"

namespace flashgau {

cudaError_t checkpoint_rows_odd(int what, const CheckpointArgs &a, int dtype, int num_sms,
                                cudaStream_t stream, CheckpointGrid *g) {
  return a.form == kBlocks ? rows<kBlocks>(what, a, dtype, num_sms, stream, g)
                           : rows<kElements>(what, a, dtype, num_sms, stream, g);
}

}  // namespace flashgau
