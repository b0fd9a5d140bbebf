// tq_ragged_64.cu -- the ragged attention kernels (tq_ragged_mma.cuh) of head dimension 64.
#include "tq_ragged_mma.cuh"

namespace tq {
namespace ragged {
TQ_RAGGED_DIM(64)
}  // namespace ragged
}  // namespace tq
