// tq_ragged_256.cu -- the ragged attention kernels (tq_ragged_mma.cuh) of head dimension 256.
#include "tq_ragged_mma.cuh"

namespace tq {
namespace ragged {
TQ_RAGGED_DIM(256)
}  // namespace ragged
}  // namespace tq
