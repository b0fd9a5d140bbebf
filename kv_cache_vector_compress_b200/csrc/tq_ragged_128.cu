// tq_ragged_128.cu -- the ragged attention kernels (tq_ragged_mma.cuh) of head dimension 128.
#include "tq_ragged_mma.cuh"

namespace tq {
namespace ragged {
TQ_RAGGED_DIM(128)
}  // namespace ragged
}  // namespace tq
