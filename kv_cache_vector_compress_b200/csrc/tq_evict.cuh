// tq_evict.cuh -- the eviction call as its kernels take it.
#pragma once

#include "tq_internal.cuh"

namespace tq {

constexpr int kEvictArrays = 7;  // key codes, signs, key norms, residual norms, value codes, value norms, weights

struct EvictCall {
    const void *src[kEvictArrays];
    void *dst[kEvictArrays];
    int bytes[kEvictArrays];  // of one record in each array
    int B, Hkv;
    const int32_t *lens;
    int64_t t_cap, budget, recent, out_cap;
    int32_t *kept, *out_lens;
    int32_t *counts;  // scratch: tokens kept of each slice
    int32_t *dev_status;
};

constexpr int kCopySlots = 256;  // destination slots a CTA copies
inline int64_t evict_chunks(int64_t budget) { return (budget + kCopySlots - 1) / kCopySlots; }
inline size_t evict_scratch_bytes(int B, int Hkv) { return align_up(sizeof(int32_t) * (size_t)B * Hkv, 256); }
cudaError_t launch_evict(const EvictCall &c, cudaStream_t s);

}  // namespace tq
