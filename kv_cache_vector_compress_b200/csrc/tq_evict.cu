// tq_evict.cu -- eviction by accumulated attention weight: of every (batch, KV head) slice the
// `budget` heaviest tokens, the last `recent` ones always among them, are copied in their order
// into another cache.
//
// Order of the tokens: a 32-bit key, larger is heavier.  Floats map to integers of the same order
// (the sign bit flipped, or every bit of a negative number); -0 counts as 0; NaN is 0xFFFFFFFE,
// above every number; the last `recent` tokens are 0xFFFFFFFF.  The kept set is the budget largest
// (key, smaller slot first), found by a radix selection: the threshold key's digits from the top,
// each from a histogram of the keys that match the digits before.
#include "tq_common.cuh"
#include "tq_evict.cuh"

namespace tq {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// One CTA per slice.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictCall c) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wsum[kSelWarps];
    __shared__ uint32_t s_digit, s_rank;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = blockIdx.x, b = slice / c.Hkv;
    int64_t len = c.lens[b];
    if (len < 0 || len > c.t_cap) {
        if (tid == 0 && c.dev_status) *c.dev_status = TQ_ERR_INVALID_ARG;
        len = len < 0 ? 0 : c.t_cap;
    }
    const int n = (int)len, budget = (int)c.budget;
    const int keep = n < budget ? n : budget;
    int32_t *kept = c.kept + (int64_t)slice * budget;
    if (tid == 0) {
        c.counts[slice] = keep;
        if (slice == b * c.Hkv) c.out_lens[b] = keep;
    }
    if (n <= budget) {
        for (int t = tid; t < n; t += kSelThreads) kept[t] = t;
        return;
    }
    const float *w = (const float *)c.src[6] + (int64_t)slice * c.t_cap;
    const int safe = n - (int)c.recent;  // slots from here on are kept
    auto key_at = [&](int t) { return t >= safe ? 0xFFFFFFFFu : weight_key(w[t]); };
    // the threshold: the keep-th largest key, found 11, 11 and 10 bits at a time
    uint32_t prefix = 0, mask = 0, rank = (uint32_t)keep;  // the rank-th largest of the keys that match
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t dm = pass < 2 ? 2047u : 1023u;
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int t = tid; t < n; t += kSelThreads) {
            const uint32_t k = key_at(t);
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & dm], 1u);
        }
        __syncthreads();
        // suffix sums over the bins, two a thread, from the top: thread 0 takes the highest two
        const int hi = kBins - 1 - 2 * tid;
        const uint32_t h1 = hist[hi], h0 = hist[hi - 1];
        uint32_t x = h1 + h0;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        uint32_t above = x - (h1 + h0);
        for (int u = 0; u < warp; ++u) above += wsum[u];
        if (above < rank && rank <= above + h1) {
            s_digit = (uint32_t)hi;
            s_rank = rank - above;
        } else if (above + h1 < rank && rank <= above + h1 + h0) {
            s_digit = (uint32_t)hi - 1;
            s_rank = rank - above - h1;
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= dm << shift;
        rank = s_rank;
        __syncthreads();
    }
    // kept: keys above the threshold, and the first `rank` slots whose key equals it
    uint32_t gt_before = 0, eq_before = 0;
    for (int t0 = 0; t0 < n; t0 += kSelThreads) {
        const int t = t0 + tid;
        const uint32_t k = t < n ? key_at(t) : 0u;
        const uint32_t gt = t < n && k > prefix, eq = t < n && k == prefix;
        uint32_t x = gt | (eq << 16);
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        uint32_t off = 0, all = 0;
        for (int u = 0; u < kSelWarps; ++u) {
            const uint32_t v = wsum[u];
            if (u < warp) off += v;
            all += v;
        }
        x += off - (gt | (eq << 16));  // before this thread
        const uint32_t ngt = gt_before + (x & 0xFFFFu), neq = eq_before + (x >> 16);
        if (gt || (eq && neq < rank)) kept[ngt + min(neq, rank)] = t;
        gt_before += all & 0xFFFFu;
        eq_before += all >> 16;
        __syncthreads();
    }
}

constexpr int kCopyThreads = 256;

template <typename T>
__device__ __forceinline__ void copy_records(const void *src, void *dst, int per, int64_t src0, int64_t dst0,
                                             const int32_t *idx, int cnt, int tid) {
    const T *s = (const T *)src;
    T *o = (T *)dst;
    for (int e = tid; e < cnt * per; e += kCopyThreads) {
        const int j = e / per, k = e - j * per;
        o[(dst0 + j) * per + k] = s[(src0 + idx[j]) * per + k];
    }
}

// kCopySlots kept records of one slice per CTA, array by array, in the widest words that every
// record of the array is aligned to.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(EvictCall c, int chunks) {
    __shared__ int32_t idx[kCopySlots];
    const int slice = blockIdx.x / chunks, tid = threadIdx.x;
    const int j0 = (blockIdx.x - slice * chunks) * kCopySlots;
    const int cnt = min(kCopySlots, c.counts[slice] - j0);
    if (cnt <= 0) return;
    if (tid < cnt) idx[tid] = c.kept[(int64_t)slice * c.budget + j0 + tid];
    __syncthreads();
    const int64_t src0 = (int64_t)slice * c.t_cap, dst0 = (int64_t)slice * c.out_cap + j0;
    for (int a = 0; a < kEvictArrays; ++a) {
        const int by = c.bytes[a];
        if (by % 16 == 0) copy_records<uint4>(c.src[a], c.dst[a], by / 16, src0, dst0, idx, cnt, tid);
        else if (by % 8 == 0) copy_records<uint2>(c.src[a], c.dst[a], by / 8, src0, dst0, idx, cnt, tid);
        else if (by % 4 == 0) copy_records<uint32_t>(c.src[a], c.dst[a], by / 4, src0, dst0, idx, cnt, tid);
        else copy_records<uint16_t>(c.src[a], c.dst[a], by / 2, src0, dst0, idx, cnt, tid);
    }
}

}  // namespace

cudaError_t launch_evict(const EvictCall &c, cudaStream_t s) {
    evict_select_kernel<<<(unsigned)(c.B * c.Hkv), kSelThreads, 0, s>>>(c);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int chunks = (int)evict_chunks(c.budget);
    evict_copy_kernel<<<(unsigned)(chunks * c.B * c.Hkv), kCopyThreads, 0, s>>>(c, chunks);
    return cudaGetLastError();
}

}  // namespace tq
