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
#include "tq_launch.cuh"

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

// This warp's exclusive prefix of the warps' sums, and their total.
__device__ __forceinline__ uint32_t before_warp(const uint32_t *wsum, int warp, int lane, uint32_t *all) {
    const uint32_t v = wsum[lane];
    uint32_t s = v;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, s, o);
        if (lane >= o) s += y;
    }
    *all = __shfl_sync(kFull, s, 31);
    return __shfl_sync(kFull, s - v, warp);
}

// One CTA per slice; a thread holds up to KPT keys in registers, loaded at once, so that the slice is
// read once while it has at most KPT x 1024 tokens (longer ones in rounds, read again from L2 by each
// step).  Three histograms in shared memory find the threshold; then every warp's counts of each group of 32
// keys are scanned together, which gives each key its place.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictCall c) {
    constexpr int ROUND = KPT * kSelThreads;
    grid_go();
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t cnt[KPT * kSelWarps];  // [group of a round][warp]: keys above | keys equal << 16
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
    const int rounds = (n - 1) / ROUND + 1;
    uint32_t key[KPT];
    auto load = [&](int round) {
        const int t0 = round * ROUND + tid;
        float v[KPT];
#pragma unroll
        for (int i = 0; i < KPT; ++i) v[i] = t0 + i * kSelThreads < n ? w[t0 + i * kSelThreads] : 0.f;
#pragma unroll
        for (int i = 0; i < KPT; ++i) key[i] = t0 + i * kSelThreads >= safe ? 0xFFFFFFFFu : weight_key(v[i]);
    };
    load(0);
    // the threshold: the keep-th largest key, found 11, 11 and 10 bits at a time
    uint32_t prefix = 0, mask = 0, rank = (uint32_t)keep;  // the rank-th largest of the keys that match
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t dm = pass < 2 ? 2047u : 1023u;
        for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int r = 0; r < rounds; ++r) {
            if (rounds > 1) load(r);
            const int t0 = r * ROUND + tid;
#pragma unroll
            for (int i = 0; i < KPT; ++i)
                if (t0 + i * kSelThreads < n && (key[i] & mask) == prefix) atomicAdd(&hist[(key[i] >> shift) & dm], 1u);
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
        uint32_t all;
        const uint32_t above = x - (h1 + h0) + before_warp(wsum, warp, lane, &all);
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
    }
    // kept: keys above the threshold, and the first `rank` slots whose key equals it
    uint32_t gt_before = 0, eq_before = 0;
    for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) load(r);
        const int t0 = r * ROUND + tid;
        uint32_t gt[KPT], eq[KPT];
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const bool there = t0 + i * kSelThreads < n;
            gt[i] = __ballot_sync(kFull, there && key[i] > prefix);
            eq[i] = __ballot_sync(kFull, there && key[i] == prefix);
            if (lane == 0) cnt[i * kSelWarps + warp] = __popc(gt[i]) | ((uint32_t)__popc(eq[i]) << 16);
        }
        __syncthreads();
        // exclusive prefix sums of the counts in slot order, KPT a thread in the first 32 warps' lanes
        uint32_t all = 0;
        {
            const uint32_t x = tid < KPT * kSelWarps ? cnt[tid] : 0u;
            uint32_t s = x;
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(kFull, s, o);
                if (lane >= o) s += y;
            }
            if (lane == 31) wsum[warp] = s;
            __syncthreads();
            const uint32_t off = before_warp(wsum, warp, lane, &all);
            if (tid < KPT * kSelWarps) cnt[tid] = off + s - x;
        }
        __syncthreads();
        const uint32_t below = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < KPT; ++i) {
            const uint32_t base = cnt[i * kSelWarps + warp];
            const uint32_t ngt = gt_before + (base & 0xFFFFu) + __popc(gt[i] & below);
            const uint32_t neq = eq_before + (base >> 16) + __popc(eq[i] & below);
            if (((gt[i] >> lane) & 1u) || (((eq[i] >> lane) & 1u) && neq < rank))
                kept[ngt + min(neq, rank)] = t0 + i * kSelThreads;
        }
        gt_before += all & 0xFFFFu;
        eq_before += all >> 16;
        __syncthreads();
    }
}

constexpr int kCopyThreads = 256;

// `per` words of type T a record: every thread takes pieces in turn, four loads on their way at once.
template <typename T>
__device__ __forceinline__ void copy_records(const void *src, void *dst, int per, int64_t src0, int64_t dst0,
                                             const int32_t *idx, int cnt, int tid) {
    const T *s = (const T *)src + src0 * per;
    T *o = (T *)dst + dst0 * per;
    const int all = cnt * per;
    for (int e0 = tid; e0 < all; e0 += 4 * kCopyThreads) {
        T v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = e0 + u * kCopyThreads, j = e / per;
            if (e < all) v[u] = s[(int64_t)idx[j] * per + (e - j * per)];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int e = e0 + u * kCopyThreads;
            if (e < all) o[e] = v[u];
        }
    }
}

__device__ __forceinline__ void copy_wide(const EvictCall &c, int a, int64_t src0, int64_t dst0, const int32_t *idx,
                                          int cnt, int tid) {
    const int by = c.bytes[a];
    if (by % 16 == 0) copy_records<uint4>(c.src[a], c.dst[a], by / 16, src0, dst0, idx, cnt, tid);
    else if (by % 8 == 0) copy_records<uint2>(c.src[a], c.dst[a], by / 8, src0, dst0, idx, cnt, tid);
    else copy_records<uint32_t>(c.src[a], c.dst[a], by / 4, src0, dst0, idx, cnt, tid);
}

// kCopySlots kept records of one slice per CTA, a thread a record for the norms and weights, and the
// widest words that every record is aligned to for the packed arrays.  Bound by the bytes moved.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(EvictCall c, int chunks) {
    static_assert(kCopySlots == kCopyThreads, "a thread a record");
    __shared__ int32_t idx[kCopySlots];
    grid_wait();
    const int slice = blockIdx.x / chunks, tid = threadIdx.x;
    const int j0 = (blockIdx.x - slice * chunks) * kCopySlots;
    const int cnt = min(kCopySlots, c.counts[slice] - j0);
    if (cnt <= 0) return;
    const int64_t src0 = (int64_t)slice * c.t_cap, dst0 = (int64_t)slice * c.out_cap + j0;
    if (tid < cnt) {
        const int32_t i = c.kept[(int64_t)slice * c.budget + j0 + tid];
        idx[tid] = i;
        const int64_t s = src0 + i, o = dst0 + tid;
        const uint16_t kn = ((const uint16_t *)c.src[2])[s], kr = ((const uint16_t *)c.src[3])[s];
        const uint16_t vn = ((const uint16_t *)c.src[5])[s];
        const uint32_t wt = ((const uint32_t *)c.src[6])[s];
        ((uint16_t *)c.dst[2])[o] = kn;
        ((uint16_t *)c.dst[3])[o] = kr;
        ((uint16_t *)c.dst[5])[o] = vn;
        ((uint32_t *)c.dst[6])[o] = wt;
    }
    __syncthreads();
    copy_wide(c, 4, src0, dst0, idx, cnt, tid);
    copy_wide(c, 0, src0, dst0, idx, cnt, tid);
    copy_wide(c, 1, src0, dst0, idx, cnt, tid);
}

template <int KPT>
cudaError_t launch_select(const EvictCall &c, cudaStream_t s) {
    evict_select_kernel<KPT><<<(unsigned)(c.B * c.Hkv), kSelThreads, 0, s>>>(c);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictCall &c, cudaStream_t s) {
    // as few keys a thread as hold the longest slice in one round
    const cudaError_t e = c.t_cap <= 2 * kSelThreads    ? launch_select<2>(c, s)
                          : c.t_cap <= 8 * kSelThreads  ? launch_select<8>(c, s)
                          : c.t_cap <= 16 * kSelThreads ? launch_select<16>(c, s)
                                                        : launch_select<32>(c, s);
    if (e != cudaSuccess) return e;
    const int chunks = (int)evict_chunks(c.budget);
    return launch_after(evict_copy_kernel, (unsigned)(chunks * c.B * c.Hkv), kCopyThreads, 0, s, c, chunks);
}

}  // namespace tq
