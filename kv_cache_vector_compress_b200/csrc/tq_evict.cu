// tq_evict.cu -- eviction by accumulated attention weight: of every (batch, KV head) slice the
// `budget` heaviest tokens, the last `recent` ones always among them, are copied in their order
// into another cache.
//
// Order of the tokens: a 32-bit key, larger is heavier.  Floats map to integers of the same order
// (the sign bit flipped, or every bit of a negative number); -0 counts as 0; NaN is 0xFFFFFFFE,
// above every number; the last `recent` tokens are 0xFFFFFFFF.  The kept set is the budget largest
// (key, smaller slot first), found by a radix selection: the threshold key's digits from the top,
// each from a histogram of the keys that match the digits before.
#include <type_traits>

#include "tq_common.cuh"
#include "tq_evict.cuh"
#include "tq_launch.cuh"
#include "tq_serve.cuh"

namespace tq {

namespace {

constexpr int kBins = 2048;
constexpr int kAtOnce = 8;  // weights a thread has on their way at once
constexpr size_t kHeldMax = 200 * 1024;  // bytes of keys that a CTA can hold
constexpr size_t kHeldPair = 96 * 1024;  // ... that two CTAs of an SM can

// (The addition makes -0 a 0 and any NaN the positive one with all other bits set.)
__device__ __forceinline__ uint32_t weight_key(float w) {
    const int32_t u = __float_as_int(w + 0.f);
    return min((uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u), 0xFFFFFFFEu);
}

// One more in a bin of shared memory, if `yes`: one predicated instruction, no branch.
__device__ __forceinline__ void count_if(bool yes, uint32_t *bin) {
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %0, 0;\n\t"
        "@p red.shared.add.u32 [%1], 1; }" ::"r"((uint32_t)yes),
        "r"((uint32_t)__cvta_generic_to_shared(bin))
        : "memory");
}

template <uint32_t N>
using Step = std::integral_constant<uint32_t, N>;

// One CTA per slice, two an SM where the keys leave room.  HELD: the keys wait in shared memory between
// the steps; otherwise each step reads the weights again, mostly from L2.  Three histograms in shared
// memory find the threshold; then every warp takes a run of consecutive slots, counts what it keeps,
// and, with the counts of the warps before it, writes the kept slots in their order.
// Bound by instructions and the latency of the five steps: 256 slices of 4352 tokens 12 us, of 26000
// tokens 37 us (keys in registers, 1024 threads a slice: 18 and 45 us).
template <bool HELD, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) evict_select_kernel(EvictCall c) {
    constexpr int kSelWarps = kSelThreads / 32, kBinsOf = kBins / kSelThreads;  // bins of a thread
    grid_go();
    extern __shared__ uint32_t held[];  // HELD: [t_cap]
    __shared__ __align__(16) uint32_t hist[kBins];
    __shared__ uint32_t sums[2][kSelWarps];
    __shared__ uint32_t s_digit, s_rank;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = blockIdx.x, b = slice / c.Hkv;
    int64_t len = c.lens[b];
    if (len < 0 || len > c.t_cap) {
        if (tid == 0 && c.dev_status) *c.dev_status = TQ_ERR_INVALID_ARG;
        len = len < 0 ? 0 : c.t_cap;
    }
    const uint32_t n = (uint32_t)len, budget = (uint32_t)c.budget;
    const uint32_t keep = n < budget ? n : budget;
    int32_t *kept = c.kept + (int64_t)slice * budget;
    if (tid == 0) {
        c.counts[slice] = (int32_t)keep;
        if (slice == b * c.Hkv) c.out_lens[b] = (int32_t)keep;
    }
    if (n <= budget) {
        for (uint32_t t = tid; t < n; t += kSelThreads) kept[t] = (int32_t)t;
        return;
    }
    const float *w = (const float *)c.src[6] + (int64_t)slice * c.t_cap;
    const uint32_t safe = n - (uint32_t)c.recent;  // slots from here on are kept
    // the keys of slots t, t + STEP, ...: `whole`, none of them past `safe` or the end
    auto keys_at = [&](auto step, bool again, bool whole, uint32_t t, uint32_t end, uint32_t(&x)[kAtOnce]) {
        constexpr uint32_t STEP = decltype(step)::value;
        const float *p = w + t;
        const uint32_t *q = held + t;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (whole || t + i * STEP < end) x[i] = HELD && again ? q[i * STEP] : __float_as_uint(p[i * STEP]);
        if (HELD && again) return;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            x[i] = !whole && t + i * STEP >= safe ? 0xFFFFFFFFu : weight_key(__uint_as_float(x[i]));
    };
    // f(key, slot) for the slots t, t + STEP, ... below end, kAtOnce loads at a time
    auto sweep = [&](auto step, bool again, uint32_t t, uint32_t end, auto f) {
        constexpr uint32_t STEP = decltype(step)::value;
        const uint32_t plain = HELD && again ? end : min(end, safe);
        uint32_t x[kAtOnce] = {};
        for (; t + (kAtOnce - 1) * STEP < plain; t += kAtOnce * STEP) {
            keys_at(step, again, true, t, end, x);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) f(x[i], t + i * STEP);
        }
        for (; t < end; t += kAtOnce * STEP) {
            keys_at(step, again, false, t, end, x);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (t + i * STEP < end) f(x[i], t + i * STEP);
        }
    };
    const Step<kSelThreads> all_threads;
    const Step<32> one_warp;
    // the threshold: the keep-th largest key, found 11, 11 and 10 bits at a time
    uint32_t prefix = 0, mask = 0, rank = keep;  // the rank-th largest of the keys that match
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t dm = pass < 2 ? 2047u : 1023u;
#pragma unroll
        for (int k = 0; k < kBinsOf; ++k) hist[tid + k * kSelThreads] = 0;
        __syncthreads();
        if (pass == 0) {
            sweep(all_threads, false, tid, n, [&](uint32_t key, uint32_t s) {
                if (HELD) held[s] = key;
                atomicAdd(&hist[key >> 21], 1u);
            });
        } else {
            sweep(all_threads, true, tid, n, [&](uint32_t key, uint32_t) {
                count_if((key & mask) == prefix, &hist[(key >> shift) & dm]);
            });
        }
        __syncthreads();
        // suffix sums over the bins from the top: thread 0 takes the highest
        const uint32_t top = kBins - 1 - kBinsOf * tid;
        uint32_t h[kBinsOf], mine = 0;
#pragma unroll
        for (int k = 0; k < kBinsOf; ++k) mine += h[k] = hist[top - k];
        uint32_t x = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sums[0][warp] = x;
        __syncthreads();
        uint32_t above = x - mine;
        for (int k = 0; k < warp; ++k) above += sums[0][k];
        if (above < rank && rank <= above + mine) {
#pragma unroll
            for (int k = 0; k < kBinsOf; ++k) {
                if (above < rank && rank <= above + h[k]) {
                    s_digit = top - k;
                    s_rank = rank - above;
                }
                above += h[k];
            }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        mask |= dm << shift;
        rank = s_rank;
    }
    // kept: keys above the threshold, and the first `rank` slots whose key equals it
    const uint32_t run = ((n + 31) / 32 + kSelWarps - 1) / kSelWarps * 32;  // slots of a warp
    const uint32_t first = min(warp * run, n), last = n - first < run ? n : first + run;
    uint32_t gt = 0, eq = 0;
    sweep(one_warp, true, first + lane, last, [&](uint32_t key, uint32_t) {
        gt += key > prefix;
        eq += key == prefix;
    });
    gt = __reduce_add_sync(kFull, gt);
    eq = __reduce_add_sync(kFull, eq);
    if (lane == 0) sums[0][warp] = gt, sums[1][warp] = eq;
    __syncthreads();
    uint32_t ngt = 0, neq = 0;  // above and equal in the slots before
    for (int k = 0; k < warp; ++k) ngt += sums[0][k], neq += sums[1][k];
    const uint32_t below = (1u << lane) - 1u;
    int32_t *at = kept + ngt + min(neq, rank);
    auto write = [&](bool whole, uint32_t t) {
        uint32_t x[kAtOnce] = {};
        keys_at(one_warp, true, whole, t + lane, last, x);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint32_t s = t + 32 * i + lane;
            const bool there = whole || s < last;
            bool keeps = there && x[i] > prefix;
            const bool equal = there && x[i] == prefix;
            const uint32_t es = __ballot_sync(kFull, equal);
            if (es != 0) {
                keeps |= equal && neq + __popc(es & below) < rank;
                neq += __popc(es);
            }
            const uint32_t ks = __ballot_sync(kFull, keeps);
            if (keeps) at[__popc(ks & below)] = (int32_t)s;
            at += __popc(ks);
        }
    };
    uint32_t t = first;
    for (const uint32_t plain = HELD ? last : min(last, safe); t + 32 * kAtOnce <= plain; t += 32 * kAtOnce) write(true, t);
    for (; t < last; t += 32 * kAtOnce) write(false, t);
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
// widest words that every record is aligned to for the packed arrays.  Bound by DRAM: for one token
// kept of three (256 slices, 8192 kept of 26000) 102 us, in which it reads 505 MB for the 174 MB that
// are kept, since DRAM gives 64 bytes for a record of 2 to 48, and writes 174 MB: 6.7 TB/s.
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

}  // namespace

cudaError_t launch_evict(const EvictCall &c, cudaStream_t s) {
    // Keys wait in shared memory wherever they fit (256 slices, read again against held, the copy
    // included: 53.3 / 51.3 us for 4352 tokens each, 147.3 / 141.9 for 26000); where only one CTA an SM
    // does, it has the threads of two (512 threads: 147.0).
    const unsigned slices = (unsigned)(c.B * c.Hkv);
    const size_t held = sizeof(uint32_t) * (size_t)c.t_cap;
    if (held <= kHeldMax) {
        const bool alone = held > kHeldPair;
        const auto kernel = alone ? evict_select_kernel<true, 1024> : evict_select_kernel<true, 512>;
        const cudaError_t e = allow_smem((const void *)kernel, kHeldMax);
        if (e != cudaSuccess) return e;
        kernel<<<slices, alone ? 1024 : 512, held, s>>>(c);
    } else {
        evict_select_kernel<false, 512><<<slices, 512, 0, s>>>(c);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int chunks = (int)evict_chunks(c.budget);
    return launch_after(evict_copy_kernel, (unsigned)(chunks * c.B * c.Hkv), kCopyThreads, 0, s, c, chunks);
}

}  // namespace tq
