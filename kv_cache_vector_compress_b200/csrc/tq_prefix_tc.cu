// tq_prefix_tc.cu -- attention of many query rows over one shared compressed prefix (tcgen05).
//
// The rows of all sequences that read a KV head's prefix are one operand: 128 rows at a time are
// multiplied with tiles of the prefix that are decoded once for them.
//   S = Q B^T   128 x TT, B = TT tokens x (d + m): c / sigma, then +-rho, in fp16
//   O += W V    128 x d,  W = the weights in fp16, V = TT tokens x d: ||v|| (c / tau) in fp16
// The key norms multiply the scores in 32 bits.  (In the operands ||k|| rho, rounded to fp16, moved
// all of a token's signs together: the largest error of the kernel, 7e-4 of the output at 2 bits.)  The
// value norms are multiplied into the decoded operands (on the FMA pipe, which decoding leaves idle),
// scaled by a power of two 2^s a tile that puts the tile's largest norm in [2^10, 2^11): the products
// stay inside fp16 whatever the norms are.  With z = f ||k|| S and a reference N >= z - s - 15,
// W = 2^(z - s - N), and the normaliser is 2^s sum W: the partial result (N, l, o) is that of
// tq_serve.cuh.
//
// Roles: eight softmax warps (two threads a row, half of a tile's tokens each), eight decoder warps,
// one warp that issues the MMAs.  The softmax first takes the weights with the reference as it is;
// if any comes out above 2^15 (the first tile, hardly ever later) the tile is done again with a new
// reference, so that the usual path needs no maximum before its exponentials.
// Q stays in tensor memory as the A operand and W is written over the scores it came from, so that
// shared memory carries only the decoded tiles: with both operands in shared memory a 128 x 128 x 16
// product reads 128 bytes a cycle, all that there is.  Decoded tiles are double buffered, keys and
// values apart (a key tile is free again once its scores are computed).  With two score buffers
// (d <= 128) the scores of the next tile are computed while this one's softmax runs.
//
// Decoding is that of tq_ragged_mma.cuh (byte permutations), eight values of one word a 16-byte
// chunk: selector i of a word holds bits 4 n + i, so column 32 g + 8 i + n of an operand is
// coordinate 32 g + 4 n + i; sign columns go by pairs of bits (l, l + 16).  The query rows are laid
// out the same way by the preparation and the results put in order by the partial's writer.
// The value tile has its d columns contiguous for each token: the B operand is MN-major.
//
// The packed words arrive by asynchronous copies, two tiles ahead.  (Fetched into registers a tile
// ahead they cost twice the instructions, and the wait for one tile's words often waited for the
// next one's too.)
//
// Bound by the decoders: 128 tokens of d = 128 at 3 bits take them 3200 cycles, the MMAs of the tile
// 1470, the softmax less than the decoders.  256 rows on each of 8 prefixes of 131072 tokens, d = 128,
// 3 bits: 197 to 217 us (368 000 cycles), 0.79 to 0.87 PFLOP/s where a large bf16 matrix product measures 1.66.  Sixteen
// decoder warps with registers moved to them from the softmax, and a separate warp for the copies,
// took as long; there is no room for more registers in flight.
//
// Every wait is bounded; one that runs out sets TQ_ERR_TIMEOUT in dev_status.
#include <float.h>

#include <type_traits>

#include "tq_decode.cuh"
#include "tq_f32x2.cuh"
#include "tq_launch.cuh"
#include "tq_serve.cuh"
#include "tq_sm100.cuh"

namespace tq {

namespace {

using namespace sm100;
using namespace decode;

constexpr int kSmWarps = 8, kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kThreads = 32 * (kSmWarps + kDecWarps + 1);

template <int D, int KB_>
struct Cfg {
    static constexpr int KB = KB_, VB = KB_ + 1, VN = VB < 3 ? VB : 3;
    static constexpr int TT = prefix_tile(D);    // tokens of a tile
    static constexpr int K = D + D / 2;          // operand length of the scores
    static constexpr int G32 = D / 32, SW = D / 64;
    static constexpr int KWPT = KB * G32, VWPT = VB * G32;
    static constexpr int SB = D <= 128 ? 2 : 1;  // score buffers
    static constexpr uint32_t BLK = TT * 128;    // a block of 64 operand columns of a tile
    static constexpr uint32_t KST = (K + 63) / 64 * BLK, VST = D / 64 * BLK;
    // tensor memory columns
    static constexpr uint32_t CS = 0, CO = SB * TT, CQ = CO + D;
    static_assert(CQ + K / 2 <= 512, "tensor memory");
    // shared memory
    static constexpr uint32_t OV = 2 * KST, OM = OV + 2 * VST, OB = OM + 2 * 16;  // OM: a tile's scales
    static constexpr uint32_t OX = OB + 16 * 8 + 16;  // barriers, flags; exchanges of the halves
    // a tile's packed words: key codes, signs, value codes, then the norms from an even record on
    static constexpr uint32_t NB = (TT + 2) * 2;
    static constexpr uint32_t RS = TT * KWPT * 4, RV = RS + TT * SW * 4, RN = RV + TT * VWPT * 4;
    static constexpr uint32_t RAW = (RN + 3 * NB + 15) / 16 * 16;
    static constexpr uint32_t ON = (OX + 2 * 128 * 4 + 96 + 15) / 16 * 16;  // key norms in fp32, two tiles
    static constexpr uint32_t OR = ON + 2 * TT * 4;
    static constexpr uint32_t SMEM = OR + 3 * RAW + 1024;  // alignment
    // words of a decoder thread's share of a tile
    static constexpr int KI = TT * G32 / kDecThreads, TP = kDecThreads / G32;  // TP tokens a pass
    static constexpr int SWT = TT * SW;  // sign words of a tile: at most one a thread
    static_assert(KI * TP == TT && SWT <= kDecThreads, "shares");
};

enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPFull = 10, kEnd = 12 };

struct PrefixArgs {
    Prepared P;
    RaggedCache c;  // stride: tokens of the prefix; rows: rows of a KV head
    const uint16_t *qrows;
    const float *fscale;
    float *part;
    int splits, tiles_per;
    int32_t *dev_status;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Wait for this thread's tensor memory loads; the numbers are used only behind it.
__device__ __forceinline__ void ld_done(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Eight tries at a barrier's phase, two instructions each.
__device__ __forceinline__ bool try_wait8(uint32_t addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    return ok != 0;
}

// mbar_wait with the flag and the clock looked at after every 64 tries only: waiting warps share
// their schedulers, and the pipe that decodes, with the decoders.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const uint32_t b = smem_u32(bar);
    if (try_wait8(b, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i)
            if (try_wait8(b, parity)) return true;
        if (*abort) return false;
        if (globaltimer() - t0 > kTimeoutNs) {
            *abort = 1;
            return false;
        }
    }
}

// Four pairs of fp16 numbers, each times `f`, to 16 bytes of shared memory.
__device__ __forceinline__ void store_scaled(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t f) {
    asm volatile(
        "{\n\t.reg .b32 x, y, z, w;\n\tmul.rn.f16x2 x, %1, %5;\n\tmul.rn.f16x2 y, %2, %5;\n\tmul.rn.f16x2 z, %3, %5;\n\t"
        "mul.rn.f16x2 w, %4, %5;\n\tst.shared.v4.b32 [%0], {x, y, z, w};\n\t}" ::"r"(at),
        "r"(a), "r"(b), "r"(c), "r"(d), "r"(f)
        : "memory");
}
__device__ __forceinline__ void store_pairs(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// mma_ts by the lanes that have `lead` set.
__device__ __forceinline__ void mma_ts_if(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}

// Byte offset of 16-byte chunk c of token t in a tile of operand columns (128-byte swizzle).
template <uint32_t BLK>
__device__ __forceinline__ uint32_t chunk_at(int t, int c) {
    return (uint32_t)(c >> 3) * BLK + (uint32_t)t * 128 + (uint32_t)(((c & 7) ^ (t & 7)) << 4);
}

// MN-major B operand: 64 columns (128 bytes) of each token, 8 tokens 1024 bytes apart, the next 64
// columns `next` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t next) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(next >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <int BYTES>
__device__ __forceinline__ void cp_async(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}

// One decoder's share of the copies of an array of W words a record: every kDecThreads-th piece of a
// tile, the widest that every record is aligned to.
template <int W, int TT>
struct Copier {
    static constexpr int G = W % 4 == 0 ? 4 : W % 2 == 0 ? 2 : 1;
    static constexpr int PIECES = TT * W / G, N = (PIECES + kDecThreads - 1) / kDecThreads;
    const uint32_t *src;  // this thread's first piece of the next tile
    __device__ __forceinline__ void start(const uint32_t *array, int64_t rec, int dt) { src = array + rec * W + dt * G; }
    // the next tile, `cnt` records of it
    __device__ __forceinline__ void copy(uint8_t *dst, int cnt, int dt) {
        const int have = cnt == TT ? PIECES : cnt * W / G;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = dt + i * kDecThreads;
            if (c < have) cp_async<4 * G>(dst + c * G * 4, src + i * kDecThreads * G);
        }
        src += TT * W;
    }
};

// N words of shared memory at a multiple of N words.
template <int N>
__device__ __forceinline__ void read_words(const uint32_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 2) {
        const uint2 v = *(const uint2 *)p;
        w[0] = v.x;
        w[1] = v.y;
    } else if constexpr (N == 4) {
        const uint4 v = *(const uint4 *)p;
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = p[i];
    }
}

template <int D, int KB>
__global__ void __launch_bounds__(kThreads, 1) prefix_tc_kernel(PrefixArgs a) {
    using C = Cfg<D, KB>;
    constexpr int VB = C::VB, VN = C::VN, TT = C::TT;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;  // (an offset: the address space stays known)
    uint64_t *bars = (uint64_t *)(sm + C::OB);
    volatile int *abort_s = (volatile int *)(sm + C::OB + 16 * 8);
    uint32_t *tmem_s = (uint32_t *)(sm + C::OB + 16 * 8 + 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int unit = blockIdx.x / a.splits, split = blockIdx.x - unit * a.splits, kv = unit % a.c.slices,
              rt = unit / a.c.slices;
    const int T = (int)a.c.stride, tiles = (T - 1) / TT + 1;
    const int j0 = split * a.tiles_per, nT = min(a.tiles_per, tiles - j0);

    if (tid == 0) {
        *abort_s = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[kKFull + i], kDecWarps);
            mbar_init(&bars[kKEmpty + i], 1);
            mbar_init(&bars[kVFull + i], kDecWarps);
            mbar_init(&bars[kVEmpty + i], 1);
            mbar_init(&bars[kSFull + i], 1);
            mbar_init(&bars[kPFull + i], kSmWarps);
        }
        mbar_init(&bars[kEnd], 1);
        fence_mbar_init();
    }
    if (warp == kSmWarps + kDecWarps) {
        tmem_alloc(tmem_s, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, *tmem_s, 0);

    if (warp < kSmWarps) {
        // ------------------------------------------------------------ softmax
        // Warps w and w + 4 share the rows of lane quarter w: half h of the columns each.  They agree
        // on the reference through shared memory and a barrier of their own.
        constexpr int HC = TT / 2;  // columns of a thread
        const int quarter = warp & 3, h = warp >> 2, r128 = 32 * quarter + lane;
        const int row = rt * 128 + r128;
        const bool there = row < a.c.rows;
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        float *xch = (float *)(sm + C::OX);
        volatile int *flags = (volatile int *)(sm + C::OX + 2 * 128 * 4);  // [two tiles, gave up][half][quarter]
        auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory"); };
        grid_wait();  // the preparation's rows; nothing else here is written by the kernel before
        if (tid == 0) grid_go();
        {  // the query rows into tensor memory
            const uint4 *q = (const uint4 *)(a.qrows + ((int64_t)kv * a.c.rows + row) * C::K);
#pragma unroll 2
            for (int c = h; c < C::K / 32; c += 2) {
                uint32_t v[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 x = there ? q[4 * c + k] : make_uint4(0, 0, 0, 0);
                    v[4 * k] = x.x;
                    v[4 * k + 1] = x.y;
                    v[4 * k + 2] = x.z;
                    v[4 * k + 3] = x.w;
                }
                tmem_st16(tl + C::CQ + 16 * c, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kPFull + (C::SB - 1)]);  // phase 0 of the last buffer: Q is there
        }
        const float f = there ? a.fscale[ragged_row(a.c, kv, row)] : 0.f;
        float N = -FLT_MAX;
        f2 l2 = pack2(0.f, 0.f);
        bool ok = true;
        for (int j = 0; j < nT; ++j) {
            const int sb = j % C::SB, vs = j & 1;
            // a pair of warps stays together: one that gave up says so and leaves with the other
            if (!wait_for(&bars[kVFull + vs], (j >> 1) & 1, abort_s) ||
                !wait_for(&bars[kSFull + sb], (j / C::SB) & 1, abort_s))
                ok = false;
            tc_fence_after();
            const uint32_t ts = tl + C::CS + sb * TT;
            // s and 2^s of the tile, and the key norms of this thread's columns (the same for a whole warp)
            const float2 scl = *(const float2 *)(sm + C::OM + vs * 16);
            const float *norms = (const float *)(sm + C::ON) + vs * TT + HC * h;
            const f2 ff = pack2(f, f);
            // tokens of this thread's columns that are there (the last tile may end early)
            const int cols = T - (j0 + j) * TT - HC * h;
            // the weights, as fp16 pairs, and their sum; returns the largest pair
            uint32_t p[HC / 2];
            f2 sum_w;
            auto weigh = [&]() -> __half2 {
                const f2 nn = pack2(-(N + scl.x), -(N + scl.x));
                __half2 top = __floats2half2_rn(0.f, 0.f);
                f2 la = pack2(0.f, 0.f), lb = la;
#pragma unroll
                for (int c = 0; c < HC / 32; ++c) {
                    uint32_t s[32];
                    tmem_ld32(ts + HC * h + 32 * c, s);
                    ld_done(s);
                    float e[32];
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        const ulonglong2 kn = *(const ulonglong2 *)(norms + 32 * c + 2 * k);
                        unpack2(fma2(pack2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), mul2(kn.x, ff), nn),
                                e[2 * k], e[2 * k + 1]);
                        unpack2(fma2(pack2(__uint_as_float(s[2 * k + 2]), __uint_as_float(s[2 * k + 3])),
                                     mul2(kn.y, ff), nn),
                                e[2 * k + 2], e[2 * k + 3]);
                    }
                    if (cols < HC) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k >= cols) e[k] = -INFINITY;
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) e[k] = ex2(e[k]);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        la = add2(la, pack2(e[2 * k], e[2 * k + 1]));
                        lb = add2(lb, pack2(e[2 * k + 2], e[2 * k + 3]));
                        const __half2 h0 = __floats2half2_rn(e[2 * k], e[2 * k + 1]);
                        const __half2 h1 = __floats2half2_rn(e[2 * k + 2], e[2 * k + 3]);
                        top = __hmax2(top, __hmax2(h0, h1));
                        p[16 * c + k] = *(const uint32_t *)&h0;
                        p[16 * c + k + 1] = *(const uint32_t *)&h1;
                    }
                }
                sum_w = add2(la, lb);
                return top;
            };
            const __half2 top = weigh();
            static_assert(kHeadroom == 15.f, "2^15");
            const bool over = fmaxf(__low2float(top), __high2float(top)) > 32768.f;
            const bool any = __any_sync(kFull, over);
            if (lane == 0) flags[(j & 1) * 8 + 4 * h + quarter] = any || !ok;
            tc_fence_before();
            pair_sync();  // and both have read their scores: weights may go over them
            if (any || !ok || flags[(j & 1) * 8 + 4 * (1 - h) + quarter]) {
                // once more with a new reference: O and l move to it (O once the last product is complete)
                float mx = -FLT_MAX;
#pragma unroll 1
                for (int c = 0; c < HC / 16; ++c) {
                    uint32_t s[16];
                    tmem_ld16(ts + HC * h + 16 * c, s);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (16 * c + k < cols) mx = fmaxf(mx, __uint_as_float(s[k]) * (f * norms[16 * c + k]) - scl.x);
                }
                xch[128 * h + r128] = mx;
                pair_sync();
                mx = fmaxf(mx, xch[128 * (1 - h) + r128]);
                const float up = mx > N + kHeadroom ? mx - kTopWeight : N, sc = exp2f(N - up);
                N = up;
                l2 = mul2(l2, pack2(sc, sc));
                if (j > 0) {
                    ok = ok && wait_for(&bars[kVEmpty + ((j - 1) & 1)], ((j - 1) >> 1) & 1, abort_s);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[16];
                        tmem_ld16(tl + C::CO + (D / 2) * h + 16 * c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sc);
                        tmem_st16(tl + C::CO + (D / 2) * h + 16 * c, o);
                    }
                }
                weigh();
                if (lane == 0) flags[16 + 4 * h + quarter] = !ok;
                pair_sync();  // both have read their scores again, and the exchange
                if (!ok || flags[16 + 4 * (1 - h) + quarter]) {
                    ok = false;
                    break;
                }
            }
            l2 = fma2(sum_w, pack2(scl.y, scl.y), l2);
#pragma unroll
            for (int c = 0; c < HC / 32; ++c) {
                uint32_t v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = p[16 * c + k];
                tmem_st16(ts + HC / 2 * h + 16 * c, v);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kPFull + sb]);
        }
        ok = ok && wait_for(&bars[kVEmpty + ((nT - 1) & 1)], ((nT - 1) >> 1) & 1, abort_s);
        tc_fence_after();
        float la, lb;
        unpack2(l2, la, lb);
        if (h == 1) xch[r128] = la + lb;
        pair_sync();
        if (__all_sync(kFull, ok)) {
            float *pp = a.part + (((int64_t)split * a.c.slices + kv) * a.c.rows + row) * partial_stride(D);
            if (there && h == 0) *(float4 *)pp = make_float4(N, la + lb + xch[r128], 0.f, 0.f);
            const float tau = a.P.serve->tau;
#pragma unroll 1
            for (int g = h; g < D / 32; g += 2) {
                uint32_t o[32];
                tmem_ld32(tl + C::CO + 32 * g, o);
                ld_done(o);
                if (there)
#pragma unroll
                    for (int n = 0; n < 8; ++n)
                        *(float4 *)(pp + 4 + 32 * g + 4 * n) =
                            make_float4(__uint_as_float(o[n]) * tau, __uint_as_float(o[8 + n]) * tau,
                                        __uint_as_float(o[16 + n]) * tau, __uint_as_float(o[24 + n]) * tau);
            }
        }
        tc_fence_before();
    } else if (warp < kSmWarps + kDecWarps) {
        // ------------------------------------------------------------ decoders
        const int dt = tid - 32 * kSmWarps;
        const ServeTables *tab = a.P.serve;
        const Lut kh = load_lut<(1 << KB)>(tab->kh);
        const Lut vh = load_lut<(1 << VN)>(tab->vh + (VB == 4 ? 8 : 0));
        const int64_t rec0 = (int64_t)kv * T;
        const uint32_t sbase = smem_u32(sm);
        // This thread's words: of word g of tokens tk, tk + TP, ...: eight tokens (the rows of a swizzle
        // pattern) x every word, then the next eight tokens; and sign word sg of token ts.
        const int tk = (dt & 7) + 8 * (dt / (8 * C::G32)), g = (dt >> 3) % C::G32;
        const int ts = (dt & 7) + 8 * (dt / (8 * C::SW)), sg = (dt >> 3) % C::SW;
        uint32_t koff[4], soff[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            koff[u] = chunk_at<C::BLK>(tk, 4 * g + u);
            soff[u] = chunk_at<C::BLK>(ts, D / 8 + 4 * sg + u);
        }
        Copier<C::KWPT, TT> ck;
        Copier<C::SW, TT> cs;
        Copier<C::VWPT, TT> cv;
        const int64_t first = rec0 + (int64_t)j0 * TT;
        ck.start(a.c.kcodes, first, dt);
        cs.start(a.c.ksigns, first, dt);
        cv.start(a.c.vcodes, first, dt);
        // Norms in words of two, from the even record at or below a tile's first (tiles are even, so
        // the parity is the same for all); a word that would pass the end of the array as its one half
        // that is there.  The first 128 threads copy the keys' two, the others the values'.
        static_assert(TT / 2 + 1 <= 128, "norm words");
        const int odd = (int)(first & 1), nw = dt & 127;
        const uint16_t *n0 = (dt < 128 ? a.c.knorm : a.c.vnorm) + first - odd + 2 * nw;
        const uint16_t *n1 = a.c.krnorm + first - odd + 2 * nw;
        int64_t n_at = first - odd + 2 * nw;
        const uint32_t nd = C::RN + (dt < 128 ? 0 : 2 * C::NB) + 4 * nw;
        auto issue = [&](int j, int slot) {
            if (j < nT) {
                const int cnt = min(TT, T - (j0 + j) * TT);
                uint8_t *r = sm + C::OR + (uint32_t)slot * C::RAW;
                ck.copy(r, cnt, dt);
                cs.copy(r + C::RS, cnt, dt);
                cv.copy(r + C::RV, cnt, dt);
                if (nw < (odd + cnt + 1) >> 1) {
                    if (n_at + 2 <= a.c.records) {
                        cp_async<4>(r + nd, n0);
                        if (dt < 128) cp_async<4>(r + nd + C::NB, n1);
                    } else {
                        *(uint16_t *)(r + nd) = *n0;
                        if (dt < 128) *(uint16_t *)(r + nd + C::NB) = *n1;
                    }
                }
                n0 += TT;
                n1 += TT;
                n_at += TT;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // The exponent field of the largest of the tile's norms, at least 1 (fp16 bits are in the order
        // of the numbers; infinities and NaN count as the largest number).  Every warp takes it itself.
        auto top_field = [&](const uint16_t *n, int cnt) -> int {
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < TT / 32; ++i)
                if (lane + 32 * i < cnt) mx = max(mx, (uint32_t)(n[lane + 32 * i] & 0x7FFFu));
            mx = __reduce_max_sync(kFull, mx) >> 10;
            return min(max((int)mx, 1), 30);
        };
        auto power = [](int e) { return __int_as_float((127 + e) << 23); };
        auto pair_of = [](float v) {  // (v, v) in fp16
            const __half2 x = __float2half2_rn(v);
            return *(const uint32_t *)&x;
        };
        // Decode tile j.  A warp whose wait gave up still takes part in the barriers, which the others wait at.
        bool live = true;
        int slot = 0;  // j % 3
        auto decode_tile = [&](int j, auto stage) {
            constexpr int st = decltype(stage)::value;  // j % 2
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            // every decoder's copies of this tile have landed, and the last tile's words are read
            asm volatile("bar.sync 5, %0;" ::"n"(kDecThreads) : "memory");
            issue(j + 2, slot == 0 ? 2 : slot - 1);
            const uint8_t *r = sm + C::OR + (uint32_t)slot * C::RAW;
            slot = slot == 2 ? 0 : slot + 1;
            const int cnt = min(TT, T - (j0 + j) * TT);
            const uint16_t *rn = (const uint16_t *)(r + C::RN) + odd;
            const uint16_t *rkn = rn, *rkr = rn + C::NB / 2, *rvn = rn + C::NB;
            live = live && (j < 2 || wait_for(&bars[kKEmpty + st], ((j >> 1) - 1) & 1, abort_s));
            if (!live) return;
            const uint32_t kt = sbase + st * C::KST;
            // the value norms' exponent is field - 15; 2^ve puts it at 10
            const int ve = 25 - top_field(rvn, cnt);
            const float vscale = power(ve);
#pragma unroll
            for (int i = 0; i < C::KI; ++i) {
                const int tok = tk + i * C::TP;  // (past the end: any codes, whose scores are not used)
                uint32_t w[KB], x[4];
                read_words<KB>((const uint32_t *)r + tok * C::KWPT + g * KB, w);
                selectors<KB>(w, x);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t a0, a1, a2, a3;
                    look_up(kh, x[u], 0u, a0, a1);
                    look_up(kh, x[u] >> 16, 0u, a2, a3);
                    store_pairs(kt + koff[u] + i * C::TP * 128, a0, a1, a2, a3);
                }
            }
            if (dt < C::SWT) {
                const uint32_t neg = ts < cnt ? (rkr[ts] ^ 0x8000u) * 0x10001u : 0u;  // (-rho, -rho)
                const uint32_t w = ((const uint32_t *)(r + C::RS))[ts * C::SW + sg];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    store_pairs(kt + soff[u], ((w << (15 - 4 * u)) & 0x80008000u) ^ neg,
                                ((w << (14 - 4 * u)) & 0x80008000u) ^ neg, ((w << (13 - 4 * u)) & 0x80008000u) ^ neg,
                                ((w << (12 - 4 * u)) & 0x80008000u) ^ neg);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kKFull + st]);

            live = j < 2 || wait_for(&bars[kVEmpty + st], ((j >> 1) - 1) & 1, abort_s);
            if (!live) return;
            const uint32_t vt = sbase + C::OV + st * C::VST;
            if (dt == 0) *(float2 *)(sm + C::OM + st * 16) = make_float2((float)ve, vscale);
            if (dt < TT) ((float *)(sm + C::ON))[st * TT + dt] = dt < cnt ? f16_bits_to_f32(rkn[dt]) : 0.f;
#pragma unroll
            for (int i = 0; i < C::KI; ++i) {
                const int tok = tk + i * C::TP;
                const uint32_t nv = pair_of(tok < cnt ? f16_bits_to_f32(rvn[tok]) * vscale : 0.f);
                uint32_t w[VB];
                read_words<VB>((const uint32_t *)(r + C::RV) + tok * C::VWPT + g * VB, w);
                if constexpr (VB == 4) {
#pragma unroll
                    for (int p = 0; p < 3; ++p) w[p] = ~(w[p] ^ w[3]);
                }
                uint32_t x[4];
                selectors<VN>(w, x);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t f0 = 0, f1 = 0;
                    if constexpr (VB == 4) {  // the top bit is the sign
                        const uint32_t sg = (w[3] >> u) & 0x11111111u;
                        f0 = prmt(0x80u, 0u, sg);
                        f1 = prmt(0x80u, 0u, sg >> 16);
                    }
                    uint32_t a0, a1, a2, a3;
                    look_up(vh, x[u], f0, a0, a1);
                    look_up(vh, x[u] >> 16, f1, a2, a3);
                    store_scaled(vt + koff[u] + i * C::TP * 128, a0, a1, a2, a3, nv);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kVFull + st]);
        };
        issue(0, 0);
        issue(1, 1);
        for (int j = 0; j < nT; j += 2) {
            decode_tile(j, std::integral_constant<int, 0>{});
            if (j + 1 < nT) decode_tile(j + 1, std::integral_constant<int, 1>{});
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
        // ------------------------------------------------------------ MMAs
        // The whole warp runs this and its first lane issues: descriptors stay warp-uniform, an add of
        // a constant each.
        const uint32_t sbase = smem_u32(sm);
        constexpr uint32_t is = idesc_f16_f32(128, TT), iv = idesc_f16_f32(128, D) | (1u << 16);
        const uint32_t lead = lane == 0 ? 1u : 0u;
        const uint64_t kd0 = sdesc_sw128(sbase), vd0 = sdesc_mn(sbase + C::OV, C::BLK);
        // The scores of tile j go over the weights of tile j - SB, which that tile's value product reads
        // from tensor memory: they wait until it is complete.  (MMAs run in the order of their issue only
        // where they have one accumulator and shape, as the steps of one sum do; these have two.)
        auto scores = [&](int j) -> bool {
            const int st = j & 1, sb = j % C::SB, old = j - C::SB;
            if (old >= 0 && !wait_for(&bars[kVEmpty + (old & 1)], (old >> 1) & 1, abort_s)) return false;
            if (!wait_for(&bars[kKFull + st], (j >> 1) & 1, abort_s)) return false;
            tc_fence_after();
            const uint64_t kd = kd0 + (uint64_t)(st * (C::KST >> 4));
            const uint32_t acc = tmem + C::CS + sb * TT;
#pragma unroll
            for (int k = 0; k < C::K / 16; ++k)
                mma_ts_if(lead, acc, tmem + C::CQ + 8 * k, kd + (((k >> 2) * C::BLK + (k & 3) * 32) >> 4), is, k ? 1u : 0u);
            if (lead) {
                mma_commit(&bars[kKEmpty + st]);
                mma_commit(&bars[kSFull + sb]);
            }
            __syncwarp();
            return true;
        };
        // Q arrived as phase 0 of the last score buffer's W barrier
        bool ok = wait_for(&bars[kPFull + (C::SB - 1)], 0, abort_s) && scores(0);
        for (int j = 0; ok && j < nT; ++j) {
            const int st = j & 1, sb = j % C::SB;
            if (C::SB == 2 && j + 1 < nT) ok = scores(j + 1);
            const uint32_t ph = (uint32_t)(j / C::SB + (sb == C::SB - 1 ? 1 : 0)) & 1;
            ok = ok && wait_for(&bars[kVFull + st], (j >> 1) & 1, abort_s) && wait_for(&bars[kPFull + sb], ph, abort_s);
            if (!ok) break;
            tc_fence_after();
            const uint64_t vd = vd0 + (uint64_t)(st * (C::VST >> 4));
#pragma unroll
            for (int k = 0; k < TT / 16; ++k)
                mma_ts_if(lead, tmem + C::CO, tmem + C::CS + sb * TT + 8 * k, vd + (k * 2048 >> 4), iv,
                          (j | k) ? 1u : 0u);
            if (lead) mma_commit(&bars[kVEmpty + st]);
            __syncwarp();
            if (C::SB == 1 && j + 1 < nT) ok = scores(j + 1);
        }
        if (!ok) {  // gave up: products under way end before the memory that they use is given back
            if (lead) mma_commit(&bars[kEnd]);
            __syncwarp();
            const uint64_t t0 = globaltimer();
            while (!try_wait8(smem_u32(&bars[kEnd]), 0) && globaltimer() - t0 < kTimeoutNs) {
            }
        }
    }
    __syncthreads();
    if (warp == kSmWarps + kDecWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *abort_s && a.dev_status) atomicExch(a.dev_status, (int)TQ_ERR_TIMEOUT);
}

template <int D, int KB>
cudaError_t launch_one(const PrefixArgs &a, int row_tiles, cudaStream_t s) {
    using C = Cfg<D, KB>;
    cudaError_t e = allow_smem((const void *)prefix_tc_kernel<D, KB>, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(prefix_tc_kernel<D, KB>, (unsigned)(a.splits * a.c.slices * row_tiles), kThreads, C::SMEM, s, a);
}

template <int D>
cudaError_t launch_dim(const PrefixArgs &a, int row_tiles, cudaStream_t s) {
    switch (a.P.kbeta) {
        case 1: return launch_one<D, 1>(a, row_tiles, s);
        case 2: return launch_one<D, 2>(a, row_tiles, s);
        case 3: return launch_one<D, 3>(a, row_tiles, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

// One CTA an SM: the token tiles of a KV head are split so that all (KV head, row tile) pairs
// together take one wave, and no split is empty.
PrefixSplit prefix_split(int d, int Hkv, int64_t rows, int64_t t_prefix) {
    const int64_t tiles = (t_prefix + prefix_tile(d) - 1) / prefix_tile(d), units = Hkv * ((rows + 127) / 128);
    int64_t splits = kSms / units;
    if (splits < 1) splits = 1;
    if (splits > tiles) splits = tiles;
    PrefixSplit p;
    p.tiles_per = (int)((tiles + splits - 1) / splits);
    p.splits = (int)((tiles + p.tiles_per - 1) / p.tiles_per);
    return p;
}

cudaError_t launch_prefix_tc(const Prepared &P, const RaggedCache &c, const uint16_t *qrows, const float *fscale,
                             float *part, const PrefixSplit &sp, int32_t *dev_status, cudaStream_t s) {
    PrefixArgs a;
    a.P = P;
    a.c = c;
    a.qrows = qrows;
    a.fscale = fscale;
    a.part = part;
    a.splits = sp.splits;
    a.tiles_per = sp.tiles_per;
    a.dev_status = dev_status;
    const int row_tiles = (c.rows + 127) / 128;
    switch (P.d) {
        case 64: return launch_dim<64>(a, row_tiles, s);
        case 128: return launch_dim<128>(a, row_tiles, s);
        case 256: return launch_dim<256>(a, row_tiles, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace tq
