// tq_prefix_tc.cu -- attention of many query rows over one shared compressed prefix (tcgen05).
//
// The rows of all sequences that read a KV head's prefix are one operand: 128 rows at a time are
// multiplied with tiles of the prefix that are decoded once for them.
//   S = Q B^T   128 x TT, B = TT tokens x (d + m): centroids c / sigma, then +-rho (both fp16)
//   O += W V    128 x d,  W = 2^(y - N) in fp16, V = TT tokens x d: centroids c / tau
// (tq_serve.cuh: y = z + log2 ||v||, the reference N, partial results.)
//
// Roles: four softmax warps (a thread a row), eight decoder warps, one warp that issues the MMAs.
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
// Every wait is bounded; one that runs out sets TQ_ERR_TIMEOUT in dev_status.
#include <float.h>

#include "tq_decode.cuh"
#include "tq_serve.cuh"
#include "tq_sm100.cuh"

namespace tq {

namespace {

using namespace sm100;
using namespace decode;

constexpr int kSmWarps = 4, kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kThreads = 32 * (kSmWarps + kDecWarps + 1);
constexpr int kSms = 148;  // grid sizing (fixed so scratch sizes do not vary)

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
    static constexpr uint32_t OV = 2 * KST, OM = OV + 2 * VST, META = 3 * TT * 4, OB = OM + 2 * META;
    static constexpr uint32_t SMEM = OB + 16 * 8 + 16 + 1024;  // barriers, flags, alignment
    // words of a decoder thread's share of a tile
    static constexpr int KI = TT * G32 / kDecThreads, SI = (TT * SW + kDecThreads - 1) / kDecThreads;
};

enum Bar { kKFull = 0, kKEmpty = 2, kVFull = 4, kVEmpty = 6, kSFull = 8, kPFull = 10 };

struct PrefixArgs {
    Prepared P;
    RaggedCache c;  // stride: tokens of the prefix; rows: rows of a KV head
    const uint16_t *qrows;
    const float *fscale;
    float *part;
    int splits, tiles_per;
    int32_t *dev_status;
};

// ---- two fp32 numbers a register pair
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
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

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

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

// What a decoder thread has fetched of one tile.
template <class C>
struct Share {
    uint32_t k[C::KI][C::KB], s[C::SI], v[C::KI][C::VB];
    uint16_t rho[C::SI], vn[C::KI], kn, mv;
};

template <int D, int KB>
__global__ void __launch_bounds__(kThreads, 1) prefix_tc_kernel(PrefixArgs a) {
    using C = Cfg<D, KB>;
    constexpr int VB = C::VB, VN = C::VN, TT = C::TT;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = (uint64_t *)(sm + C::OB);
    volatile int *abort_s = (volatile int *)(sm + C::OB + 16 * 8);
    uint32_t *tmem_s = (uint32_t *)(sm + C::OB + 16 * 8 + 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int kv = blockIdx.x / a.splits, split = blockIdx.x - kv * a.splits, rt = blockIdx.y;
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
        fence_mbar_init();
    }
    if (warp == kSmWarps + kDecWarps) {
        tmem_alloc(tmem_s, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;

    if (warp < kSmWarps) {
        // ------------------------------------------------------------ softmax: a thread a row
        const int row = rt * 128 + tid;
        const bool there = row < a.c.rows;
        const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16);
        {  // the query rows into tensor memory
            const uint4 *q = (const uint4 *)(a.qrows + ((int64_t)kv * a.c.rows + row) * C::K);
#pragma unroll
            for (int c = 0; c < C::K / 32; ++c) {
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
        const f2 ff = pack2(f, f);
        float N = -FLT_MAX;
        f2 l2 = pack2(0.f, 0.f);
        bool ok = true;
        for (int j = 0; j < nT; ++j) {
            const int sb = j % C::SB, vs = j & 1;
            if (!mbar_wait(&bars[kVFull + vs], (j >> 1) & 1, abort_s) ||
                !mbar_wait(&bars[kSFull + sb], (j / C::SB) & 1, abort_s)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t ts = tl + C::CS + sb * TT;
            const float *meta = (const float *)(sm + C::OM + vs * C::META);
            // y of 32 tokens as 16 pairs
            auto ys = [&](const uint32_t (&s)[32], int c, f2 (&y)[16]) {
                const float4 *kn4 = (const float4 *)(meta + 32 * c), *lv4 = (const float4 *)(meta + TT + 32 * c);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 kn = kn4[k], lv = lv4[k];
                    const f2 s0 = pack2(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1]));
                    const f2 s1 = pack2(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3]));
                    y[2 * k] = fma2(mul2(s0, ff), pack2(kn.x, kn.y), pack2(lv.x, lv.y));
                    y[2 * k + 1] = fma2(mul2(s1, ff), pack2(kn.z, kn.w), pack2(lv.z, lv.w));
                }
            };
            float mx = -FLT_MAX;
            {
                uint32_t s[2][32];
                tmem_ld32(ts, s[0]);
#pragma unroll
                for (int c = 0; c < TT / 32; ++c) {
                    ld_done(s[c & 1]);
                    if (c + 1 < TT / 32) tmem_ld32(ts + 32 * (c + 1), s[(c + 1) & 1]);
                    f2 y[16];
                    ys(s[c & 1], c, y);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float u, v;
                        unpack2(y[k], u, v);
                        mx = fmaxf(mx, fmaxf(u, v));
                    }
                }
            }
            if (__any_sync(kFull, mx > N + 8.f)) {
                // move the reference: O and l to the new one (O once the last product is complete)
                const float up = fmaxf(mx, N), sc = exp2f(N - up);
                N = up;
                l2 = mul2(l2, pack2(sc, sc));
                if (j > 0) {
                    if (!mbar_wait(&bars[kVEmpty + ((j - 1) & 1)], ((j - 1) >> 1) & 1, abort_s)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(tl + C::CO + 16 * c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sc);
                        tmem_st16(tl + C::CO + 16 * c, o);
                    }
                }
            }
            const f2 nn = pack2(-N, -N);
            {
                uint32_t s[2][32];
                tmem_ld32(ts, s[0]);
#pragma unroll
                for (int c = 0; c < TT / 32; ++c) {
                    ld_done(s[c & 1]);
                    if (c + 1 < TT / 32) tmem_ld32(ts + 32 * (c + 1), s[(c + 1) & 1]);
                    f2 y[16];
                    ys(s[c & 1], c, y);
                    const float4 *rv4 = (const float4 *)(meta + 2 * TT + 32 * c);
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 rv = rv4[k];
                        float w0, w1, w2, w3;
                        unpack2(add2(y[2 * k], nn), w0, w1);
                        unpack2(add2(y[2 * k + 1], nn), w2, w3);
                        w0 = ex2(w0);
                        w1 = ex2(w1);
                        w2 = ex2(w2);
                        w3 = ex2(w3);
                        l2 = fma2(pack2(w0, w1), pack2(rv.x, rv.y), l2);
                        l2 = fma2(pack2(w2, w3), pack2(rv.z, rv.w), l2);
                        __half2 h0 = __floats2half2_rn(w0, w1), h1 = __floats2half2_rn(w2, w3);
                        p[2 * k] = *(uint32_t *)&h0;
                        p[2 * k + 1] = *(uint32_t *)&h1;
                    }
                    // over scores that are read already (the next chunk's are further on)
                    tmem_st16(ts + 16 * c, p);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kPFull + sb]);
        }
        ok = ok && mbar_wait(&bars[kVEmpty + ((nT - 1) & 1)], ((nT - 1) >> 1) & 1, abort_s);
        tc_fence_after();
        ok = __all_sync(kFull, ok);
        if (ok) {
            float *pp = a.part + (((int64_t)split * a.c.slices + kv) * a.c.rows + row) * partial_stride(D);
            float la, lb;
            unpack2(l2, la, lb);
            if (there) *(float4 *)pp = make_float4(N, la + lb, 0.f, 0.f);
            const float tau = a.P.serve->tau;
#pragma unroll 1
            for (int g = 0; g < D / 32; ++g) {
                uint32_t o[32];
                tmem_ld32(tl + C::CO + 32 * g, o);
                tmem_ld_wait();
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
        // word item x of a tile: eight tokens x every group, then the next eight tokens
        auto item = [&](int x, int per, int &t, int &g) {
            t = (x & 7) + 8 * (x / (8 * per));
            g = (x >> 3) % per;
        };
        auto fetch = [&](int j, Share<C> &h) {
            const int t0 = (j0 + j) * TT;
#pragma unroll
            for (int i = 0; i < C::KI; ++i) {
                int t, g;
                item(dt + i * kDecThreads, C::G32, t, g);
                const bool in = t0 + t < T;
                const int64_t rec = rec0 + t0 + t;
#pragma unroll
                for (int p = 0; p < KB; ++p) h.k[i][p] = in ? a.c.kcodes[rec * C::KWPT + g * KB + p] : 0u;
#pragma unroll
                for (int p = 0; p < VB; ++p) h.v[i][p] = in ? a.c.vcodes[rec * C::VWPT + g * VB + p] : 0u;
                h.vn[i] = in ? a.c.vnorm[rec] : (uint16_t)0;
            }
#pragma unroll
            for (int i = 0; i < C::SI; ++i) {
                int t, g;
                item(dt + i * kDecThreads, C::SW, t, g);
                const bool in = dt + i * kDecThreads < TT * C::SW && t0 + t < T;
                h.s[i] = in ? a.c.ksigns[(rec0 + t0 + t) * C::SW + g] : 0u;
                h.rho[i] = in ? a.c.krnorm[rec0 + t0 + t] : (uint16_t)0;
            }
            const bool in = dt < TT && t0 + dt < T;
            h.kn = in ? a.c.knorm[rec0 + t0 + dt] : (uint16_t)0;
            h.mv = in ? a.c.vnorm[rec0 + t0 + dt] : (uint16_t)0;
        };
        Share<C> cur, nxt;
        fetch(0, cur);
        for (int j = 0; j < nT; ++j) {
            const int st = j & 1;
            if (j + 1 < nT) fetch(j + 1, nxt);
            if (j >= 2 && !mbar_wait(&bars[kKEmpty + st], ((j >> 1) - 1) & 1, abort_s)) break;
            uint8_t *kt = sm + st * C::KST;
#pragma unroll
            for (int i = 0; i < C::KI; ++i) {
                int t, g;
                item(dt + i * kDecThreads, C::G32, t, g);
                uint32_t x[4];
                selectors<KB>(cur.k[i], x);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint4 o;
                    look_up(kh, x[u], 0u, o.x, o.y);
                    look_up(kh, x[u] >> 16, 0u, o.z, o.w);
                    *(uint4 *)(kt + chunk_at<C::BLK>(t, 4 * g + u)) = o;
                }
            }
#pragma unroll
            for (int i = 0; i < C::SI; ++i) {
                int t, g;
                item(dt + i * kDecThreads, C::SW, t, g);
                const uint32_t neg = (uint32_t)(cur.rho[i] ^ 0x8000u) * 0x10001u, w = cur.s[i];
                if (dt + i * kDecThreads < TT * C::SW)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint4 o;
                        o.x = ((w << (15 - 4 * u)) & 0x80008000u) ^ neg;
                        o.y = ((w << (14 - 4 * u)) & 0x80008000u) ^ neg;
                        o.z = ((w << (13 - 4 * u)) & 0x80008000u) ^ neg;
                        o.w = ((w << (12 - 4 * u)) & 0x80008000u) ^ neg;
                        *(uint4 *)(kt + chunk_at<C::BLK>(t, D / 8 + 4 * g + u)) = o;
                    }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kKFull + st]);

            if (j >= 2 && !mbar_wait(&bars[kVEmpty + st], ((j >> 1) - 1) & 1, abort_s)) break;
            uint8_t *vt = sm + C::OV + st * C::VST;
            if (dt < TT) {
                float *meta = (float *)(sm + C::OM + st * C::META);
                const bool in = (j0 + j) * TT + dt < T;
                const float v = f16_bits_to_f32(cur.mv), vc = fmaxf(v, kMinNorm);
                meta[dt] = f16_bits_to_f32(cur.kn);
                meta[TT + dt] = !in ? -INFINITY : v != v ? v : log2f(vc);
                meta[2 * TT + dt] = in ? 1.f / vc : 0.f;
            }
#pragma unroll
            for (int i = 0; i < C::KI; ++i) {
                int t, g;
                item(dt + i * kDecThreads, C::G32, t, g);
                // a value of norm 0 (or a token past the end) is 0: an empty table
                const bool some = (cur.vn[i] & 0x7FFFu) != 0;
                const Lut tb = {some ? vh.h0 : 0u, some ? vh.h1 : 0u, some ? vh.l0 : 0u, some ? vh.l1 : 0u};
                uint32_t w[VB];
#pragma unroll
                for (int p = 0; p < VB; ++p) w[p] = VB == 4 && p < 3 ? ~(cur.v[i][p] ^ cur.v[i][VB - 1]) : cur.v[i][p];
                uint32_t x[4];
                selectors<VN>(w, x);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t f0 = 0, f1 = 0;
                    if constexpr (VB == 4) {  // the top bit is the sign
                        const uint32_t sg = (w[3] >> u) & 0x11111111u;
                        f0 = prmt(some ? 0x80u : 0u, 0u, sg);
                        f1 = prmt(some ? 0x80u : 0u, 0u, sg >> 16);
                    }
                    uint4 o;
                    look_up(tb, x[u], f0, o.x, o.y);
                    look_up(tb, x[u] >> 16, f1, o.z, o.w);
                    *(uint4 *)(vt + chunk_at<C::BLK>(t, 4 * g + u)) = o;
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kVFull + st]);
            cur = nxt;
        }
    } else if (lane == 0) {
        // ------------------------------------------------------------ MMAs
        const uint32_t sbase = smem_u32(sm);
        constexpr uint32_t is = idesc_f16_f32(128, TT), iv = idesc_f16_f32(128, D) | (1u << 16);
        auto scores = [&](int j) -> bool {
            const int st = j & 1, sb = j % C::SB;
            if (!mbar_wait(&bars[kKFull + st], (j >> 1) & 1, abort_s)) return false;
            tc_fence_after();
            const uint32_t kb = sbase + st * C::KST;
#pragma unroll
            for (int k = 0; k < C::K / 16; ++k)
                mma_ts(tmem + C::CS + sb * TT, tmem + C::CQ + 8 * k, sdesc_sw128(kb + (k >> 2) * C::BLK + (k & 3) * 32), is,
                       k ? 1u : 0u);
            mma_commit(&bars[kKEmpty + st]);
            mma_commit(&bars[kSFull + sb]);
            return true;
        };
        // Q arrived as phase 0 of the last score buffer's W barrier
        bool ok = mbar_wait(&bars[kPFull + (C::SB - 1)], 0, abort_s) && scores(0);
        for (int j = 0; ok && j < nT; ++j) {
            const int st = j & 1, sb = j % C::SB;
            // the next scores go over the weights of tile j - 1: once their product is complete
            if (C::SB == 2 && j + 1 < nT)
                ok = (j == 0 || mbar_wait(&bars[kVEmpty + ((j - 1) & 1)], ((j - 1) >> 1) & 1, abort_s)) && scores(j + 1);
            const uint32_t ph = (uint32_t)(j / C::SB + (sb == C::SB - 1 ? 1 : 0)) & 1;
            ok = ok && mbar_wait(&bars[kVFull + st], (j >> 1) & 1, abort_s) && mbar_wait(&bars[kPFull + sb], ph, abort_s);
            if (!ok) break;
            tc_fence_after();
            const uint32_t vb = sbase + C::OV + st * C::VST;
#pragma unroll
            for (int k = 0; k < TT / 16; ++k)
                mma_ts(tmem + C::CO, tmem + C::CS + sb * TT + 8 * k, sdesc_mn(vb + k * 2048, C::BLK), iv,
                       (j | k) ? 1u : 0u);
            mma_commit(&bars[kVEmpty + st]);
            if (C::SB == 1 && j + 1 < nT)
                ok = mbar_wait(&bars[kVEmpty + st], (j >> 1) & 1, abort_s) && scores(j + 1);
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
    cudaError_t e = cudaFuncSetAttribute(prefix_tc_kernel<D, KB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)C::SMEM);
    if (e != cudaSuccess) return e;
    dim3 grid((unsigned)(a.splits * a.c.slices), (unsigned)row_tiles);
    prefix_tc_kernel<D, KB><<<grid, kThreads, C::SMEM, s>>>(a);
    return cudaGetLastError();
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
