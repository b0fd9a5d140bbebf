// tq_ragged_mma.cuh -- attention over caches of different lengths for a few query rows per slice,
// on the tensor cores (mma.sync m16n8k16), straight from the packed records.
//
// A warp takes 32 tokens at a time.  Scores: A = 16 tokens x 16 coordinates decoded from the packed
// words, B = query rows.  Value sums, transposed: A = 16 coordinates x 16 tokens, B = the softmax
// weights of the rows.  Both products sum over an index whose order is free (coordinates, tokens),
// and the rows of the value product may be any permutation of the coordinates, so each lane is
// given the coordinates that make its decoding cheapest: all of them from one or two words.
//
// Decoding: tq_decode.cuh; for the value product, whose pairs run along the tokens, two tokens'
// codes are interleaved nibble by nibble.
//
// Precision.  A query row is split in two fp16 numbers, hi + lo, in two columns of B, whose sums are
// added: the scores keep 22 bits of Q, and the key operands are exact for 1 bit and to 2^-21 for 2 bits
// (ServeTables: a well chosen scale; the Beta law 2^-19.6).  For 3 bits they are off by 3e-5 at most,
// 8e-6 on average, with that scale (the Beta law 5e-5 at most); F32 adds a second table, which costs as much again as the first.  Value sums: fp16
// weights and centroids for 16-bit outputs; F32 splits both.
//
// Bound by decoding: its byte permutations and logic run on the ALU pipe, which takes an instruction
// every other cycle and is 52 to 54% busy with the three or four warps a scheduler that the registers
// allow; the matrix instructions take 13 to 16% of theirs, DRAM a quarter.
// 256 slices of 4096 tokens on average, 4 rows, d = 128, 3 bits: 62 us, 1.7 TB/s of records and
// weights; 32 slices of 65536, d = 256, 4 bits: 300 us, 1.8 TB/s.  More CTAs an SM with fewer
// registers each were slower.
#pragma once

#include <float.h>

#include "tq_decode.cuh"
#include "tq_launch.cuh"
#include "tq_serve.cuh"

namespace tq {
namespace ragged {

using namespace decode;

constexpr int NW = 4;  // warps per CTA

template <int D, int KB_, int NT_, bool F32_>
struct Cfg {
    static constexpr int KB = KB_, VB = KB_ + 1, NT = NT_;
    static constexpr bool F32 = F32_;
    static constexpr int ROWS = 4 * NT;  // query rows of a CTA
    static constexpr int G32 = D / 32, M = D / 2, SW = M / 32;
    static constexpr int KWPT = KB * G32, VWPT = VB * G32;
    static constexpr int NG = D >= 128 ? D / 128 : 1;  // key words (of each plane) of a lane
    static constexpr int NI = D >= 128 ? 4 : 2;        // selectors from one word
    static constexpr int KC = D / 16, KS = KC + D / 32;  // products: codes, then signs
    static constexpr int PW = D / 16;                  // sign pairs of a lane
    static constexpr int LPW = 256 / D;                // lanes that share a sign word
    static constexpr int VH = D >= 256 ? 2 : 1;        // halves of a value word that a lane takes
    static constexpr int NO = F32 ? NT : 1;            // value accumulators
    static constexpr int TILES = D / 16;
    static constexpr bool BREG = D * NT <= 128;        // query fragments in registers
    // a stage of the ring: key codes, signs, value codes
    static constexpr uint32_t OS = kStage * KWPT * 4, OV = OS + kStage * SW * 4, STAGE = OV + kStage * VWPT * 4;
    static constexpr uint32_t CAP = D >= 256 ? 68 * 1024 : 48 * 1024;
    static constexpr int NST0 = CAP / (NW * STAGE);
    static constexpr int NST = NST0 < 2 ? 2 : NST0 > 4 ? 4 : NST0;
    static constexpr uint32_t MERGE = NW * ROWS * (D + 2) * 4;
    static constexpr uint32_t RING0 = NW * NST * STAGE, RING = RING0 > MERGE ? RING0 : (MERGE + 15) / 16 * 16;
    static constexpr uint32_t OMETA = RING, OB = OMETA + NW * 32 * 16, SMEM = OB + (BREG ? 0 : NT * KS * 32 * 8);
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

template <int BYTES>
__device__ __forceinline__ void cp_async(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
}

// A warp's copies of an array of W words a record: stage after stage, in the widest pieces that every
// record is aligned to.
template <int W>
struct Copier {
    static constexpr int G = W % 4 == 0 ? 4 : W % 2 == 0 ? 2 : 1;
    static constexpr int PIECES = kStage * W / G, N = (PIECES + 31) / 32;
    const uint32_t *src;  // this lane's first piece of the next stage
    __device__ __forceinline__ void start(const uint32_t *array, int64_t rec, int lane) { src = array + rec * W + lane * G; }
    // the next stage, `cnt` records of it; the one after is `step` stages on
    __device__ __forceinline__ void copy(uint8_t *dst, int cnt, int step, int lane) {
        uint32_t *d = (uint32_t *)dst + lane * G;
        if (cnt == kStage) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (PIECES % 32 == 0 || lane + 32 * i < PIECES) cp_async<4 * G>(d + 32 * i * G, src + 32 * i * G);
        } else {
            const int have = cnt * W / G;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (lane + 32 * i < have) cp_async<4 * G>(d + 32 * i * G, src + 32 * i * G);
        }
        src += (int64_t)step * kStage * W;
    }
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// One CTA: its pieces of the slices (tq_serve.cuh) for one block of ROWS query rows.  Each warp
// takes every NW-th stage of a piece through its own ring of asynchronous copies and keeps its own
// reference, sums and accumulators; they meet at the end of the piece.
//
// The reference N of a row moves only when some y exceeds it by more than 15: then the accumulators
// are rescaled (rare after the first stages), so that the usual path has no reduction over lanes.
template <int D, int KB, int NT, bool F32>
__global__ void __launch_bounds__(NW * 32, D >= 256 || F32 || NT > 1 ? 3 : 4)
    ragged_mma_kernel(const __grid_constant__ RaggedPair pair) {
    using C = Cfg<D, KB, NT, F32>;
    constexpr int VB = C::VB, VN = VB < 3 ? VB : 3;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, t4 = lane & 3;
    const bool second = (int)blockIdx.x >= pair.first;
    const RaggedArgs &a = pair.a[second];
    const int id = (int)blockIdx.x - (second ? pair.first : 0), cta = id % a.c.ctas, rblk = id / a.c.ctas;
    const int rblks = (a.c.rows + C::ROWS - 1) / C::ROWS;
    const ServeTables *T = a.P.serve;
    const Lut kh = load_lut<(1 << KB)>(T->kh);
    const Lut kl = load_lut<KB == 3 && F32 ? 8 : 1>(T->kl);
    // 4-bit values: the upper half of the table, magnitudes in ascending order
    const Lut vh = load_lut<(1 << VN)>(T->vh + (VB == 4 ? 8 : 0));
    const Lut vl = load_lut<F32 ? (1 << VN) : 1>(T->vl + (VB == 4 ? 8 : 0));
    const float tau = T->tau;
    // 2-bit keys: the four centroids as pairs of bytes; 2^16 where the compiler does not see it
    const uint32_t kp0 = T->kh[0] | ((uint32_t)T->kh[1] << 16), kp1 = T->kh[2] | ((uint32_t)T->kh[3] << 16);
    const uint32_t k16 = pair.two16;
    grid_wait();
    grid_go();
    const int64_t total = ragged_total(a.c);
    const int64_t w1 = cta_first(total, a.c.ctas, cta + 1);
    int64_t w = cta_first(total, a.c.ctas, cta);
    if (w >= w1) return;
    const int r0 = rblk * C::ROWS, nr = min(C::ROWS, a.c.rows - r0);
    uint8_t *ring = smem + (size_t)warp * C::NST * C::STAGE;
    float4 *meta = (float4 *)(smem + C::OMETA) + warp * 32;
    uint2 *bfrag = (uint2 *)(smem + C::OB);
    float *mrg = (float *)smem;
    const int vg = D >= 256 ? gid : D == 128 ? gid >> 1 : gid >> 2;  // value word of this lane
    const int vhalf = D >= 256 ? 0 : D == 128 ? gid & 1 : (gid >> 1) & 1;

    Piece pc;
    for (; w < w1; w += pc.counted) {
        pc = piece_at(a.c, w, w1);
        __syncthreads();  // the last piece's merge is read
        // ---- the warp's stages: pc.s0 + warp, + NW, ...
        const int64_t rec0 = pc.slice * a.c.stride;
        const int64_t first = pc.s0 + warp;
        // (32-bit counts: a slice has at most 2^26 stages)
        const int mine = first < pc.s1 ? (int)((pc.s1 - first + NW - 1) / NW) : 0;
        Copier<C::KWPT> ck;
        Copier<C::SW> cs;
        Copier<C::VWPT> cv;
        ck.start(a.c.kcodes, rec0 + first * kStage, lane);
        cs.start(a.c.ksigns, rec0 + first * kStage, lane);
        cv.start(a.c.vcodes, rec0 + first * kStage, lane);
        const int t_first = (int)(first * kStage);
        uint32_t fill = 0;  // byte offset of the slot that is filled next
        auto issue = [&](int i) {
            if (i < mine) {
                const int cnt = min(kStage, pc.len - (t_first + i * (NW * kStage)));
                ck.copy(ring + fill, cnt, NW, lane);
                cs.copy(ring + fill + C::OS, cnt, NW, lane);
                cv.copy(ring + fill + C::OV, cnt, NW, lane);
                fill = fill == (C::NST - 1) * C::STAGE ? 0 : fill + C::STAGE;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        uint16_t nk = 0, nrho = 0, nv = 0;  // the next stage's norms, a token a lane
        const uint16_t *pk = a.c.knorm + rec0 + t_first + lane, *pr = a.c.krnorm + rec0 + t_first + lane;
        const uint16_t *pv = a.c.vnorm + rec0 + t_first + lane;
        auto norms = [&](int i) {
            if (i < mine && t_first + i * (NW * kStage) + lane < pc.len) {
                nk = *pk;
                nrho = *pr;
                nv = *pv;
            }
            pk += NW * kStage;
            pr += NW * kStage;
            pv += NW * kStage;
        };
#pragma unroll
        for (int k = 0; k < C::NST - 1; ++k) issue(k);
        norms(0);
        // ---- query fragments of the slice
        const uint2 *qf = a.frag + ((int64_t)pc.slice * rblks + rblk) * (NT * C::KS * 32);
        uint2 breg[C::BREG ? NT * C::KS : 1];
        if constexpr (C::BREG) {
#pragma unroll
            for (int k = 0; k < NT * C::KS; ++k) breg[k] = qf[k * 32 + lane];
        } else {
            for (int e = tid; e < NT * C::KS * 32; e += NW * 32) bfrag[e] = qf[e];
        }
        float f[NT], N[NT], l[NT], o[C::NO][C::TILES][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = 4 * t + t4;
            f[t] = row < nr ? a.fscale[ragged_row(a.c, pc.slice, r0 + row)] : 0.f;
            // Rows that fill the block hold whatever the scratch held.  They stay in their own columns, and
            // with this reference they never call for a rescaling, which moves all rows' references.
            N[t] = row < nr ? -FLT_MAX : INFINITY;
            l[t] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < C::NO; ++t)
#pragma unroll
            for (int i = 0; i < C::TILES; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[t][i][k] = 0.f;
        if constexpr (!C::BREG) __syncthreads();

        uint32_t slot = 0;
        for (int i_st = 0; i_st < mine; ++i_st) {
            __syncwarp();  // every lane has read the stage whose slot is filled next, and its norms
            issue(i_st + C::NST - 1);
            const int t0 = t_first + i_st * (NW * kStage);
            {
                // kn, (-rho, -rho), log2 ||v||, 1 / ||v|| (negative where ||v|| is 0); tokens past the
                // end get y = -inf
                const bool there = t0 + lane < pc.len;
                const float v = f16_bits_to_f32(nv), vc = fmaxf(v, kMinNorm);
                float4 x;
                x.x = there ? f16_bits_to_f32(nk) : 0.f;
                const uint32_t neg = there ? (uint32_t)(nrho ^ 0x8000u) : 0u;
                x.y = __uint_as_float(neg | (neg << 16));
                x.z = !there ? -INFINITY : v != v ? v : F32 ? log2f(vc) : lg2(vc);
                x.w = v == 0.f ? -1.f / vc : 1.f / vc;
                meta[lane] = x;
            }
            norms(i_st + 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(C::NST - 1) : "memory");
            __syncwarp();
            const uint8_t *st = ring + slot;
            slot = slot == (C::NST - 1) * C::STAGE ? 0 : slot + C::STAGE;
            const uint32_t *skc = (const uint32_t *)st, *sks = (const uint32_t *)(st + C::OS),
                           *svc = (const uint32_t *)(st + C::OV);
            auto up = [&](uint32_t x, int kk) { return kk ? half_up(x, k16) : x; };
            auto bf = [&](int nt, int ks) -> uint2 {
                if constexpr (C::BREG) return breg[nt * C::KS + ks];
                else return bfrag[(nt * C::KS + ks) * 32 + lane];
            };
#pragma unroll
            for (int blk = 0; blk < 2; ++blk) {
                // ---- scores of 16 tokens: this lane's are tA and tA + 8, of rows 4 nt + t4
                const int tA = 16 * blk + gid;
                const float4 mA = meta[tA], mB = meta[tA + 8];
                float acc[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
#pragma unroll
                for (int gg = 0; gg < C::NG; ++gg) {
                    const int g = D >= 128 ? t4 * C::NG + gg : t4 >> 1;
                    uint32_t wA[KB], wB[KB];
#pragma unroll
                    for (int p = 0; p < KB; ++p) {
                        wA[p] = skc[tA * C::KWPT + g * KB + p];
                        wB[p] = skc[(tA + 8) * C::KWPT + g * KB + p];
                    }
                    if constexpr (KB == 1) {
                        constexpr int PR = D >= 128 ? 16 : 8;
                        if (D < 128) {
                            wA[0] <<= 8 * (1 - (t4 & 1));
                            wB[0] <<= 8 * (1 - (t4 & 1));
                        }
                        const uint32_t one = (T->kh[1] ^ 0x8000u) * 0x10001u;  // (-c, -c)
#pragma unroll
                        for (int k = 0; k < PR / 2; ++k) {
                            const uint32_t a0 = ((wA[0] << (PR - 1 - 2 * k)) & 0x80008000u) ^ one;
                            const uint32_t a1 = ((wB[0] << (PR - 1 - 2 * k)) & 0x80008000u) ^ one;
                            const uint32_t a2 = ((wA[0] << (PR - 2 - 2 * k)) & 0x80008000u) ^ one;
                            const uint32_t a3 = ((wB[0] << (PR - 2 - 2 * k)) & 0x80008000u) ^ one;
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma(acc[t], a0, a1, a2, a3, bf(t, gg * (PR / 2) + k));
                        }
                    } else if constexpr (KB == 2) {
                        constexpr int NP = D >= 128 ? 8 : 4;
                        const int sh = D >= 128 ? 0 : 4 * (t4 & 1);
                        Pairs2 sA(wA[0] >> sh, wA[KB - 1] >> sh), sB(wB[0] >> sh, wB[KB - 1] >> sh);
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            const uint32_t uA = sA.selector(i), uB = sB.selector(i);
                            const uint32_t a0 = prmt(kp0, kp1, uA), a1 = prmt(kp0, kp1, uB);
                            const uint32_t a2 = prmt(kp0, kp1, half_up(uA, k16)), a3 = prmt(kp0, kp1, half_up(uB, k16));
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma(acc[t], a0, a1, a2, a3, bf(t, gg * NP + i));
                        }
                    } else {
                        if (D < 128) {
#pragma unroll
                            for (int p = 0; p < KB; ++p) {
                                wA[p] >>= 2 * (t4 & 1);
                                wB[p] >>= 2 * (t4 & 1);
                            }
                        }
                        uint32_t xA[4], xB[4];
                        selectors<KB>(wA, xA);
                        selectors<KB>(wB, xB);
#pragma unroll
                        for (int i = 0; i < C::NI; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int ks = (gg * C::NI + i) * 2 + h;
                                uint32_t a0, a1, a2, a3;
                                look_up(kh, xA[i] >> (16 * h), 0u, a0, a2);
                                look_up(kh, xB[i] >> (16 * h), 0u, a1, a3);
#pragma unroll
                                for (int t = 0; t < NT; ++t) mma(acc[t], a0, a1, a2, a3, bf(t, ks));
                                if constexpr (KB == 3 && F32) {
                                    look_up(kl, xA[i] >> (16 * h), 0u, a0, a2);
                                    look_up(kl, xB[i] >> (16 * h), 0u, a1, a3);
#pragma unroll
                                    for (int t = 0; t < NT; ++t) mma(acc[t], a0, a1, a2, a3, bf(t, ks));
                                }
                            }
                    }
                }
                {
                    const int sh = 16 - C::PW - (t4 % C::LPW) * C::PW;
                    const uint32_t sA = sks[tA * C::SW + t4 / C::LPW] << sh;
                    const uint32_t sB = sks[(tA + 8) * C::SW + t4 / C::LPW] << sh;
                    const uint32_t nA = __float_as_uint(mA.y), nB = __float_as_uint(mB.y);
#pragma unroll
                    for (int k = 0; k < C::PW / 2; ++k) {
                        const uint32_t a0 = ((sA << (C::PW - 1 - 2 * k)) & 0x80008000u) ^ nA;
                        const uint32_t a1 = ((sB << (C::PW - 1 - 2 * k)) & 0x80008000u) ^ nB;
                        const uint32_t a2 = ((sA << (C::PW - 2 - 2 * k)) & 0x80008000u) ^ nA;
                        const uint32_t a3 = ((sB << (C::PW - 2 - 2 * k)) & 0x80008000u) ^ nB;
#pragma unroll
                        for (int t = 0; t < NT; ++t) mma(acc[t], a0, a1, a2, a3, bf(t, C::KC + k));
                    }
                }
                // ---- weights
                float yA[NT], yB[NT];
                bool over = false;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float zA = (acc[t][0] + acc[t][1]) * (mA.x * f[t]);
                    const float zB = (acc[t][2] + acc[t][3]) * (mB.x * f[t]);
                    if (a.zbuf && 4 * t + t4 < nr) {
                        float *zp = a.zbuf + ((int64_t)pc.slice * a.c.rows + r0 + 4 * t + t4) * a.c.stride + t0 + tA;
                        if (t0 + tA < pc.len) zp[0] = zA;
                        if (t0 + tA + 8 < pc.len) zp[8] = zB;
                    }
                    yA[t] = zA + mA.z;
                    yB[t] = zB + mB.z;
                    over |= fmaxf(yA[t], yB[t]) > N[t] + kHeadroom;
                }
                if (__any_sync(kFull, over)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float mx = fmaxf(yA[t], yB[t]);
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                        mx = fmaxf(mx - kTopWeight, N[t]);
                        const float sc = exp2f(N[t] - mx);
                        N[t] = mx;
                        l[t] *= sc;
#pragma unroll
                        for (int i = 0; i < C::TILES; ++i) {
                            if constexpr (F32 || NT == 1) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) o[F32 ? t : 0][i][k] *= sc;
                            } else {
                                o[0][i][t] *= sc;
                                o[0][i][2 + t] *= sc;
                            }
                        }
                    }
                }
                // B of the value product: column 2 t4 + c of this lane is (row t4; hi, lo) when F32 or
                // with one row tile (lo = 0 then), and row 4 c + t4 with two
                uint2 pb[C::NO];
                {
                    float pA[NT], pB[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        pA[t] = ex2(yA[t] - N[t]);
                        pB[t] = ex2(yB[t] - N[t]);
                        l[t] = fmaf(pA[t], fabsf(mA.w), l[t]);
                        l[t] = fmaf(pB[t], fabsf(mB.w), l[t]);
                        pA[t] = mA.w < 0.f ? 0.f : pA[t];
                        pB[t] = mB.w < 0.f ? 0.f : pB[t];
                    }
#pragma unroll
                    for (int t = 0; t < C::NO; ++t) {
                        __half2 hA, hB;
                        if constexpr (F32) {
                            const __half uA = __float2half_rn(pA[t]), uB = __float2half_rn(pB[t]);
                            hA = __halves2half2(uA, __float2half_rn(pA[t] - __half2float(uA)));
                            hB = __halves2half2(uB, __float2half_rn(pB[t] - __half2float(uB)));
                        } else {
                            hA = __floats2half2_rn(pA[0], NT > 1 ? pA[NT - 1] : 0.f);
                            hB = __floats2half2_rn(pB[0], NT > 1 ? pB[NT - 1] : 0.f);
                        }
                        pb[t].x = transpose8x8(*(uint32_t *)&hA);
                        pb[t].y = transpose8x8(*(uint32_t *)&hB);
                    }
                }
                // ---- value sums: tokens 2 t4, 2 t4 + 1 (AB) and 8 + 2 t4, 9 + 2 t4 (CD) of the block
                const int tV = 16 * blk + 2 * t4;
                uint32_t wv[4][VB];
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int p = 0; p < VB; ++p)
                        wv[k][p] = svc[(tV + (k & 1) + 8 * (k >> 1)) * C::VWPT + vg * VB + p];
                if constexpr (VB == 4) {  // magnitude selectors: the code's low bits, inverted below the middle
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int p = 0; p < 3; ++p) wv[k][p] = ~(wv[k][p] ^ wv[k][3]);
                }
#pragma unroll
                for (int hv = 0; hv < C::VH; ++hv) {
                    // two tokens a byte: four bits of each, of one half of every byte of the words
                    uint32_t y[2][VB];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int p = 0; p < VB; ++p) {
                            const int hs = D >= 256 ? hv : vhalf;
                            y[k][p] = pick(wv[2 * k][p] >> (4 * hs), wv[2 * k + 1][p] << (4 - 4 * hs), 0x0F0F0F0Fu);
                            if (D < 128) y[k][p] >>= 2 * (gid & 1);
                        }
                    uint32_t x[2][4];
                    selectors<VN>(y[0], x[0]);
                    selectors<VN>(y[1], x[1]);
#pragma unroll
                    for (int i = 0; i < C::NI; ++i) {
                        uint32_t sg[2] = {0, 0};
                        if constexpr (VB == 4) {
                            sg[0] = (y[0][3] >> i) & 0x11111111u;
                            sg[1] = (y[1][3] >> i) & 0x11111111u;
                        }
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk) {
                            const int tile = (hv * C::NI + i) * 2 + kk;
                            const uint32_t f0 = VB == 4 ? prmt(0x80u, 0u, sg[0] >> (16 * kk)) : 0u;
                            const uint32_t f1 = VB == 4 ? prmt(0x80u, 0u, sg[1] >> (16 * kk)) : 0u;
                            uint32_t a0, a1, a2, a3;
                            look_up(vh, up(x[0][i], kk), f0, a0, a1);
                            look_up(vh, up(x[1][i], kk), f1, a2, a3);
#pragma unroll
                            for (int t = 0; t < C::NO; ++t) mma(o[t][tile], a0, a1, a2, a3, pb[t]);
                            if constexpr (F32) {
                                look_up(vl, up(x[0][i], kk), f0, a0, a1);
                                look_up(vl, up(x[1][i], kk), f1, a2, a3);
#pragma unroll
                                for (int t = 0; t < C::NO; ++t) mma(o[t][tile], a0, a1, a2, a3, pb[t]);
                            }
                        }
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();  // every warp is done with its ring

        // ---- the warps' results meet: [warp][row](N, l), then [warp][row][d]
        float *mo = mrg + NW * C::ROWS * 2;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float s = l[t];
            s += __shfl_xor_sync(kFull, s, 4);
            s += __shfl_xor_sync(kFull, s, 8);
            s += __shfl_xor_sync(kFull, s, 16);
            if (gid == 0) {
                mrg[(warp * C::ROWS + 4 * t + t4) * 2] = N[t];
                mrg[(warp * C::ROWS + 4 * t + t4) * 2 + 1] = s;
            }
        }
#pragma unroll
        for (int hv = 0; hv < C::VH; ++hv)
#pragma unroll
            for (int i = 0; i < C::NI; ++i)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int up = 0; up < 2; ++up) {
                        const int tile = (hv * C::NI + i) * 2 + kk;
                        const int j = 32 * vg + 16 * kk + 8 * up + 4 * (D >= 256 ? hv : vhalf) + i +
                                      (D >= 128 ? 0 : 2 * (gid & 1));
                        float *at = mo + (size_t)warp * C::ROWS * D + j;
                        if constexpr (F32 || NT == 1) {
#pragma unroll
                            for (int t = 0; t < C::NO; ++t)
                                at[(4 * t + t4) * D] = o[t][tile][2 * up] + o[t][tile][2 * up + 1];
                        } else {
                            at[t4 * D] = o[0][tile][2 * up];
                            at[(4 + t4) * D] = o[0][tile][2 * up + 1];
                        }
                    }
        __syncthreads();
        for (int e = tid; e < nr * D; e += NW * 32) {
            const int r = e / D, j = e % D;
            float Nm = -FLT_MAX;
#pragma unroll
            for (int u = 0; u < NW; ++u) Nm = fmaxf(Nm, mrg[(u * C::ROWS + r) * 2]);
            float s = 0.f, L = 0.f;
#pragma unroll
            for (int u = 0; u < NW; ++u) {
                const float sc = exp2f(mrg[(u * C::ROWS + r) * 2] - Nm);
                s = fmaf(sc, mo[((size_t)u * C::ROWS + r) * D + j], s);
                L = fmaf(sc, mrg[(u * C::ROWS + r) * 2 + 1], L);
            }
            float *pp = a.part + ((int64_t)(cta + pc.slice) * a.c.rows + r0 + r) * partial_stride(D);
            pp[4 + j] = s * tau;
            if (j == 0) {
                pp[0] = Nm;
                pp[1] = L;
            }
        }
    }
}

template <int D, int KB, int NT, bool F32>
cudaError_t launch_one(const RaggedPair &a, cudaStream_t s) {
    using C = Cfg<D, KB, NT, F32>;
    cudaError_t e = allow_smem((const void *)ragged_mma_kernel<D, KB, NT, F32>, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(ragged_mma_kernel<D, KB, NT, F32>, (unsigned)a.total, NW * 32, C::SMEM, s, a);
}

// The instances of one head dimension; defined in tq_ragged_<D>.cu.
template <int D>
cudaError_t launch_dim(const RaggedPair &a, bool f32, int row_block, cudaStream_t s);

template <int D, int KB>
cudaError_t launch_bits(const RaggedPair &a, bool f32, int row_block, cudaStream_t s) {
    if constexpr (D < 256) {
        if (row_block == 8) return f32 ? launch_one<D, KB, 2, true>(a, s) : launch_one<D, KB, 2, false>(a, s);
    }
    return f32 ? launch_one<D, KB, 1, true>(a, s) : launch_one<D, KB, 1, false>(a, s);
}

#define TQ_RAGGED_DIM(D)                                                                              \
    template <>                                                                                       \
    cudaError_t launch_dim<D>(const RaggedPair &a, bool f32, int row_block, cudaStream_t s) {         \
        switch (a.a[0].P.kbeta) {                                                                     \
            case 1: return launch_bits<D, 1>(a, f32, row_block, s);                                   \
            case 2: return launch_bits<D, 2>(a, f32, row_block, s);                                   \
            case 3: return launch_bits<D, 3>(a, f32, row_block, s);                                   \
            default: return cudaErrorInvalidValue;                                                    \
        }                                                                                             \
    }

}  // namespace ragged
}  // namespace tq
