// tq_serve.cu -- what surrounds the attention kernels of tq_attend_shared and tq_attend_weigh: the
// preparation of the query rows and operand tables, the merge of the partial results and the
// addition of the softmax weights; and the plain kernel for the shapes without a tensor-core one.
#include <float.h>
#include <math.h>

#include <atomic>
#include <cstring>

#include <cuda_bf16.h>

#include "tq_f32x2.cuh"
#include "tq_launch.cuh"
#include "tq_serve.cuh"

namespace tq {

namespace {

// ------------------------------------------------------------------ preparation

constexpr int kPrepThreads = 256;
constexpr int kPrepCols = 64;  // operands of a CTA; 4 threads share one, a quarter of the sum each

struct PrepArgs {
    Prepared P;
    const void *q;
    tq_dtype dtype;
    int64_t rows;
    int rows_in, Hkv;
    float scale;
    float *qprep, *fscale;
    // fragments of the ragged tensor-core kernel, own caches and prefix (null: not wanted)
    uint16_t *own_frag, *pre_frag;
    int row_block, prefix_blocks;
    uint16_t *qrows;  // rows of the many-row prefix kernel (null: not wanted)
    // contexts: the caller's lengths and the prefix, as the division reads them
    const int32_t *lens;
    int B;
    int64_t t_cap, t_prefix;
    int32_t *len_own;   // [B], then [1] of the prefix
    int64_t *cum_own;   // [B + 1], then [2] of the prefix
    int32_t *dev_status;
};

__device__ __forceinline__ float load_elem(const void *p, tq_dtype t, int64_t i) {
    if (t == TQ_F16) return __half2float(((const __half *)p)[i]);
    if (t == TQ_BF16) return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
    return ((const float *)p)[i];
}

// Sums over this thread's quarter of the coordinates j of w[j ld] x[j][row], two rows a number: the
// first of w's loads are in v already, the others go CH at a time.
constexpr int kPrepFirst = 32;
template <int CH, int ROWS>
__device__ __forceinline__ void quarter_dot(float (&v)[kPrepFirst], const float *w, int64_t ld, const float *x,
                                            int count, f2 (&acc)[ROWS / 2]) {
#pragma unroll 1
    for (int j0 = 0; j0 < count; j0 += CH) {
        if (j0 > 0) {
#pragma unroll
            for (int k = 0; k < CH; ++k) v[k] = w[(j0 + k) * ld];
        }
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            const f2 vv = pack2(v[k], v[k]);
#pragma unroll
            for (int r = 0; r < ROWS / 4; ++r) {
                const ulonglong2 y = *(const ulonglong2 *)(x + (j0 + k) * ROWS + 4 * r);
                acc[2 * r] = fma2(vv, y.x, acc[2 * r]);
                acc[2 * r + 1] = fma2(vv, y.y, acc[2 * r + 1]);
            }
        }
    }
}

// An operand split hi + lo into the fragments of its row: lo goes to the next column's lane, 4 lanes on.
__device__ __forceinline__ void put_split(uint16_t *at, float v) {
    const __half hi = __float2half_rn(v);
    at[0] = __half_as_ushort(hi);
    at[16] = __half_as_ushort(__float2half_rn(v - __half2float(hi)));
}

// Where the fragments of row r of a slice (of `blocks` blocks of `block` rows) begin.
__device__ __forceinline__ int64_t frag_row(int64_t slice, int blocks, int block, int d, int r) {
    const int ks_all = d / 16 + d / 32, blk = r / block, nt = (r - blk * block) >> 2;
    return (((slice * blocks + blk) * (block >> 2) + nt) * ks_all * 32 + 8 * (r & 3)) * 4;
}

// q_rot = R q and sq = S q in fp32, scaled (see the header), as the attention kernels take them.
// A CTA computes kPrepCols operands of kPrepRows rows (8, or 16 when there are many): latency bound at
// a few rows (three dependent steps: the rows, the loads of R^T in flight together, the exchange of
// the quarters; 4.3 us), and at many by its reads of R^T and S^T from L2 (d = 128: 9.4 us for 1024
// rows, 14 us for 2048 in blocks of 16).  The last CTA lays out the contexts instead.
template <int kPrepRows>
__global__ void __launch_bounds__(kPrepThreads, 3) serve_prep_kernel(PrepArgs a) {
    constexpr int kQuads = kPrepRows / 4, kParts = kPrepThreads / 32 / kQuads;
    grid_go();
    extern __shared__ __align__(16) float qT[];  // [d][kPrepRows]
    __shared__ float red[4][kPrepRows][kPrepCols];
    __shared__ float rmax[kParts][kPrepRows];
    __shared__ int64_t wsum[kPrepThreads / 32];
    const Prepared &P = a.P;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int d = P.d, m = P.m, n = d + m;
    if (blockIdx.x == gridDim.x - 1) {
        // clamped lengths and the stages before each sequence (a block-wide scan, 256 at a time)
        int64_t before = 0;
        for (int b0 = 0; b0 < a.B; b0 += kPrepThreads) {
            const int b = b0 + tid;
            int64_t len = 0;
            if (b < a.B && a.lens) {
                len = a.lens[b];
                if (len < 0 || len > a.t_cap) {
                    if (a.dev_status) *a.dev_status = TQ_ERR_INVALID_ARG;
                    len = len < 0 ? 0 : a.t_cap;
                }
                a.len_own[b] = (int32_t)len;
            }
            const int64_t st = counted_stages(len);
            int64_t x = st;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(kFull, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) wsum[warp] = x;
            __syncthreads();
            int64_t off = before, all = 0;
            for (int w = 0; w < kPrepThreads / 32; ++w) {
                if (w < warp) off += wsum[w];
                all += wsum[w];
            }
            if (b < a.B) a.cum_own[b] = off + x - st;
            before += all;
            __syncthreads();
        }
        if (tid == 0) {
            a.cum_own[a.B] = before;
            a.len_own[a.B] = (int32_t)a.t_prefix;
            a.cum_own[a.B + 1] = 0;
            a.cum_own[a.B + 2] = counted_stages(a.t_prefix);
        }
        return;
    }
    const int cols = (n + kPrepCols - 1) / kPrepCols;
    const int64_t r0 = (int64_t)(blockIdx.x / cols) * kPrepRows;
    const int nr = (int)min((int64_t)kPrepRows, a.rows - r0);
    const int cb = (blockIdx.x % cols) * kPrepCols;
    // this thread's operand c and quarter of the sum; the loads that need no row first
    const int c = cb + (tid & 63), q4 = tid >> 6, part = d >> 2;
    const int64_t ld = c < d ? d : m;
    const float *w = (c < d ? P.RT + c : P.ST + (c - d)) + q4 * part * ld;
    float v[kPrepFirst];
#pragma unroll
    for (int k = 0; k < kPrepFirst; ++k) v[k] = c < n && k < part ? w[k * ld] : 0.f;
    // ... and all that does not depend on the sums: the scales and the places of this warp's results
    const float qbound = P.serve->qbound, sigma = P.serve->sigma, gamma = sqrtf(1.5707963267948966f) / (float)m;
    int place[2] = {0, 0};  // of operands cb + lane and + 32, in 16-bit numbers from the row's beginning
    if (a.own_frag || a.pre_frag) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int oc = cb + lane + 32 * k;
            const int at = d == 64    ? frag_place(64, P.kbeta, oc)
                           : d == 128 ? frag_place(128, P.kbeta, oc)
                                      : frag_place(256, P.kbeta, oc);
            place[k] = ((at >> 4) * 32 + ((at >> 2) & 3)) * 4 + (at & 3);
        }
    }
    {  // a warp four rows (stored together, for fewer bank conflicts), part of their coordinates
        const int rq = 4 * (warp % kQuads), jp = warp / kQuads;
        float mx[4] = {};
        for (int j = 32 * jp + lane; j < d; j += 32 * kParts) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = rq + k < nr ? load_elem(a.q, a.dtype, (r0 + rq + k) * d + j) : 0.f;
            *(float4 *)(qT + j * kPrepRows + rq) = make_float4(x[0], x[1], x[2], x[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], fabsf(x[k]));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float x = warp_max(mx[k]);
            if (lane == 0) rmax[jp][rq + k] = x;
        }
    }
    __syncthreads();
    {
        f2 acc[kPrepRows / 2];
#pragma unroll
        for (int r = 0; r < kPrepRows / 2; ++r) acc[r] = pack2(0.f, 0.f);
        if (c < n) {
            const float *x = qT + q4 * part * kPrepRows;
            if (part >= 32) quarter_dot<32, kPrepRows>(v, w, ld, x, part, acc);
            else quarter_dot<8, kPrepRows>(v, w, ld, x, part, acc);
        }
#pragma unroll
        for (int r = 0; r < kPrepRows / 2; ++r) unpack2(acc[r], red[q4][2 * r][tid & 63], red[q4][2 * r + 1][tid & 63]);
    }
    __syncthreads();
#pragma unroll 1
    for (int r = warp; r < nr; r += kPrepThreads / 32) {
        const int row = (int)r0 + r, slice = row / a.rows_in, rr = row - slice * a.rows_in;
        const int b = slice / a.Hkv, kv = slice - b * a.Hkv;
        const int pr = b * a.rows_in + rr;
        float qmax = rmax[0][r];
#pragma unroll
        for (int k = 1; k < kParts; ++k) qmax = fmaxf(qmax, rmax[k][r]);
        const float bound = qmax * qbound * sqrtf((float)d);
        const int e = (bound > 0.f && bound < INFINITY) ? min(max(ilogbf(bound) - 14, -126), 126) : 0;
        const float down = exp2f((float)-e);
        if (lane == 0 && cb == 0) a.fscale[row] = a.scale * kLog2eF * exp2f((float)e);
        uint16_t *own = nullptr, *pre = nullptr;
        if (a.own_frag)
            own = a.own_frag + frag_row(slice, (a.rows_in + a.row_block - 1) / a.row_block, a.row_block, d, rr);
        if (a.pre_frag) pre = a.pre_frag + frag_row(kv, a.prefix_blocks, a.row_block, d, pr);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int cc = lane + 32 * k, oc = cb + cc;
            if (oc >= n) break;
            const float x = ((red[0][r][cc] + red[1][r][cc]) + (red[2][r][cc] + red[3][r][cc])) *
                            ((oc < d ? sigma : gamma) * down);
            if (a.qprep) a.qprep[(int64_t)row * n + oc] = x;
            if (own) put_split(own + place[k], x);
            if (pre) put_split(pre + place[k], x);
            if (a.qrows)
                a.qrows[((int64_t)kv * a.B * a.rows_in + pr) * n + prefix_column(d, oc)] =
                    __half_as_ushort(__float2half_rn(x));
        }
    }
}

// ------------------------------------------------------------------ the plain kernel

constexpr int kPlThreads = 128;
constexpr int kPlRows = 4;
constexpr int kPlTile = 128;  // tokens per step, one per thread
constexpr int kPlCoord = kMaxDim / kPlThreads;

// One CTA: its pieces of the slices, for kPlRows query rows (blockIdx.y).  Scores with a thread a
// token, online softmax, then the weighted value sum with a thread a coordinate; fp32 throughout.
__global__ void __launch_bounds__(kPlThreads) ragged_plain_kernel(RaggedArgs a) {
    grid_go();  // (launched behind a complete preparation)
    extern __shared__ __align__(16) float sm[];  // qs[(d + m)][kPlRows], ps[kPlRows][kPlTile]
    __shared__ float kcen[kMaxLevels], vcen[kMaxLevels];
    __shared__ float red[kPlRows][kPlThreads / 32], rowN[kPlRows], rowA[kPlRows];
    const Prepared &P = a.P;
    const int d = P.d, m = P.m, n = d + m, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *qs = sm, *ps = sm + n * kPlRows;
    if (tid < kMaxLevels) {
        kcen[tid] = P.cb->kc[tid] / P.serve->sigma;
        vcen[tid] = P.cb->vc[tid];
    }
    const int64_t total = ragged_total(a.c);
    const int64_t w1 = cta_first(total, a.c.ctas, blockIdx.x + 1);
    const int r0 = blockIdx.y * kPlRows, nr = min(kPlRows, a.c.rows - r0);
    const int kw = P.kbeta * (d >> 5), sw = m >> 5, vw = P.vbeta * (d >> 5);
    Piece pc;
    for (int64_t w = cta_first(total, a.c.ctas, blockIdx.x); w < w1; w += pc.counted) {
        pc = piece_at(a.c, w, w1);
        const int64_t rec0 = pc.slice * a.c.stride;
        const int t_end = (int)min((int64_t)pc.len, pc.s1 * kStage);
        __syncthreads();
        for (int e = tid; e < n * kPlRows; e += kPlThreads) {
            const int r = e / n, c = e - r * n;
            qs[c * kPlRows + r] = r < nr ? a.qprep[ragged_row(a.c, pc.slice, r0 + r) * n + c] : 0.f;
        }
        float f[kPlRows], l[kPlRows], o[kPlRows][kPlCoord];
#pragma unroll
        for (int r = 0; r < kPlRows; ++r) {
            f[r] = r < nr ? a.fscale[ragged_row(a.c, pc.slice, r0 + r)] : 0.f;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < kPlCoord; ++c) o[r][c] = 0.f;
        }
        // (a finite first reference: NaN, which a maximum leaves out, and -infinity make their own weights)
        if (tid < kPlRows) rowN[tid] = -FLT_MAX;
        __syncthreads();
        for (int t0 = (int)(pc.s0 * kStage); t0 < t_end; t0 += kPlTile) {
            const int t = t0 + tid, nt = min(kPlTile, t_end - t0);
            float y[kPlRows], rv = 0.f;
#pragma unroll
            for (int r = 0; r < kPlRows; ++r) y[r] = -INFINITY;
            if (tid < nt) {
                const int64_t rec = rec0 + t;
                float acc[kPlRows] = {}, acc2[kPlRows] = {};
                for (int g = 0; g < (d >> 5); ++g) {
                    uint32_t wd[4] = {0, 0, 0, 0};
                    for (int p = 0; p < P.kbeta; ++p) wd[p] = a.c.kcodes[rec * kw + g * P.kbeta + p];
                    for (int b = 0; b < 32; ++b) {
                        const int idx = ((wd[0] >> b) & 1) | (((wd[1] >> b) & 1) << 1) | (((wd[2] >> b) & 1) << 2);
                        const float c = kcen[idx];
                        const float4 q4 = *(const float4 *)(qs + (32 * g + b) * kPlRows);
                        acc[0] = fmaf(q4.x, c, acc[0]);
                        acc[1] = fmaf(q4.y, c, acc[1]);
                        acc[2] = fmaf(q4.z, c, acc[2]);
                        acc[3] = fmaf(q4.w, c, acc[3]);
                    }
                }
                for (int g = 0; g < sw; ++g) {
                    const uint32_t wd = a.c.ksigns[rec * sw + g];
                    for (int b = 0; b < 32; ++b) {
                        const float c = (wd >> b) & 1 ? 1.f : -1.f;
                        const float4 q4 = *(const float4 *)(qs + (d + 32 * g + b) * kPlRows);
                        acc2[0] = fmaf(q4.x, c, acc2[0]);
                        acc2[1] = fmaf(q4.y, c, acc2[1]);
                        acc2[2] = fmaf(q4.z, c, acc2[2]);
                        acc2[3] = fmaf(q4.w, c, acc2[3]);
                    }
                }
                const float kn = f16_bits_to_f32(a.c.knorm[rec]), rho = f16_bits_to_f32(a.c.krnorm[rec]);
                const float vr = f16_bits_to_f32(a.c.vnorm[rec]), vn = fmaxf(vr, kMinNorm);
                const float lv = vr != vr ? vr : log2f(vn);
                rv = 1.f / vn;
#pragma unroll
                for (int r = 0; r < kPlRows; ++r) {
                    const float z = f[r] * kn * fmaf(rho, acc2[r], acc[r]);
                    if (a.zbuf && r < nr) a.zbuf[((int64_t)pc.slice * a.c.rows + r0 + r) * a.c.stride + t] = z;
                    y[r] = z + lv;
                }
            }
            // the rows' maxima, and the references
#pragma unroll
            for (int r = 0; r < kPlRows; ++r) {
                const float mx = warp_max(y[r]);
                if (lane == 0) red[r][warp] = mx;
            }
            __syncthreads();
            if (tid < kPlRows) {
                const float old = rowN[tid];
                float mx = old;
                for (int u = 0; u < kPlThreads / 32; ++u) mx = fmaxf(mx, red[tid][u]);
                rowN[tid] = mx;
                rowA[tid] = exp2f(old - mx);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kPlRows; ++r) {
                const float w8 = exp2f(y[r] - rowN[r]);
                ps[r * kPlTile + tid] = w8;
                l[r] = fmaf(l[r], rowA[r], w8 * rv);
#pragma unroll
                for (int c = 0; c < kPlCoord; ++c) o[r][c] *= rowA[r];
            }
            __syncthreads();
            for (int u = 0; u < nt; ++u) {
                const int64_t rec = rec0 + t0 + u;
                const bool zero = (a.c.vnorm[rec] & 0x7FFF) == 0;
                float w8[kPlRows];
#pragma unroll
                for (int r = 0; r < kPlRows; ++r) w8[r] = ps[r * kPlTile + u];
#pragma unroll
                for (int c = 0; c < kPlCoord; ++c) {
                    const int j = tid + kPlThreads * c;
                    if (j < d) {
                        const uint32_t *vp = a.c.vcodes + rec * vw + (j >> 5) * P.vbeta;
                        int idx = 0;
                        for (int p = 0; p < P.vbeta; ++p) idx |= ((vp[p] >> (j & 31)) & 1u) << p;
                        const float x = zero ? 0.f : vcen[idx];
#pragma unroll
                        for (int r = 0; r < kPlRows; ++r) o[r][c] = fmaf(w8[r], x, o[r][c]);
                    }
                }
            }
        }
        // the piece's partial
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kPlRows; ++r) {
            const float s = warp_sum(l[r]);
            if (lane == 0) red[r][warp] = s;
        }
        __syncthreads();
        for (int r = 0; r < nr; ++r) {
            float *pp = a.part + ((int64_t)(blockIdx.x + pc.slice) * a.c.rows + r0 + r) * partial_stride(d);
            if (tid == 0) {
                float s = 0.f;
                for (int u = 0; u < kPlThreads / 32; ++u) s += red[r][u];
                pp[0] = rowN[r];
                pp[1] = s;
            }
        }
#pragma unroll
        for (int r = 0; r < kPlRows; ++r) {
            if (r >= nr) break;
            float *pp = a.part + ((int64_t)(blockIdx.x + pc.slice) * a.c.rows + r0 + r) * partial_stride(d);
#pragma unroll
            for (int c = 0; c < kPlCoord; ++c) {
                const int j = tid + kPlThreads * c;
                if (j < d) pp[4 + j] = o[r][c];
            }
        }
    }
}

// ------------------------------------------------------------------ merge and weights

constexpr int kFinThreads = 512;
constexpr int kMgParts = 4;      // partials of a warp on their way at once
constexpr int kWtTokens = 1024;  // tokens of a weighing CTA
constexpr int kWtRows = 64;      // rows whose normalisers it holds at a time

struct FinishArgs {
    Prepared P;
    RaggedCache own, prefix;
    const float *own_part, *pre_part;
    int tc_splits;  // > 0: the prefix's partials are those of the many-row kernel
    int64_t rows;
    int rows_in, Hkv;
    tq_dtype dtype;
    void *out;
    unsigned merge_ctas;  // the CTAs behind them weigh
    const float *zbuf;
    float *weights;
    int chunks;  // weighing CTAs of a slice
    float *lse;  // log2 of the rows' normalisers, for weighing CTAs behind the merge (null: they take their own)
    int csplit;  // merging CTAs of a block of rows, a part of the columns each
};

// Partials of one row and cache: (N, l, -, -, o[d]) at base + i * step.
struct Parts {
    const float *base;
    int64_t step;
    int n;
};

__device__ __forceinline__ Parts parts_of(const RaggedCache &c, const float *part, int slice, int r, int ps) {
    Parts g = {nullptr, 0, 0};
    int c0, c1;
    if (c.slices > 0 && slice_ctas(c, slice, &c0, &c1)) {
        g.base = part + ((int64_t)(c0 + slice) * c.rows + r) * ps;
        g.step = (int64_t)c.rows * ps;
        g.n = c1 - c0 + 1;
    }
    return g;
}

// log2 of the sum of 2^z over a row's partials; +infinity when there is nothing.  A whole warp.
__device__ __forceinline__ float log_sum(const Parts &g, int lane) {
    float mx = -INFINITY, s = 0.f;
    for (int i = lane; i < g.n; i += 32) {
        const float2 h = *(const float2 *)(g.base + i * g.step);
        const float up = fmaxf(mx, h.x);
        s = (up == -INFINITY ? 0.f : s * exp2f(mx - up)) + (h.x == -INFINITY ? 0.f : h.y * exp2f(h.x - up));
        mx = up;
    }
    const float all = warp_max(mx);
    s = warp_sum(mx == -INFINITY ? 0.f : s * exp2f(mx - all));
    return s == 0.f ? INFINITY : all + log2f(s);
}

// weights[slice][t] += sum over the slice's rows, in ascending order, of 2^(z - log2 of the row's
// normaliser), kWtTokens tokens a CTA; bound by the 4 rows + 8 bytes a token that it moves.
template <int THREADS, bool LSE>
__device__ __forceinline__ void weigh_tokens(const FinishArgs &a, unsigned id, float *lse) {
    constexpr int PT = kWtTokens / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = partial_stride(a.P.d);
    const int slice = (int)(id / a.chunks), R = a.own.rows;
    const int t0 = (int)(id - (unsigned)slice * a.chunks) * kWtTokens + tid;
    grid_wait();
    const int len = a.own.len[slice / a.own.per_seq];
    if (t0 - tid >= len) return;
    float s[PT] = {};
    for (int r0 = 0; r0 < R; r0 += kWtRows) {
        const int nr = min(kWtRows, R - r0);
        __syncthreads();
        for (int r = warp; r < nr; r += THREADS / 32) {
            const float x = LSE ? a.lse[(int64_t)slice * R + r0 + r]
                                : log_sum(parts_of(a.own, a.own_part, slice, r0 + r, ps), lane);
            if (lane == 0) lse[r] = x;
        }
        __syncthreads();
        const float *z = a.zbuf + ((int64_t)slice * R + r0) * a.own.stride + t0;
#pragma unroll 4
        for (int r = 0; r < nr; ++r)
#pragma unroll
            for (int k = 0; k < PT; ++k)
                if (t0 + k * THREADS < len) s[k] += exp2f(z[r * a.own.stride + k * THREADS] - lse[r]);
    }
#pragma unroll
    for (int k = 0; k < PT; ++k)
        if (t0 + k * THREADS < len) a.weights[slice * a.own.stride + t0 + k * THREADS] += s[k];
}

constexpr int kWtThreads = 256;

__global__ void __launch_bounds__(kWtThreads) serve_weigh_kernel(FinishArgs a) {
    __shared__ float lse[kWtRows];
    weigh_tokens<kWtThreads, true>(a, blockIdx.x, lse);
}

// Merging CTAs: out = R^T o / l for kMgRows rows.  16 / kMgRows warps a row add its partials, a share
// of the list each, in the order of the context and rescaled to their largest reference as they come;
// the rows are then rotated back together, several threads an output.  A row without a token is
// zero.  Latency bound at a few rows: the partials' and R's loads are issued before anything waits,
// and the code is kept short (it is fetched anew by every launch).
template <int kMgRows>
__global__ void __launch_bounds__(kFinThreads) serve_finish_kernel(FinishArgs a) {
    constexpr int kMgWarps = kFinThreads / 32 / kMgRows;
    grid_go();
    extern __shared__ __align__(16) float osm[];  // [kMgWarps][d][kMgRows]
    __shared__ __align__(16) float red[kFinThreads * kMgRows];
    __shared__ float2 head[kMgWarps][kMgRows];
    if (blockIdx.x >= a.merge_ctas) {
        weigh_tokens<kFinThreads, false>(a, blockIdx.x - a.merge_ctas, red);
        return;
    }
    const int d = a.P.d, ps = partial_stride(d), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)(blockIdx.x / a.csplit) * kMgRows;
    // this thread's column of R^T o (the first of several past 512 columns) and its share of the sum
    const int cw = d / a.csplit, c0 = (int)(blockIdx.x % a.csplit) * cw;
    const int ncol = min(cw, kFinThreads), ks = min(kFinThreads / ncol, d / 4), part = d / ks;
    const int share = tid / ncol, cl = tid - share * ncol, i0 = share * part;
    const bool works = share < ks;
    const float *w = a.P.R + (int64_t)i0 * d + c0 + cl;
    float first[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) first[k] = works && k < part ? w[(int64_t)k * d] : 0.f;
    {
        const int r4 = warp / kMgWarps, q = warp % kMgWarps;
        const int64_t row = row0 + r4;
        Parts g[2] = {{nullptr, 0, 0}, {nullptr, 0, 0}};
        grid_wait();
        if (row < a.rows) {  // where the row's partials are
            const int slice = (int)(row / a.rows_in), r = (int)(row - (int64_t)slice * a.rows_in);
            const int b = slice / a.Hkv, kv = slice - b * a.Hkv;
            if (a.tc_splits) {
                g[0].base = a.pre_part + ((int64_t)kv * a.prefix.rows + b * a.rows_in + r) * ps;
                g[0].step = (int64_t)a.Hkv * a.prefix.rows * ps;
                g[0].n = a.tc_splits;
            } else {
                g[0] = parts_of(a.prefix, a.pre_part, kv, b * a.rows_in + r, ps);
            }
            g[1] = parts_of(a.own, a.own_part, slice, r, ps);
        }
        // the prefix's partials, then the own ones, as one list; this warp's share of it
        const int all = g[0].n + g[1].n, per = (all + kMgWarps - 1) / kMgWarps;
        const int p0 = min(q * per, all), p1 = min(p0 + per, all);
        for (int j0 = 0; j0 < d; j0 += 256) {  // two groups of 128 coordinates at a time, four a lane of each
            const bool two = j0 + 128 < d;
            const int ja = min(j0 + 4 * lane, d - 4), jb = two ? j0 + 128 + 4 * lane : ja;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
            float N = -INFINITY, L = 0.f;
#pragma unroll 1
            for (int p = p0; p < p1; p += kMgParts) {
                float2 h[kMgParts];
                float4 ox[kMgParts], oy[kMgParts];
#pragma unroll
                for (int k = 0; k < kMgParts; ++k) {
                    // (past the end: the last partial again, with nothing in it)
                    const int e = min(p + k, p1 - 1);
                    const bool pre = e < g[0].n;
                    const float *at = pre ? g[0].base + e * g[0].step : g[1].base + (e - g[0].n) * g[1].step;
                    h[k] = *(const float2 *)at;
                    ox[k] = *(const float4 *)(at + 4 + ja);
                    oy[k] = *(const float4 *)(at + 4 + jb);
                    if (p + k >= p1) h[k].x = -INFINITY;
                }
                float up = N;
#pragma unroll
                for (int k = 0; k < kMgParts; ++k) up = fmaxf(up, h[k].x);
                const float sc = N == -INFINITY ? 0.f : exp2f(N - up);
                N = up;
                L *= sc;
                x = make_float4(x.x * sc, x.y * sc, x.z * sc, x.w * sc);
                y = make_float4(y.x * sc, y.y * sc, y.z * sc, y.w * sc);
#pragma unroll
                for (int k = 0; k < kMgParts; ++k) {
                    if (h[k].x == -INFINITY) continue;
                    const float f = exp2f(h[k].x - up);
                    L = fmaf(f, h[k].y, L);
                    x = make_float4(fmaf(f, ox[k].x, x.x), fmaf(f, ox[k].y, x.y), fmaf(f, ox[k].z, x.z),
                                    fmaf(f, ox[k].w, x.w));
                    y = make_float4(fmaf(f, oy[k].x, y.x), fmaf(f, oy[k].y, y.y), fmaf(f, oy[k].z, y.z),
                                    fmaf(f, oy[k].w, y.w));
                }
            }
            auto put = [&](int j, float4 v) {
                float *o = osm + ((size_t)q * d + j) * kMgRows + r4;
                o[0] = v.x;
                o[kMgRows] = v.y;
                o[2 * kMgRows] = v.z;
                o[3 * kMgRows] = v.w;
            };
            if (j0 + 4 * lane < d) put(ja, x);
            if (two) put(jb, y);
            if (j0 == 0 && lane == 0) head[q][r4] = make_float2(N, L);
        }
    }
    __syncthreads();
    // the shares of a row together, over the normaliser
    for (int e = tid; e < d * kMgRows; e += kFinThreads) {
        const int r = e % kMgRows;
        float N = -INFINITY, L = 0.f, v = 0.f;
#pragma unroll
        for (int q = 0; q < kMgWarps; ++q) N = fmaxf(N, head[q][r].x);
#pragma unroll
        for (int q = 0; q < kMgWarps; ++q) {
            const float2 h = head[q][r];
            const float f = h.x == -INFINITY ? 0.f : exp2f(h.x - N);
            L = fmaf(f, h.y, L);
            v = fmaf(f, osm[(size_t)q * d * kMgRows + e], v);
        }
        osm[e] = L != 0.f ? v / L : 0.f;
        if (a.lse && e < kMgRows && c0 == 0 && row0 + r < a.rows) a.lse[row0 + r] = L == 0.f ? INFINITY : N + log2f(L);
    }
    __syncthreads();
#pragma unroll 1
    for (int cc = 0; cc < cw; cc += ncol) {  // once up to 512 columns
        f2 acc[kMgRows / 2];
#pragma unroll
        for (int r = 0; r < kMgRows / 2; ++r) acc[r] = pack2(0.f, 0.f);
        const ulonglong2 *o4 = (const ulonglong2 *)(osm + i0 * kMgRows);
        auto add = [&](float v, int k) {
            const f2 vv = pack2(v, v);
#pragma unroll
            for (int r = 0; r < kMgRows / 4; ++r) {
                const ulonglong2 x = o4[k * (kMgRows / 4) + r];
                acc[2 * r] = fma2(vv, x.x, acc[2 * r]);
                acc[2 * r + 1] = fma2(vv, x.y, acc[2 * r + 1]);
            }
        };
        if (works) {
            if (cc == 0) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (k < part) add(first[k], k);
            }
#pragma unroll 8
            for (int k = cc == 0 ? 32 : 0; k < part; ++k) add(w[(int64_t)k * d + cc], k);
#pragma unroll
            for (int r = 0; r < kMgRows / 4; ++r) {
                float4 x;
                unpack2(acc[2 * r], x.x, x.y);
                unpack2(acc[2 * r + 1], x.z, x.w);
                *(float4 *)(red + (share * ncol + cl) * kMgRows + 4 * r) = x;
            }
        }
        __syncthreads();
        for (int e = tid; e < kMgRows * ncol; e += kFinThreads) {
            const int r = e % kMgRows, c = e / kMgRows;
            float v = 0.f;
            for (int k = 0; k < ks; ++k) v += red[k * ncol * kMgRows + e];
            if (row0 + r < a.rows) {
                const int64_t at = (row0 + r) * d + c0 + cc + c;
                if (a.dtype == TQ_F16) ((__half *)a.out)[at] = __float2half_rn(v);
                else if (a.dtype == TQ_BF16) ((__nv_bfloat16 *)a.out)[at] = __float2bfloat16_rn(v);
                else ((float *)a.out)[at] = v;
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t allow_smem(const void *kernel, size_t bytes) {
    // kernels seen on each device, in a table of their own addresses; entries only ever appear
    constexpr int kSlots = 128, kDevices = 16;
    static std::atomic<const void *> seen[kDevices][kSlots];
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool listed = dev >= 0 && dev < kDevices;
    size_t at = ((uintptr_t)kernel >> 4) % kSlots;
    for (int i = 0; listed && i < kSlots; ++i, at = (at + 1) % kSlots) {
        const void *k = seen[dev][at].load(std::memory_order_acquire);
        if (k == kernel) return cudaSuccess;
        if (!k) break;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess || !listed) return e;
    for (int i = 0; i < kSlots; ++i, at = (at + 1) % kSlots) {
        const void *none = nullptr;
        if (seen[dev][at].compare_exchange_strong(none, kernel) || none == kernel) break;
    }
    return cudaSuccess;
}

cudaError_t launch_ragged_plain(const RaggedArgs &a, cudaStream_t s) {
    const size_t smem = sizeof(float) * ((size_t)(a.P.d + a.P.m) * kPlRows + kPlRows * kPlTile);
    dim3 grid((unsigned)a.c.ctas, (unsigned)((a.c.rows + kPlRows - 1) / kPlRows));
    ragged_plain_kernel<<<grid, kPlThreads, smem, s>>>(a);
    return cudaGetLastError();
}

namespace ragged {
template <int D>
cudaError_t launch_dim(const RaggedPair &a, bool f32, int row_block, cudaStream_t s);
extern template cudaError_t launch_dim<64>(const RaggedPair &, bool, int, cudaStream_t);
extern template cudaError_t launch_dim<128>(const RaggedPair &, bool, int, cudaStream_t);
extern template cudaError_t launch_dim<256>(const RaggedPair &, bool, int, cudaStream_t);
}  // namespace ragged

bool ragged_mma_supported(const Prepared &P) {
    return (P.d == 64 || P.d == 128 || P.d == 256) && P.m == P.d / 2 && P.kbeta >= 1 && P.kbeta <= 3 &&
           P.vbeta == P.kbeta + 1;
}

int ragged_mma_ctas_per_sm(const Prepared &P) { return P.d >= 256 ? 3 : 4; }

// A CTA takes eight rows where that saves decoding worth more than the CTAs it costs: more than eight
// rows, or more than four over at least twelve stages for every CTA that fits the GPU.  Blocks of
// eight against four for 8 rows a slice of 16-bit queries at d = 128, in us: 8 slices of 1000 tokens
// 20.6 / 18.5, 16 slices of 8000 41.2 / 36.9, 64 slices of 8000 71.8 / 80.0.  At d = 256 four are
// always faster (30.8 / 24.8, 69 / 61, 161 / 152): eight rows' accumulators leave few registers.
int ragged_mma_rows(const Prepared &P, int64_t rows, int64_t stages) {
    if (P.d >= 256 || rows <= 4) return 4;
    return rows > 8 || stages >= 12 * kSms * ragged_mma_ctas_per_sm(P) ? 8 : 4;
}

cudaError_t launch_ragged_mma(const RaggedArgs &own, const RaggedArgs &prefix, const ServePlan &plan, bool f32,
                              cudaStream_t s) {
    RaggedPair p;
    p.a[0] = own;
    p.a[1] = prefix;
    p.two16 = 1u << 16;
    auto blocks = [&](const RaggedCache &c) { return (c.rows + plan.row_block - 1) / plan.row_block; };
    p.first = plan.own_ctas ? plan.own_ctas * blocks(own.c) : 0;
    p.total = p.first + (plan.prefix_ctas ? plan.prefix_ctas * blocks(prefix.c) : 0);
    switch (own.P.d) {
        case 64: return ragged::launch_dim<64>(p, f32, plan.row_block, s);
        case 128: return ragged::launch_dim<128>(p, f32, plan.row_block, s);
        case 256: return ragged::launch_dim<256>(p, f32, plan.row_block, s);
        default: return cudaErrorInvalidValue;
    }
}

namespace {
// CTAs among which the stages of a cache are divided: enough to fill the GPU once together with
// the row blocks, and no more than there are fours of counted stages, one for each warp of a CTA
// (eights: 16.4 us instead of 14.4 for 4 slices of 200 tokens, 18.5 instead of 17.9 for 2 of 4000).
int division(int64_t slices, int64_t cap, int64_t row_blocks, int per_sm) {
    const int64_t most = slices * ((counted_stages(cap) + 3) / 4);
    int64_t want = ((int64_t)kSms * per_sm + row_blocks - 1) / row_blocks;
    if (want > most) want = most;
    return (int)(want < 1 ? 1 : want);
}
}  // namespace

ServePlan plan_serve(const Prepared &P, tq_dtype dtype, int B, int Hq, int Hkv, int Nq, int64_t t_prefix,
                     int64_t t_cap, bool weigh) {
    ServePlan p;
    memset(&p, 0, sizeof(p));
    const int R = Hq / Hkv * Nq;
    const int64_t rows = (int64_t)B * Hq * Nq, n = P.d + P.m;
    const bool f32 = dtype == TQ_F32;
    p.fast = ragged_mma_supported(P);
    p.row_block = kPlRows;
    const int per_sm = p.fast ? ragged_mma_ctas_per_sm(P) : 4;
    // More than eight 16-bit rows on one prefix: the many-row kernel.  Ragged against many-row, 8 KV
    // heads, 16000 tokens, in us: 12 rows 30.5 / 23.1 (d = 64), 40.5 / 26.8 (128), 60.0 / 47.3 (256), 64
    // rows 57.9 / 25.0, 88.1 / 31.0, 289 / 58.6; 1000 tokens, 12 rows 14.4 / 14.6, 17.9 / 15.7, 25.5 / 20.1.
    // Up to eight the queries keep their 22 bits.  With own caches it is a launch more (6 to 12 us), worth it
    // from 40 million rows x tokens x coordinates on: 33 million 21.5 / 22.4 (64 rows a head on 1000
    // tokens, d = 64), 21.7 / 24.8 (32, 1000, 128), 27.5 / 32.3 (16, 1000, 256), 49 million 26.8 / 24.8 (12
    // of 4 heads, 16000, 64), 27.1 / 25.6 (12, 4000, 128), 65 million 30.5 / 28.1 (64, 1000, 128).
    const bool tc = p.fast && !f32 && t_prefix > 0 && (int64_t)B * R > 8 &&
                    (t_cap == 0 || rows * t_prefix >= 40000000 / P.d);
    // the ragged kernel takes both caches in one launch, in blocks of the larger number of rows
    if (p.fast) {
        const bool pre = t_prefix > 0 && !tc;
        const int64_t stages = (int64_t)B * Hkv * counted_stages(t_cap) + (pre ? Hkv * counted_stages(t_prefix) : 0);
        p.row_block = ragged_mma_rows(P, pre ? (int64_t)B * R : R, stages);
    }
    if (t_cap > 0) p.own_ctas = division((int64_t)B * Hkv, t_cap, (R + p.row_block - 1) / p.row_block, per_sm);
    if (tc) p.tc = prefix_split(P.d, Hkv, (int64_t)B * R, t_prefix);
    else if (t_prefix > 0)
        p.prefix_ctas = division(Hkv, t_prefix, ((int64_t)B * R + p.row_block - 1) / p.row_block, per_sm);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    p.lens = take(sizeof(int32_t) * ((size_t)B + 1));
    p.cum = take(sizeof(int64_t) * ((size_t)B + 3));
    p.qprep = take(p.fast ? 0 : sizeof(float) * (size_t)(rows * n));
    // hi and lo of each operand, 2 bytes each, for whole blocks of rows
    auto frag_bytes = [&](int64_t slices, int64_t r, int block) {
        return (size_t)(slices * ((r + block - 1) / block) * block * n * 4);
    };
    p.own_frag = take(p.fast && t_cap > 0 ? frag_bytes((int64_t)B * Hkv, R, p.row_block) : 0);
    p.pre_frag = take(p.fast && p.prefix_ctas ? frag_bytes(Hkv, (int64_t)B * R, p.row_block) : 0);
    p.qrows = take(tc ? sizeof(uint16_t) * (size_t)(rows * n) : 0);
    p.fscale = take(sizeof(float) * (size_t)rows);
    p.lse = take(weigh ? sizeof(float) * (size_t)rows : 0);
    p.zbuf = take(weigh ? sizeof(float) * (size_t)rows * (size_t)t_cap : 0);
    const size_t ps = sizeof(float) * partial_stride(P.d);
    p.own_part = take(p.own_ctas ? ps * ((size_t)p.own_ctas + (size_t)B * Hkv) * R : 0);
    p.pre_part = take(p.prefix_ctas ? ps * ((size_t)p.prefix_ctas + Hkv) * (size_t)B * R : 0);
    if (tc) p.pre_part = take(ps * (size_t)p.tc.splits * Hkv * (size_t)B * R);
    p.total = o;
    return p;
}

cudaError_t launch_serve(const ServeCall &call, const ServePlan &plan, void *scratch, cudaStream_t s) {
    char *base = (char *)scratch;
    const Prepared &P = call.P;
    const int R = call.Hq / call.Hkv * call.Nq;
    PrepArgs pa;
    memset(&pa, 0, sizeof(pa));
    pa.P = P;
    pa.q = call.q;
    pa.dtype = call.dtype;
    pa.rows = call.rows;
    pa.rows_in = R;
    pa.Hkv = call.Hkv;
    pa.scale = call.scale;
    pa.fscale = (float *)(base + plan.fscale);
    if (!plan.fast) pa.qprep = (float *)(base + plan.qprep);
    if (plan.fast && plan.own_ctas) pa.own_frag = (uint16_t *)(base + plan.own_frag);
    if (plan.fast && plan.prefix_ctas) pa.pre_frag = (uint16_t *)(base + plan.pre_frag);
    if (plan.tc.splits) pa.qrows = (uint16_t *)(base + plan.qrows);
    pa.row_block = plan.row_block;
    pa.prefix_blocks = (int)(((int64_t)call.B * R + plan.row_block - 1) / plan.row_block);
    pa.lens = call.lens;
    pa.B = call.B;
    pa.t_cap = call.t_cap;
    pa.t_prefix = call.t_prefix;
    pa.len_own = (int32_t *)(base + plan.lens);
    pa.cum_own = (int64_t *)(base + plan.cum);
    pa.dev_status = call.dev_status;
    // Rows that fill the GPU several times over: twice as many a CTA, for half the reads of R.  Whole calls
    // on a prefix of 64 tokens with 8 against 16 rows a CTA, in us: 2048 rows 31.1 / 28.2 (d = 128), 65.4 /
    // 60.1 (256), 4096 rows 32.5 / 30.5 (64), 16384 rows 93.9 / 79.8, 148 / 129, 378 / 321.
    const int64_t cols = (P.d + P.m + kPrepCols - 1) / kPrepCols;
    const bool many = call.rows * cols >= 8 * 4 * kSms && P.d <= 256;
    const int prep_rows = many ? 16 : 8;
    const unsigned prep_ctas = (unsigned)((call.rows + prep_rows - 1) / prep_rows * cols + 1);
    const size_t prep_smem = sizeof(float) * prep_rows * P.d;
    if (many) serve_prep_kernel<16><<<prep_ctas, kPrepThreads, prep_smem, s>>>(pa);
    else serve_prep_kernel<8><<<prep_ctas, kPrepThreads, prep_smem, s>>>(pa);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    RaggedArgs own, pre;
    memset(&own, 0, sizeof(own));
    own.P = P;
    own.qprep = pa.qprep;
    own.fscale = pa.fscale;
    pre = own;
    own.frag = (const uint2 *)pa.own_frag;
    pre.frag = (const uint2 *)pa.pre_frag;
    if (plan.own_ctas) {
        own.c = call.own;
        own.c.len = pa.len_own;
        own.c.cum = pa.cum_own;
        own.c.slices = call.B * call.Hkv;
        own.c.per_seq = call.Hkv;
        own.c.nseq = call.B;
        own.c.rows = own.c.rows_in = R;
        own.c.ctas = plan.own_ctas;
        own.part = (float *)(base + plan.own_part);
        own.zbuf = call.weights ? (float *)(base + plan.zbuf) : nullptr;
        if (!plan.fast) e = launch_ragged_plain(own, s);
        if (e != cudaSuccess) return e;
    }
    if (call.t_prefix > 0) {
        pre.c = call.prefix;
        pre.c.len = pa.len_own + call.B;
        pre.c.cum = pa.cum_own + call.B + 1;
        pre.c.slices = pre.c.per_seq = call.Hkv;
        pre.c.nseq = 1;
        pre.c.rows_in = R;
        pre.c.rows = call.B * R;
        pre.c.rows_outer = (int64_t)call.Hkv * R;
        pre.c.ctas = plan.prefix_ctas;
        pre.part = (float *)(base + plan.pre_part);
        if (!plan.fast) e = launch_ragged_plain(pre, s);
        if (e != cudaSuccess) return e;
    }
    if (plan.fast && (plan.own_ctas || plan.prefix_ctas)) {
        e = launch_ragged_mma(own, pre, plan, call.dtype == TQ_F32, s);
        if (e != cudaSuccess) return e;
    }
    if (plan.tc.splits) {
        // behind the own caches: its decoders need nothing of the call and have begun when those end (32
        // requests, prefix 8192: 47.1 us, 48.6 the other way round)
        e = launch_prefix_tc(P, pre.c, pa.qrows, pa.fscale, pre.part, plan.tc, call.dev_status, s);
        if (e != cudaSuccess) return e;
    }
    FinishArgs fa;
    memset(&fa, 0, sizeof(fa));
    fa.P = P;
    fa.own = own.c;
    fa.prefix = pre.c;
    fa.own_part = own.part;
    fa.pre_part = pre.part;
    fa.tc_splits = plan.tc.splits;
    fa.rows = call.rows;
    fa.rows_in = R;
    fa.Hkv = call.Hkv;
    fa.dtype = call.dtype;
    fa.out = call.out;
    // A CTA fills an SM: blocks of few rows, as long as they make one wave (1024 rows: whole calls of 93.2
    // us with blocks of 4, 89.9 with 8; 2048 rows: 254 with 4, 244 with 16).  Fewer rows than that: the
    // columns of a block go to several CTAs, which merge the same partials each.
    const int mg_rows = call.rows <= 4 * kSms ? 4 : call.rows <= 8 * kSms ? 8 : 16;
    const int64_t blocks = (call.rows + mg_rows - 1) / mg_rows;
    fa.csplit = 1;
    while (fa.csplit < P.d / 64 && blocks * fa.csplit * 2 <= kSms) fa.csplit *= 2;
    const int64_t merge = blocks * fa.csplit;
    int64_t weigh = 0;
    if (call.weights) {
        fa.zbuf = own.zbuf;
        fa.weights = call.weights;
        fa.chunks = (int)((call.t_cap + kWtTokens - 1) / kWtTokens);
        weigh = (int64_t)fa.chunks * call.B * call.Hkv;
    }
    fa.merge_ctas = (unsigned)merge;
    const auto finish = mg_rows == 4   ? serve_finish_kernel<4>
                        : mg_rows == 8 ? serve_finish_kernel<8>
                                       : serve_finish_kernel<16>;
    const size_t fin_smem = sizeof(float) * (kFinThreads / 32) * P.d;
    if (fin_smem >= 8 * 1024) {  // with the static arrays it can be above what is allowed without asking
        e = allow_smem((const void *)finish, sizeof(float) * (kFinThreads / 32) * kMaxDim);
        if (e != cudaSuccess) return e;
    }
    // Few weighing CTAs ride along with the merging ones; many get a launch of their own, where more of
    // them fit an SM (8 against 1: 11 against 50 us for 2048 of them).
    const bool along = weigh <= kSms;
    if (!along) fa.lse = (float *)(base + plan.lse);
    e = launch_after(finish, (unsigned)(merge + (along ? weigh : 0)), kFinThreads, fin_smem, s, fa);
    if (e != cudaSuccess || along) return e;
    return launch_after(serve_weigh_kernel, (unsigned)weigh, kWtThreads, 0, s, fa);
}

}  // namespace tq
