// tq_serve.cu -- what surrounds the attention kernels of tq_attend_shared and tq_attend_weigh: the
// preparation of the query rows and operand tables, the merge of the partial results and the
// addition of the softmax weights; and the plain kernel for the shapes without a tensor-core one.
#include <math.h>

#include <cuda_bf16.h>

#include "tq_serve.cuh"

namespace tq {

namespace {

// ------------------------------------------------------------------ preparation

constexpr int kPrepThreads = 256;
constexpr int kPrepRows = 4;   // query rows a CTA takes
constexpr int kPrepCols = 8;   // outputs a thread takes at most: (1024 + 1024) / 256

struct PrepArgs {
    Prepared P;
    const void *q;
    tq_dtype dtype;
    int64_t rows;
    float scale;
    int fast;
    ServeTables *tables;
    float *qprep, *fscale;
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

// The scale sigma of the keys' codebook.  1 bit: sigma = c, so that the operand is 1.  2 bits:
// sigma = c_1 / (1 + i / 1024) with the i for which c_2 / sigma is nearest to an fp16 number (a
// rational approximation of their ratio: about 2^-21 off for the Gaussian law), so that one fp16
// operand is enough for 32-bit scores.  3 bits: sigma = c_1; the operand is split in two.
// Called by a whole warp; the same value in every lane.
__device__ float key_sigma(const Prepared &P, int lane) {
    const float c1 = P.cb->kc[(1 << P.kbeta) / 2];
    if (P.kbeta != 2) return c1;
    const double a = c1, b = P.cb->kc[3];
    float best = INFINITY;
    int at = 0;
    for (int i = lane; i < 1024; i += 32) {
        const double h = 1.0 + i * (1.0 / 1024.0), v = b / a * h;
        const double e = fabs((double)__half2float(__double2half(v)) / v - 1.0);
        if ((float)e < best) {
            best = (float)e;
            at = i;
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        const float ob = __shfl_xor_sync(kFull, best, o);
        const int oa = __shfl_xor_sync(kFull, at, o);
        if (ob < best || (ob == best && oa < at)) {
            best = ob;
            at = oa;
        }
    }
    return (float)(a / (1.0 + at * (1.0 / 1024.0)));
}

__device__ void split_f16(float v, uint16_t *hi, uint16_t *lo) {
    const __half h = __float2half_rn(v);
    *hi = __half_as_ushort(h);
    *lo = __half_as_ushort(__float2half_rn(v - __half2float(h)));
}

// q_rot = R q and sq = S q of kPrepRows rows per CTA, scaled (see the header), in fp32 by fmaf in
// ascending j.  The last CTA writes the tables and the contexts' lengths instead.  Reads R and S
// once per CTA from L2 (98 KB at d = 128).
__global__ void __launch_bounds__(kPrepThreads) serve_prep_kernel(PrepArgs a) {
    extern __shared__ __align__(16) float qT[];  // [d][kPrepRows]
    __shared__ float sig;
    __shared__ uint32_t rmax[kPrepRows];
    __shared__ int64_t wsum[kPrepThreads / 32];
    const Prepared &P = a.P;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int d = P.d, m = P.m, n = d + m;
    if (blockIdx.x == gridDim.x - 1) {
        const float sigma = a.fast ? key_sigma(P, lane) : 1.f;
        if (tid < 8) {
            const int K = 1 << P.kbeta;
            split_f16(tid < K ? P.cb->kc[tid] / sigma : 0.f, &a.tables->kh[tid], &a.tables->kl[tid]);
        }
        const int V = 1 << P.vbeta;
        // the largest value centroid lands in [8, 16): its low half stays a normal fp16 number
        const float tau = exp2f((float)(ilogbf(P.cb->vc[V - 1]) - 3));
        if (tid < 16) split_f16(tid < V ? P.cb->vc[tid] / tau : 0.f, &a.tables->vh[tid], &a.tables->vl[tid]);
        if (tid == 0) a.tables->tau = tau;
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
            const int64_t st = (len + kStage - 1) / kStage;
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
            a.cum_own[a.B + 2] = (a.t_prefix + kStage - 1) / kStage;
        }
        return;
    }
    const int64_t r0 = (int64_t)blockIdx.x * kPrepRows;
    const int nr = (int)min((int64_t)kPrepRows, a.rows - r0);
    for (int e = tid; e < kPrepRows * d; e += kPrepThreads) {
        const int r = e / d, j = e - r * d;
        qT[j * kPrepRows + r] = r < nr ? load_elem(a.q, a.dtype, (r0 + r) * d + j) : 0.f;
    }
    if (tid < kPrepRows) rmax[tid] = 0u;
    if (warp == 0) {
        const float s = a.fast ? key_sigma(P, lane) : 1.f;
        if (lane == 0) sig = s;
    }
    __syncthreads();
    const float gamma = sqrtf(1.5707963267948966f) / (float)m;
    float acc[kPrepCols][kPrepRows];
#pragma unroll
    for (int o = 0; o < kPrepCols; ++o) {
#pragma unroll
        for (int r = 0; r < kPrepRows; ++r) acc[o][r] = 0.f;
        const int c = tid + o * kPrepThreads;
        if (c < n) {
            const float *w = c < d ? P.RT + c : P.ST + (c - d);
            const int ld = c < d ? d : m;
#pragma unroll 16
            for (int j = 0; j < d; ++j) {
                const float v = w[(int64_t)j * ld];
                const float4 q4 = *(const float4 *)(qT + j * kPrepRows);
                acc[o][0] = fmaf(v, q4.x, acc[o][0]);
                acc[o][1] = fmaf(v, q4.y, acc[o][1]);
                acc[o][2] = fmaf(v, q4.z, acc[o][2]);
                acc[o][3] = fmaf(v, q4.w, acc[o][3]);
            }
            const float f = c < d ? sig : gamma;
#pragma unroll
            for (int r = 0; r < kPrepRows; ++r) acc[o][r] *= f;
        }
    }
    // the row's exponent: the largest operand in [2^11, 2^12), far from both ends of fp16's range
    // (its low half, 2^-11 of it, stays a normal number); rows of zeros, infinities and NaN keep 0
    if (a.fast) {
#pragma unroll
        for (int r = 0; r < kPrepRows; ++r) {
            float mx = 0.f;
#pragma unroll
            for (int o = 0; o < kPrepCols; ++o) mx = fmaxf(mx, fabsf(acc[o][r]));
            mx = warp_max(mx);
            if (lane == 0) atomicMax(&rmax[r], __float_as_uint(mx));  // nonnegative: ordered as integers
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kPrepRows; ++r) {
        if (r >= nr) break;
        const float mx = __uint_as_float(rmax[r]);
        const int e = (mx > 0.f && mx < INFINITY) ? min(max(ilogbf(mx) - 11, -126), 126) : 0;
        const float down = exp2f((float)-e);
#pragma unroll
        for (int o = 0; o < kPrepCols; ++o) {
            const int c = tid + o * kPrepThreads;
            if (c < n) a.qprep[(r0 + r) * n + c] = acc[o][r] * down;
        }
        if (tid == 0) a.fscale[r0 + r] = a.scale * kLog2eF * exp2f((float)e);
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
    extern __shared__ __align__(16) float sm[];  // qs[(d + m)][kPlRows], ps[kPlRows][kPlTile]
    __shared__ float kcen[kMaxLevels], vcen[kMaxLevels];
    __shared__ float red[kPlRows][kPlThreads / 32], rowN[kPlRows], rowA[kPlRows];
    const Prepared &P = a.P;
    const int d = P.d, m = P.m, n = d + m, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *qs = sm, *ps = sm + n * kPlRows;
    if (tid < kMaxLevels) {
        kcen[tid] = P.cb->kc[tid];
        vcen[tid] = P.cb->vc[tid];
    }
    const int64_t total = ragged_total(a.c);
    const int64_t w1 = cta_first(total, a.c.ctas, blockIdx.x + 1);
    const int r0 = blockIdx.y * kPlRows, nr = min(kPlRows, a.c.rows - r0);
    const int kw = P.kbeta * (d >> 5), sw = m >> 5, vw = P.vbeta * (d >> 5);
    Piece pc;
    for (int64_t w = cta_first(total, a.c.ctas, blockIdx.x); w < w1; w += pc.s1 - pc.s0) {
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
        if (tid < kPlRows) rowN[tid] = -INFINITY;
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
                const float vn = fmaxf(f16_bits_to_f32(a.c.vnorm[rec]), kMinNorm), lv = log2f(vn);
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
                rowA[tid] = old == -INFINITY ? 0.f : exp2f(old - mx);
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kPlRows; ++r) {
                const float N = rowN[r], w8 = N == -INFINITY ? 0.f : exp2f(y[r] - N);
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

// ------------------------------------------------------------------ merge

constexpr int kMgThreads = 128;
constexpr int kMgRows = 4;

struct MergeArgs {
    Prepared P;
    RaggedCache own, prefix;
    const float *own_part, *pre_part;
    int64_t rows;
    int rows_in, Hkv;
    tq_dtype dtype;
    void *out;
    float *lse;  // log2 of the row's sum of 2^z, or null
};

// The partials of one row, one range of CTAs per cache: base + i * step.
struct PartRange {
    const float *base;
    int64_t step;
    int n;
};

__device__ __forceinline__ PartRange parts_of(const RaggedCache &c, const float *part, int slice, int r, int ps) {
    PartRange g = {nullptr, 0, 0};
    int c0, c1;
    if (c.slices > 0 && slice_ctas(c, slice, &c0, &c1)) {
        g.base = part + ((int64_t)(c0 + slice) * c.rows + r) * ps;
        g.step = (int64_t)c.rows * ps;
        g.n = c1 - c0 + 1;
    }
    return g;
}

// out = R^T o / l of kMgRows rows per CTA: the partials of each row are rescaled to their largest
// reference and added in the order of the context (a warp a row), then the rows are rotated back
// together, so that R is read once per CTA.  A row without a token is zero.
__global__ void __launch_bounds__(kMgThreads) serve_merge_kernel(MergeArgs a) {
    extern __shared__ __align__(16) float osm[];  // [d][kMgRows]
    const int d = a.P.d, ps = partial_stride(d), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * kMgRows;
    {
        const int64_t row = row0 + warp;
        const bool there = row < a.rows;
        float inv = 0.f, N = -INFINITY;
        PartRange g[2] = {{nullptr, 0, 0}, {nullptr, 0, 0}};
        if (there) {
            const int slice = (int)(row / a.rows_in), r = (int)(row % a.rows_in);
            const int b = slice / a.Hkv, kv = slice - b * a.Hkv;
            g[0] = parts_of(a.prefix, a.pre_part, kv, b * a.rows_in + r, ps);
            g[1] = parts_of(a.own, a.own_part, slice, r, ps);
            for (int k = 0; k < 2; ++k)
                for (int i = lane; i < g[k].n; i += 32) N = fmaxf(N, g[k].base[i * g[k].step]);
            N = warp_max(N);
            float L = 0.f;
            for (int k = 0; k < 2; ++k)
                for (int i = lane; i < g[k].n; i += 32) {
                    const float *p = g[k].base + i * g[k].step;
                    L += N == -INFINITY ? 0.f : p[1] * exp2f(p[0] - N);
                }
            L = warp_sum(L);
            inv = L != 0.f ? 1.f / L : 0.f;
            if (lane == 0 && a.lse) a.lse[row] = L == 0.f ? INFINITY : N + log2f(L);
        }
        for (int j0 = 0; j0 < d; j0 += 32) {
            const int j = j0 + lane;
            float acc = 0.f;
            for (int k = 0; k < 2; ++k)
#pragma unroll 4
                for (int i = 0; i < g[k].n; ++i) {
                    const float *p = g[k].base + i * g[k].step;
                    const float w = N == -INFINITY ? 0.f : exp2f(p[0] - N);
                    acc = fmaf(w, p[4 + j], acc);
                }
            osm[j * kMgRows + warp] = acc * inv;
        }
    }
    __syncthreads();
    for (int j = tid; j < d; j += kMgThreads) {
        float acc[kMgRows] = {};
#pragma unroll 16
        for (int i = 0; i < d; ++i) {
            const float v = a.P.R[(int64_t)i * d + j];
            const float4 o4 = *(const float4 *)(osm + i * kMgRows);
            acc[0] = fmaf(v, o4.x, acc[0]);
            acc[1] = fmaf(v, o4.y, acc[1]);
            acc[2] = fmaf(v, o4.z, acc[2]);
            acc[3] = fmaf(v, o4.w, acc[3]);
        }
#pragma unroll
        for (int r = 0; r < kMgRows; ++r) {
            if (row0 + r >= a.rows) break;
            const int64_t at = (row0 + r) * d + j;
            if (a.dtype == TQ_F16) ((__half *)a.out)[at] = __float2half_rn(acc[r]);
            else if (a.dtype == TQ_BF16) ((__nv_bfloat16 *)a.out)[at] = __float2bfloat16_rn(acc[r]);
            else ((float *)a.out)[at] = acc[r];
        }
    }
}

// ------------------------------------------------------------------ softmax weights

constexpr int kWtThreads = 256;

// weights[slice][t] += sum over the slice's rows of 2^(z - lse): one thread a token, the rows in
// ascending order.  Bound by the 4 rows + 8 bytes a token that it moves.
__global__ void __launch_bounds__(kWtThreads) serve_weigh_kernel(RaggedCache c, const float *__restrict__ zbuf,
                                                                 const float *__restrict__ lse,
                                                                 float *__restrict__ weights) {
    const int slice = blockIdx.y;
    const int t = blockIdx.x * kWtThreads + threadIdx.x;
    if (t >= c.len[slice / c.per_seq]) return;
    const float *z = zbuf + (int64_t)slice * c.rows * c.stride + t;
    const float *L = lse + (int64_t)slice * c.rows;
    float s = 0.f;
    for (int r = 0; r < c.rows; ++r) s += exp2f(z[r * c.stride] - L[r]);
    weights[slice * c.stride + t] += s;
}

}  // namespace

cudaError_t launch_ragged_plain(const RaggedArgs &a, cudaStream_t s) {
    const size_t smem = sizeof(float) * ((size_t)(a.P.d + a.P.m) * kPlRows + kPlRows * kPlTile);
    dim3 grid((unsigned)a.c.ctas, (unsigned)((a.c.rows + kPlRows - 1) / kPlRows));
    ragged_plain_kernel<<<grid, kPlThreads, smem, s>>>(a);
    return cudaGetLastError();
}

namespace ragged {
template <int D>
cudaError_t launch_dim(const RaggedArgs &a, bool f32, int row_block, cudaStream_t s);
extern template cudaError_t launch_dim<64>(const RaggedArgs &, bool, int, cudaStream_t);
extern template cudaError_t launch_dim<128>(const RaggedArgs &, bool, int, cudaStream_t);
extern template cudaError_t launch_dim<256>(const RaggedArgs &, bool, int, cudaStream_t);
}  // namespace ragged

bool ragged_mma_supported(const Prepared &P) {
    return (P.d == 64 || P.d == 128 || P.d == 256) && P.m == P.d / 2 && P.kbeta >= 1 && P.kbeta <= 3 &&
           P.vbeta == P.kbeta + 1;
}

// Eight rows a CTA when there are more than four, but for 32-bit results of 256 coordinates, whose
// accumulators would not fit the registers.
int ragged_mma_rows(const Prepared &P, bool f32, int64_t rows) {
    return rows <= 4 || (f32 && P.d >= 256) ? 4 : 8;
}

int ragged_mma_ctas_per_sm(const Prepared &P) { return P.d >= 256 ? 3 : 4; }

cudaError_t launch_ragged_mma(const RaggedArgs &a, bool f32, int row_block, cudaStream_t s) {
    switch (a.P.d) {
        case 64: return ragged::launch_dim<64>(a, f32, row_block, s);
        case 128: return ragged::launch_dim<128>(a, f32, row_block, s);
        case 256: return ragged::launch_dim<256>(a, f32, row_block, s);
        default: return cudaErrorInvalidValue;
    }
}

namespace {
// CTAs among which the stages of a cache are divided: enough to fill the GPU once together with
// the row blocks, and no more than there are stages.
int division(int64_t slices, int64_t cap, int64_t row_blocks, int per_sm) {
    const int64_t most = slices * ((cap + kStage - 1) / kStage);
    int64_t want = (148ll * per_sm + row_blocks - 1) / row_blocks;
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
    p.prefix_block = kPlRows;
    const int per_sm = p.fast ? ragged_mma_ctas_per_sm(P) : 4;
    if (p.fast) {
        p.row_block = ragged_mma_rows(P, f32, R);
        p.prefix_block = ragged_mma_rows(P, f32, (int64_t)B * R);
    }
    if (t_cap > 0) p.own_ctas = division((int64_t)B * Hkv, t_cap, (R + p.row_block - 1) / p.row_block, per_sm);
    if (t_prefix > 0)
        p.prefix_ctas = division(Hkv, t_prefix, ((int64_t)B * R + p.prefix_block - 1) / p.prefix_block, per_sm);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    p.tables = take(sizeof(ServeTables));
    p.lens = take(sizeof(int32_t) * ((size_t)B + 1));
    p.cum = take(sizeof(int64_t) * ((size_t)B + 3));
    p.qprep = take(sizeof(float) * (size_t)(rows * n));
    p.fscale = take(sizeof(float) * (size_t)rows);
    p.lse = take(weigh ? sizeof(float) * (size_t)rows : 0);
    p.zbuf = take(weigh ? sizeof(float) * (size_t)rows * (size_t)t_cap : 0);
    const size_t ps = sizeof(float) * partial_stride(P.d);
    p.own_part = take(p.own_ctas ? ps * ((size_t)p.own_ctas + (size_t)B * Hkv) * R : 0);
    p.pre_part = take(p.prefix_ctas ? ps * ((size_t)p.prefix_ctas + Hkv) * (size_t)B * R : 0);
    p.total = o;
    return p;
}

cudaError_t launch_serve(const ServeCall &call, const ServePlan &plan, void *scratch, cudaStream_t s) {
    char *base = (char *)scratch;
    const Prepared &P = call.P;
    PrepArgs pa;
    pa.P = P;
    pa.q = call.q;
    pa.dtype = call.dtype;
    pa.rows = call.rows;
    pa.scale = call.scale;
    pa.fast = plan.fast;
    pa.tables = (ServeTables *)(base + plan.tables);
    pa.qprep = (float *)(base + plan.qprep);
    pa.fscale = (float *)(base + plan.fscale);
    pa.lens = call.lens;
    pa.B = call.B;
    pa.t_cap = call.t_cap;
    pa.t_prefix = call.t_prefix;
    pa.len_own = (int32_t *)(base + plan.lens);
    pa.cum_own = (int64_t *)(base + plan.cum);
    pa.dev_status = call.dev_status;
    serve_prep_kernel<<<(unsigned)((call.rows + kPrepRows - 1) / kPrepRows + 1), kPrepThreads,
                        sizeof(float) * kPrepRows * P.d, s>>>(pa);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    const int R = call.Hq / call.Hkv * call.Nq;
    RaggedArgs own, pre;
    memset(&own, 0, sizeof(own));
    own.P = P;
    own.tables = pa.tables;
    own.qprep = pa.qprep;
    own.fscale = pa.fscale;
    pre = own;
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
        e = plan.fast ? launch_ragged_mma(own, call.dtype == TQ_F32, plan.row_block, s) : launch_ragged_plain(own, s);
        if (e != cudaSuccess) return e;
    }
    if (plan.prefix_ctas) {
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
        e = plan.fast ? launch_ragged_mma(pre, call.dtype == TQ_F32, plan.prefix_block, s)
                      : launch_ragged_plain(pre, s);
        if (e != cudaSuccess) return e;
    }
    MergeArgs ma;
    ma.P = P;
    ma.own = own.c;
    ma.prefix = pre.c;
    ma.own_part = own.part;
    ma.pre_part = pre.part;
    ma.rows = call.rows;
    ma.rows_in = R;
    ma.Hkv = call.Hkv;
    ma.dtype = call.dtype;
    ma.out = call.out;
    ma.lse = call.weights ? (float *)(base + plan.lse) : nullptr;
    serve_merge_kernel<<<(unsigned)((call.rows + kMgRows - 1) / kMgRows), kMgThreads,
                         sizeof(float) * kMgRows * P.d, s>>>(ma);
    e = cudaGetLastError();
    if (e != cudaSuccess || !call.weights) return e;
    dim3 grid((unsigned)((call.t_cap + kWtThreads - 1) / kWtThreads), (unsigned)(call.B * call.Hkv));
    serve_weigh_kernel<<<grid, kWtThreads, 0, s>>>(own.c, own.zbuf, ma.lse, call.weights);
    return cudaGetLastError();
}

}  // namespace tq
