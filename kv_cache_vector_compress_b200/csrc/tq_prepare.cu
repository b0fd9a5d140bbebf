// tq_prepare.cu -- derive the kernels' operand copies of R and S into the workspace.
#include <math.h>
#include <string.h>

#include "tq_common.cuh"
#include "tq_internal.cuh"

namespace tq {

namespace {

__global__ void prepare_kernel(const float *__restrict__ R, const float *__restrict__ S, int d, int m,
                               Codebooks cb, WsHeader hdr, char *__restrict__ ws, WsLayout L) {
    float *Rc = (float *)(ws + L.R);
    float *RT = (float *)(ws + L.RT);
    float *ST = (float *)(ws + L.ST);
    float *SpT = (float *)(ws + L.SpT);
    const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t nth = (int64_t)gridDim.x * blockDim.x;
    if (tid == 0) {
        *(WsHeader *)(ws + L.header) = hdr;
        *(Codebooks *)(ws + L.codebooks) = cb;
    }
    uint16_t *Rhi = (uint16_t *)(ws + L.Rsw);
    uint16_t *Rlo = Rhi + (size_t)d * d;
    for (int64_t e = tid; e < (int64_t)d * d; e += nth) {
        int i = (int)(e / d), j = (int)(e % d);
        float v = R[e];
        Rc[e] = v;
        RT[(int64_t)j * d + i] = v;
        // split operand: R * 2^s = hi + lo, both fp16, row i = output coordinate, k = j
        const float sv = v * (float)(1 << kRScaleLog2);
        const __half hi = __float2half_rn(sv);
        const __half lo = __float2half_rn(sv - __half2float(hi));
        const size_t off = sw128_offset(d, i, j) / 2;
        Rhi[off] = __half_as_ushort(hi);
        Rlo[off] = __half_as_ushort(lo);
    }
    // keys' rotation operand [R; S] * 2^s split into fp16 hi + lo, d + m rows
    {
        const int rows = d + (m > 0 ? m : 0);
        uint16_t *Xhi = (uint16_t *)(ws + L.RSsw);
        uint16_t *Xlo = Xhi + (size_t)d * rows;
        for (int64_t e = tid; e < (int64_t)rows * d; e += nth) {
            const int i = (int)(e / d), j = (int)(e % d);
            const float v = (i < d) ? R[(int64_t)i * d + j] : S[(int64_t)(i - d) * d + j];
            const float sv = v * (float)(1 << kRScaleLog2);
            const __half hi = __float2half_rn(sv);
            const __half lo = __float2half_rn(sv - __half2float(hi));
            const size_t off = sw128_offset(rows, i, j) / 2;
            Xhi[off] = __half_as_ushort(hi);
            Xlo[off] = __half_as_ushort(lo);
        }
    }
    if (m <= 0) return;
    float *Srow = (float *)(ws + L.S);
    float *Sprow = (float *)(ws + L.Sp);
    for (int64_t e = tid; e < (int64_t)m * d; e += nth) {
        int a = (int)(e / d), j = (int)(e % d);
        ST[(int64_t)j * m + a] = S[e];
        Srow[e] = S[e];
    }
    // S' = S R^T expressed on rotated coordinates: S'[a][i] = sum_k S[a][k] R[i][k],
    // accumulated in double and rounded once.
    for (int64_t e = tid; e < (int64_t)m * d; e += nth) {
        int a = (int)(e / d), i = (int)(e % d);
        const float *sr = S + (int64_t)a * d;
        const float *rr = R + (int64_t)i * d;
        double acc = 0.0;
        for (int k = 0; k < d; ++k) acc += (double)sr[k] * (double)rr[k];
        SpT[(int64_t)i * m + a] = (float)acc;
        Sprow[e] = (float)acc;
        // split operand of S' * 2^s: row a = projection index, k = i (rotated coordinate)
        const double sv = acc * (double)(1 << kSScaleLog2);
        const __half hi = __double2half(sv);
        const __half lo = __float2half_rn((float)(sv - (double)__half2float(hi)));
        uint16_t *Shi = (uint16_t *)(ws + L.Ssw);
        uint16_t *Slo = Shi + (size_t)m * d;
        const size_t off = sw128_offset(m, a, i) / 2;
        Shi[off] = __half_as_ushort(hi);
        Slo[off] = __half_as_ushort(lo);
    }
}

// The workspace's serve tables; qbound from the rows of R and S (one CTA, a warp a row).
__global__ void __launch_bounds__(1024) prepare_serve_kernel(const float *__restrict__ R, const float *__restrict__ S,
                                                             int d, int m, ServeTables t,
                                                             ServeTables *__restrict__ out) {
    __shared__ float wmax[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float gamma = m > 0 ? sqrtf(1.5707963267948966f) / (float)m : 0.f;
    float best = 0.f;
    for (int r = warp; r < d + m; r += 32) {
        const float *row = r < d ? R + (int64_t)r * d : S + (int64_t)(r - d) * d;
        float s = 0.f;
        for (int j = lane; j < d; j += 32) s = fmaf(row[j], row[j], s);
        s = sqrtf(warp_sum(s)) * (r < d ? t.sigma : gamma);
        best = fmaxf(best, s);
    }
    if (lane == 0) wmax[warp] = best;
    __syncthreads();
    if (warp == 0) {
        best = warp_max(wmax[lane]);
        if (lane == 0) {
            t.qbound = best;
            *out = t;
        }
    }
}

void split_f16(double v, uint16_t *hi, uint16_t *lo) {
    const __half h = __float2half_rn((float)v);
    *hi = __half_as_ushort(h);
    *lo = __half_as_ushort(__float2half_rn((float)(v - (double)__half2float(h))));
}

// v less the nearest fp16 number, for v in fp16's normal range: the float's mantissa rounded to ten bits,
// ties to even (tq_prepare at 4 bits: 222 us of the host, 270 with the conversions' own functions).
double off_f16(double v) {
    float f = (float)v;
    uint32_t u;
    memcpy(&u, &f, sizeof(u));
    u = (u + 0xFFFu + ((u >> 13) & 1u)) & ~0x1FFFu;
    memcpy(&f, &u, sizeof(f));
    return v - (double)f;
}

// A codebook's operand is its centroids over a scale that may be anything, so it is chosen for the
// centroids to land near fp16 numbers: of 1024 scales that put the largest one on an fp16 number
// (in [8, 16), so that low halves are normal numbers too), the one with the least squared error by
// cell mass.  1 bit: exact.  2 bits: one ratio to approximate, so that one fp16 operand serves 32-bit
// scores: 2^-21.3 off at most for the Gaussian law; the Beta law has a ratio for each dimension, 2^-19.6
// off at most for d = 64, 128 and 256, which the tensor-core kernels take.  3 bits: 2^-15 and 2^-14.3.
double table_scale(const float *c, const float *b, int K, int dim) {
    const int h = K / 2;
    double width[kMaxLevels / 2], density[kMaxLevels / 2];  // of the cells; their products are the masses
    for (int k = h; k < K; ++k) {
        const double lo = k > h ? b[k - 1] : 0.0, up = k < K - 1 ? b[k] : 2.0 * c[k] - lo;
        width[k - h] = up - lo;
        density[k - h] = exp(-0.5 * dim * (double)c[k] * c[k]);
    }
    double best = INFINITY, scale = 1.0;
    for (int i = 0; i < 1024; ++i) {
        const double s = (double)c[K - 1] / (8.0 * (1.0 + i * (1.0 / 1024.0)));
        double e = 0.0;
        for (int k = h; k < K; ++k) {
            const double x = off_f16(c[k] / s) * s;
            e += x * x * width[k - h] * density[k - h];
        }
        if (e < best) {
            best = e;
            scale = s;
        }
    }
    return scale;
}

ServeTables serve_tables(const Codebooks &cb, int bits, int dim) {
    ServeTables t = {};
    const int V = 1 << bits, K = V / 2;
    const double tau = table_scale(cb.vc, cb.vb, V, dim), sigma = bits > 1 ? table_scale(cb.kc, cb.kb, K, dim) : 1.0;
    t.tau = (float)tau;
    t.sigma = (float)sigma;
    for (int k = 0; k < V; ++k) split_f16(cb.vc[k] / (double)t.tau, &t.vh[k], &t.vl[k]);
    for (int k = 0; bits > 1 && k < K; ++k) split_f16(cb.kc[k] / (double)t.sigma, &t.kh[k], &t.kl[k]);
    return t;
}

}  // namespace

cudaError_t launch_prepare(const tq_params *p, const Codebooks &cb, cudaStream_t s) {
    WsLayout L = ws_layout(p->dim, p->proj_dim);
    WsHeader h{kWsMagic, p->dim, p->bits, p->proj_dim};
    int64_t work = (int64_t)p->dim * (p->dim > p->proj_dim ? p->dim : p->proj_dim);
    int blocks = (int)((work + 255) / 256);
    if (blocks > 148 * 8) blocks = 148 * 8;
    if (blocks < 1) blocks = 1;
    prepare_kernel<<<blocks, 256, 0, s>>>(p->R, p->S, p->dim, p->proj_dim, cb, h,
                                         (char *)p->workspace, L);
    const cudaError_t e = cudaGetLastError();
    // (the search of the tables takes the host 10 to 50 us; not for sets that the serving calls refuse)
    if (e != cudaSuccess || p->bits < 2 || p->proj_dim < 32) return e;
    prepare_serve_kernel<<<1, 1024, 0, s>>>(p->R, p->S, p->dim, p->proj_dim, serve_tables(cb, p->bits, p->dim),
                                            (ServeTables *)((char *)p->workspace + L.serve));
    return cudaGetLastError();
}

}  // namespace tq
