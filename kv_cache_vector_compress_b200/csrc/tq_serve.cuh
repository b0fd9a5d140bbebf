// tq_serve.cuh -- what the kernels of tq_attend_shared and tq_attend_weigh share: the problem, the
// division of ragged contexts among CTAs, the scratch layout and the launchers.
//
// Estimated logits of query row r against token t, in log2 units:
//   z = f_r ||k_t|| ( sum_j Q_rj C[kidx_tj] + rho_t sum_i P_ri sgn_ti )
// Q = sigma 2^-e_r R q, P = 2^-e_r sqrt(pi/2)/m S q, C[k] = c[k] / sigma and
// f_r = 2^e_r scale log2(e).  sigma is the codebook's scale (ServeTables); e_r, one number a row,
// puts the largest operand that R, S and the row's largest |q| allow into [2^14, 2^15), so that fp16
// operands neither overflow nor lose their low halves.
//
// Softmax with the value norms inside.  With y = z + log2 ||v_t|| and a running reference
// N >= y - kHeadroom the weights w = 2^(y - N) are what multiplies the value centroids, and the
// normaliser is l = sum w / ||v_t||; both have the factor 2^-N, so
//   out = R^T (sum_t w_t c[vidx_t]) / l
// needs no product with ||v_t|| and w stays inside the range of 16-bit floats whatever the norms
// are (||v_t|| is taken as 2^-24, fp16's smallest number, where it is 0, with c as 0).
// A partial result of a row is (N, l, o = sum_t w_t c[vidx_t]); partials merge by their N.
#pragma once

#include "tq_common.cuh"
#include "tq_internal.cuh"

namespace tq {

constexpr int kSms = 148;        // grid sizing (fixed so that scratch sizes do not vary)
constexpr int kStage = 32;       // tokens of one copy stage: the unit in which contexts are divided
// The tensor-core kernels round weights to fp16, whose numbers end at 65504 and 2^-24.  A new reference
// puts the largest weight at 2^kTopWeight; it may grow to 2^kHeadroom before the next one (a rescaling
// of the sums, so not for every new maximum).  So a weight is rounded to 2^-11 of itself, or to 2^-32
// of the largest at worst.  With the largest at 1 and 2^8, two million tokens of a CTA at 2^-25.3, 5% of
// its softmax, are lost whole: 4.6% off, against 1.3% this way, most of it the 32-bit sum's.
constexpr float kTopWeight = 7.f, kHeadroom = 15.f;
constexpr float kMinNorm = 5.9604644775390625e-8f;  // 2^-24
constexpr float kLog2eF = 1.4426950408889634f;

__host__ __device__ constexpr int partial_stride(int d) { return d + 4; }  // (N, l, -, -, o[d])

// The caches of one attention pass.  `slices` slices of records, `stride` records apart; slice s
// belongs to sequence s / per_seq and holds len[s / per_seq] tokens.  A slice is attended by
// `rows` query rows, of which row r is row (r / rows_in) * rows_outer + s * rows_in + r % rows_in
// of the call's queries [B, Hkv, rows_in].
struct RaggedCache {
    const uint32_t *kcodes, *ksigns;
    const uint16_t *knorm, *krnorm;
    const uint32_t *vcodes;
    const uint16_t *vnorm;
    int64_t stride, records;  // records of the whole array (no read goes past it)
    int slices, per_seq, nseq;
    int rows, rows_in;
    int64_t rows_outer;
    const int32_t *len;  // device, [nseq], within [0, stride]
    const int64_t *cum;  // device, [nseq + 1]: counted stages of the sequences before (of one slice each)
    int ctas;            // CTAs the stages of all slices are divided among
};

__device__ __forceinline__ int64_t ragged_row(const RaggedCache &c, int slice, int r) {
    return (int64_t)(r / c.rows_in) * c.rows_outer + (int64_t)slice * c.rows_in + r % c.rows_in;
}

// The W stages of all slices, in order, are divided evenly among G = min(ctas, W) CTAs, so that none
// of these is without work; CTA i takes stages [i W / G, (i + 1) W / G) and so a piece of one or
// more slices.  A slice that is not empty counts kPieceCost stages more than it has, in front, for
// what a piece costs besides its stages (its first loads, its partial result).  Slice s's piece in
// CTA i has the partial number i + s: from one piece to the next either i or s grows, so no two
// pieces share one.
constexpr int kPieceCost = 3;
__host__ __device__ constexpr int64_t counted_stages(int64_t tokens) {
    return tokens > 0 ? (tokens + kStage - 1) / kStage + kPieceCost : 0;
}

struct Piece {
    int slice;
    int64_t s0, s1;   // stages of the slice (there may be none)
    int64_t counted;  // what the piece counts in the division
    int len;          // tokens of the slice
};

__device__ __forceinline__ int64_t ragged_total(const RaggedCache &c) { return c.cum[c.nseq] * c.per_seq; }
__device__ __forceinline__ int64_t cta_first(int64_t total, int ctas, int i) {
    const int64_t g = total < ctas ? total : ctas;
    return i >= g ? total : total * i / g;
}

// The piece that starts at stage w (< w1) of the division.  Called by whole warps.
__device__ __forceinline__ Piece piece_at(const RaggedCache &c, int64_t w, int64_t w1) {
    // the last sequence whose first stage is <= w: it has stages (all lanes of a warp look together)
    int lo = -1;
    for (int b0 = 0; b0 < c.nseq; b0 += 32) {
        const int b = b0 + (int)(threadIdx.x & 31);
        const int before = __popc(__ballot_sync(kFull, b < c.nseq && c.cum[b] * c.per_seq <= w));
        lo += before;
        if (before < 32) break;
    }
    const int64_t base = c.cum[lo] * c.per_seq, n = c.cum[lo + 1] - c.cum[lo];
    const int64_t h = (w - base) / n;
    Piece p;
    p.slice = (int)(lo * (int64_t)c.per_seq + h);
    const int64_t v0 = w - base - h * n, v1 = v0 + (w1 - w) < n ? v0 + (w1 - w) : n;
    p.counted = v1 - v0;
    p.s0 = v0 > kPieceCost ? v0 - kPieceCost : 0;
    p.s1 = v1 > kPieceCost ? v1 - kPieceCost : 0;
    p.len = c.len[lo];
    return p;
}

// The CTAs [first, last] that hold pieces of a slice; false when the slice is empty.
__device__ __forceinline__ bool slice_ctas(const RaggedCache &c, int slice, int *first, int *last) {
    const int b = slice / c.per_seq;
    const int64_t n = c.cum[b + 1] - c.cum[b];
    if (n == 0) return false;
    const int64_t total = ragged_total(c), g = total < c.ctas ? total : c.ctas;
    const int64_t w0 = c.cum[b] * c.per_seq + (int64_t)(slice - b * c.per_seq) * n, w1 = w0 + n - 1;
    // CTA i holds w exactly when floor(W i / G) <= w < floor(W (i + 1) / G)
    *first = (int)(((w0 + 1) * g - 1) / total);
    *last = (int)(((w1 + 1) * g - 1) / total);
    return true;
}

// ---- operand order.  The sums over coordinates are free in their order, so the query operands are
// laid out the way the kernels decode the packed words.

// Register kernels (tq_ragged_mma.cuh): element e (0..3) of lane t4's operand in product ks of the
// code part.  A lane takes whole words (half a word at 64 coordinates).  3-bit codes: nibble 4 h + e
// of selector i holds bit 4 (4 h + e) + i of a word.  2-bit codes: byte e of selector i holds bit
// 8 e + i.  1-bit codes are taken as the signs are.
__host__ __device__ constexpr int frag_code_coord(int D, int KB, int t4, int ks, int e) {
    const int ng = D >= 128 ? D / 128 : 1;
    if (KB == 1) {
        const int pairs = D >= 128 ? 16 : 8, j = 2 * ks + (e >> 1);
        const int g = D >= 128 ? t4 * ng + j / pairs : t4 >> 1;
        return 32 * g + (D >= 128 ? 0 : 8 * (t4 & 1)) + j % pairs + 16 * (e & 1);
    }
    if (KB == 2) {
        const int ni = D >= 128 ? 8 : 4, g = D >= 128 ? t4 * ng + ks / ni : t4 >> 1;
        return 32 * g + 8 * e + ks % ni + (D >= 128 ? 0 : 4 * (t4 & 1));
    }
    const int ni = D >= 128 ? 4 : 2, h = ks & 1, i = (ks >> 1) % ni;
    const int g = D >= 128 ? t4 * ng + (ks >> 1) / ni : t4 >> 1;
    return 32 * g + 4 * (4 * h + e) + i + (D >= 128 ? 0 : 2 * (t4 & 1));
}
// ... and of the sign part: pairs of bits (l, l + 16), D / 16 pairs a lane.
__host__ __device__ constexpr int frag_sign_coord(int D, int t4, int ks, int e) {
    const int lpw = 256 / D, pw = D / 16;
    return 32 * (t4 / lpw) + (t4 % lpw) * pw + 2 * ks + (e >> 1) + 16 * (e & 1);
}
// The inverse: operand index c (codes 0 .. D-1, then signs) to 4 (4 ks + t4) + e.
__host__ __device__ constexpr int frag_place(int D, int KB, int c) {
    if (c >= D) {
        const int s = c - D, lpw = 256 / D, pw = D / 16, word = s >> 5, l = s & 15, up = (s >> 4) & 1;
        const int t4 = word * lpw + l / pw, j = l % pw;
        return 4 * (4 * (D / 16 + j / 2) + t4) + 2 * (j & 1) + up;
    }
    const int g = c >> 5, bit = c & 31, ng = D >= 128 ? D / 128 : 1;
    if (KB == 1) {
        const int pairs = D >= 128 ? 16 : 8, l = bit & 15, up = bit >> 4;
        const int t4 = D >= 128 ? g / ng : 2 * g + (l >> 3);
        const int j = (D >= 128 ? (g % ng) * pairs : 0) + l % pairs;
        return 4 * (4 * (j / 2) + t4) + 2 * (j & 1) + up;
    }
    if (KB == 2) {
        const int i8 = bit & 7, t4 = D >= 128 ? g / ng : 2 * g + (i8 >> 2);
        const int ks = D >= 128 ? (g % ng) * 8 + i8 : i8 & 3;
        return 4 * (4 * ks + t4) + (bit >> 3);
    }
    const int ni = D >= 128 ? 4 : 2, nib = bit >> 2, i4 = bit & 3;
    const int t4 = D >= 128 ? g / ng : 2 * g + (i4 >> 1), i = D >= 128 ? i4 : i4 & 1;
    const int ks = ((D >= 128 ? g % ng : 0) * ni + i) * 2 + (nib >> 2);
    return 4 * (4 * ks + t4) + (nib & 3);
}

// Prefix kernel (tq_prefix_tc.cu): the column of operand index c (codes, then signs) in a query row.
__host__ __device__ constexpr int prefix_column(int D, int c) {
    const int g = c & ~31, bit = c & 31;
    return c < D ? g + 8 * (bit & 3) + (bit >> 2) : g + 2 * (bit & 15) + (bit >> 4);
}
__host__ __device__ constexpr int prefix_tile(int D) { return D <= 128 ? 128 : 64; }  // tokens of a tile

struct PrefixSplit {
    int splits, tiles_per;
};
PrefixSplit prefix_split(int d, int Hkv, int64_t rows, int64_t t_prefix);
// Partials [split][KV head][row] of c.rows rows on a prefix of c.stride tokens; qrows: fp16
// [KV heads, c.rows, d + m] in prefix_column order.
cudaError_t launch_prefix_tc(const Prepared &P, const RaggedCache &c, const uint16_t *qrows, const float *fscale,
                             float *part, const PrefixSplit &sp, int32_t *dev_status, cudaStream_t s);

// One call of tq_attend_shared or tq_attend_weigh.
struct ServeCall {
    Prepared P;
    const void *q;
    void *out;
    tq_dtype dtype;
    int B, Hq, Hkv, Nq;
    int64_t rows;  // B * Hq * Nq
    float scale;
    RaggedCache own, prefix;  // prefix.slices == 0: none; own.slices == 0: none
    const int32_t *lens;      // the caller's, device
    int64_t t_cap, t_prefix;
    float *weights;           // tq_attend_weigh
    int32_t *dev_status;
};

// How a call is computed: by sizes alone, so that the scratch size follows from them too.
struct ServePlan {
    bool fast;         // the tensor-core kernels (else the plain kernel)
    int row_block;     // query rows a CTA of the ragged kernel takes
    int own_ctas;      // division of the own caches (0: no own caches)
    int prefix_ctas;   // division of the prefix by the ragged kernel (0: not by it)
    PrefixSplit tc;    // splits of the prefix by the many-row kernel (0: not by it)
    // byte offsets in the scratch
    size_t lens, cum, qprep, own_frag, pre_frag, qrows, fscale, lse, zbuf, own_part, pre_part, total;
};

ServePlan plan_serve(const Prepared &P, tq_dtype dtype, int B, int Hq, int Hkv, int Nq, int64_t t_prefix,
                     int64_t t_cap, bool weigh);
cudaError_t launch_serve(const ServeCall &call, const ServePlan &plan, void *scratch, cudaStream_t s);

// Pieces of a launch_serve (each in its file)
struct RaggedArgs {
    Prepared P;
    RaggedCache c;
    const float *qprep;   // plain kernel: [rows, d + m], (Q, P) of each row
    const uint2 *frag;    // tensor cores: [slices, row blocks][row tiles of 4][products][32 lanes]
    const float *fscale;  // [rows]
    float *part;          // partials, [(ctas + slices) * c.rows, d + 4]
    float *zbuf;          // z of every (row of the slice, token): [slices, rows, stride], or null
};
cudaError_t launch_ragged_plain(const RaggedArgs &a, cudaStream_t s);
bool ragged_mma_supported(const Prepared &P);
int ragged_mma_rows(const Prepared &P, int64_t rows, int64_t stages);  // the row block for so many rows a slice
int ragged_mma_ctas_per_sm(const Prepared &P);
// One launch for the own caches and the prefix (those that the plan gives CTAs).
struct RaggedPair {
    RaggedArgs a[2];
    uint32_t two16;    // 65536
    int first, total;  // CTAs of a[0], and of both; CTA i of a cache: division i % ctas, row block i / ctas
};
cudaError_t launch_ragged_mma(const RaggedArgs &own, const RaggedArgs &prefix, const ServePlan &plan, bool f32,
                              cudaStream_t s);
// cudaFuncSetAttribute for a kernel's dynamic shared memory, once for each kernel and device.
cudaError_t allow_smem(const void *kernel, size_t bytes);

}  // namespace tq
