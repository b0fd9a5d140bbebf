// tq_serve_api.cu -- the extern "C" entry points for serving over caches of different lengths:
// argument checks, then launches.
#include <cmath>
#include <cstring>

#include "tq_evict.cuh"
#include "tq_serve.cuh"

using namespace tq;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

constexpr int64_t kMaxTokens = (int64_t)INT32_MAX - 1023;
constexpr int64_t kMaxRowsTotal = 65535 * 4;  // blocks of four rows in a grid's second dimension

tq_status check_params(const tq_params *p) {
    if (!p) return TQ_ERR_INVALID_ARG;
    if (p->dim < 32 || p->dim > kMaxDim || p->dim % 32) return TQ_ERR_INVALID_ARG;
    if (p->bits < 2 || p->bits > 4) return TQ_ERR_INVALID_ARG;
    if (p->proj_dim < 32 || p->proj_dim > kMaxProj || p->proj_dim % 32) return TQ_ERR_INVALID_ARG;
    if (!p->workspace || !aligned16(p->workspace)) return TQ_ERR_INVALID_ARG;
    if (p->workspace_bytes < ws_layout(p->dim, p->proj_dim).total) return TQ_ERR_INVALID_ARG;
    const int d = p->dim;
    return (d & (d - 1)) == 0 ? TQ_OK : TQ_ERR_UNSUPPORTED;  // 32, 64, ..., 1024, as the other calls
}

tq_status check_shape(tq_dtype dtype, int B, int Hq, int Hkv, int Nq, int64_t t_prefix, int64_t t_cap) {
    if (dtype != TQ_F16 && dtype != TQ_F32 && dtype != TQ_BF16) return TQ_ERR_INVALID_ARG;
    if (B < 1 || Hq < 1 || Hkv < 1 || Nq < 1 || Hq % Hkv) return TQ_ERR_INVALID_ARG;
    if (t_prefix < 0 || t_cap < 0 || t_prefix + t_cap < 1) return TQ_ERR_INVALID_ARG;
    if (t_prefix > kMaxTokens || t_cap > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    // CTAs that add up the weights of 1024 slots each
    if ((t_cap + 1023) / 1024 * B > INT32_MAX / 2 / Hkv) return TQ_ERR_UNSUPPORTED;
    if ((int64_t)B * Hq > kMaxRowsTotal || (int64_t)B * Hq * Nq > kMaxRowsTotal) return TQ_ERR_UNSUPPORTED;
    return TQ_OK;
}

bool good(const void *p) { return p && aligned16(p); }

// What a call reads and what it writes.
struct Range {
    const void *at;
    size_t bytes;
};
bool overlap(const Range &a, const Range &b) {
    const uintptr_t x = (uintptr_t)a.at, y = (uintptr_t)b.at;
    return a.at && b.at && x < y + b.bytes && y < x + a.bytes;
}
// No written range may lie in one that is read, nor in another written one.
bool apart(const Range *written, int nw, const Range *read, int nr) {
    for (int i = 0; i < nw; ++i) {
        for (int j = 0; j < nr; ++j)
            if (overlap(written[i], read[j])) return false;
        for (int j = 0; j < i; ++j)
            if (overlap(written[i], written[j])) return false;
    }
    return true;
}

// One attention call; weights is null for tq_attend_shared.
tq_status attend(const tq_params *p, const void *q, tq_dtype dtype, int B, int Hq, int Hkv, int Nq, int64_t t_prefix,
                 const RaggedCache &prefix, const int32_t *lens, int64_t t_cap, const RaggedCache &own, float scale,
                 float *weights, void *out, void *scratch, size_t scratch_bytes, int32_t *dev_status,
                 tq_stream_t stream) {
    tq_status st = check_params(p);
    if (st != TQ_OK) return st;
    st = check_shape(dtype, B, Hq, Hkv, Nq, t_prefix, t_cap);
    if (st != TQ_OK) return st;
    if (!good(q) || !good(out) || !good(scratch)) return TQ_ERR_INVALID_ARG;
    for (const RaggedCache *c : {&prefix, &own}) {
        if ((c == &prefix ? t_prefix : t_cap) == 0) continue;
        if (!good(c->kcodes) || !good(c->ksigns) || !good(c->knorm) || !good(c->krnorm) || !good(c->vcodes) ||
            !good(c->vnorm))
            return TQ_ERR_INVALID_ARG;
    }
    if (t_cap > 0 && !good(lens)) return TQ_ERR_INVALID_ARG;
    if (!(scale == scale)) return TQ_ERR_INVALID_ARG;  // NaN
    ServeCall call;
    memset(&call, 0, sizeof(call));
    call.P = prepared_view(p);
    const ServePlan plan = plan_serve(call.P, dtype, B, Hq, Hkv, Nq, t_prefix, t_cap, weights != nullptr);
    if (scratch_bytes < plan.total) return TQ_ERR_INVALID_ARG;
    // Kernels of the call run beside one another, and one reads what another has left in the scratch.
    // (out may be q: it is written when the rows have been read.)
    const size_t rows = (size_t)B * Hq * Nq * p->dim * (dtype == TQ_F32 ? 4 : 2), d = p->dim;
    Range read[15] = {{q, rows}, {p->workspace, ws_layout(p->dim, p->proj_dim).total}, {t_cap > 0 ? lens : nullptr, sizeof(int32_t) * (size_t)B}};
    const Range written[4] = {{scratch, plan.total},
                              {weights, sizeof(float) * (size_t)B * Hkv * (size_t)t_cap},
                              {dev_status, sizeof(int32_t)},
                              {out, rows}};
    int nr = 3;
    for (const RaggedCache *c : {&prefix, &own}) {
        const size_t n = c == &prefix ? (size_t)Hkv * t_prefix : (size_t)B * Hkv * t_cap;
        if (n == 0) continue;
        read[nr++] = {c->kcodes, n * ((p->bits - 1) * d / 8)};
        read[nr++] = {c->ksigns, n * (size_t)(p->proj_dim / 8)};
        read[nr++] = {c->knorm, n * 2};
        read[nr++] = {c->krnorm, n * 2};
        read[nr++] = {c->vcodes, n * (p->bits * d / 8)};
        read[nr++] = {c->vnorm, n * 2};
    }
    if (!apart(written, 3, read, 1) || !apart(written, 4, read + 1, nr - 1)) return TQ_ERR_INVALID_ARG;
    call.q = q;
    call.out = out;
    call.dtype = dtype;
    call.B = B;
    call.Hq = Hq;
    call.Hkv = Hkv;
    call.Nq = Nq;
    call.rows = (int64_t)B * Hq * Nq;
    call.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)p->dim);
    call.own = own;
    call.own.stride = t_cap;
    call.own.records = (int64_t)B * Hkv * t_cap;
    call.prefix = prefix;
    call.prefix.stride = t_prefix;
    call.prefix.records = (int64_t)Hkv * t_prefix;
    call.lens = t_cap > 0 ? lens : nullptr;
    call.t_cap = t_cap;
    call.t_prefix = t_prefix;
    call.weights = weights;
    call.dev_status = dev_status;
    return launch_serve(call, plan, scratch, (cudaStream_t)stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

RaggedCache cache_of(const uint32_t *kcodes, const uint32_t *ksigns, const uint16_t *knorm, const uint16_t *krnorm,
                     const uint32_t *vcodes, const uint16_t *vnorm) {
    RaggedCache c;
    memset(&c, 0, sizeof(c));
    c.kcodes = kcodes;
    c.ksigns = ksigns;
    c.knorm = knorm;
    c.krnorm = krnorm;
    c.vcodes = vcodes;
    c.vnorm = vnorm;
    return c;
}

}  // namespace

extern "C" {

size_t tq_attend_shared_scratch_bytes(const tq_params *p, tq_dtype dtype, int B, int Hq, int Hkv, int Nq,
                                      int64_t t_prefix, int64_t t_cap) {
    if (check_params(p) != TQ_OK || check_shape(dtype, B, Hq, Hkv, Nq, t_prefix, t_cap) != TQ_OK) return 0;
    return plan_serve(prepared_view(p), dtype, B, Hq, Hkv, Nq, t_prefix, t_cap, false).total;
}

tq_status tq_attend_shared(const tq_params *p, const void *q, tq_dtype dtype, int B, int Hq, int Hkv, int Nq,
                           int64_t t_prefix, const uint32_t *pkcodes, const uint32_t *pksigns,
                           const uint16_t *pknorm, const uint16_t *pkrnorm, const uint32_t *pvcodes,
                           const uint16_t *pvnorm, const int32_t *lens, int64_t t_cap, const uint32_t *kcodes,
                           const uint32_t *ksigns, const uint16_t *knorm, const uint16_t *krnorm,
                           const uint32_t *vcodes, const uint16_t *vnorm, float scale, void *out, void *scratch,
                           size_t scratch_bytes, int32_t *dev_status, tq_stream_t stream) {
    return attend(p, q, dtype, B, Hq, Hkv, Nq, t_prefix,
                  cache_of(pkcodes, pksigns, pknorm, pkrnorm, pvcodes, pvnorm), lens, t_cap,
                  cache_of(kcodes, ksigns, knorm, krnorm, vcodes, vnorm), scale, nullptr, out, scratch,
                  scratch_bytes, dev_status, stream);
}

size_t tq_attend_weigh_scratch_bytes(const tq_params *p, tq_dtype dtype, int B, int Hq, int Hkv, int Nq,
                                     int64_t t_cap) {
    if (check_params(p) != TQ_OK || check_shape(dtype, B, Hq, Hkv, Nq, 0, t_cap) != TQ_OK) return 0;
    return plan_serve(prepared_view(p), dtype, B, Hq, Hkv, Nq, 0, t_cap, true).total;
}

tq_status tq_attend_weigh(const tq_params *p, const void *q, tq_dtype dtype, int B, int Hq, int Hkv, int Nq,
                          const int32_t *lens, int64_t t_cap, const uint32_t *kcodes, const uint32_t *ksigns,
                          const uint16_t *knorm, const uint16_t *krnorm, const uint32_t *vcodes,
                          const uint16_t *vnorm, float scale, float *weights, void *out, void *scratch,
                          size_t scratch_bytes, int32_t *dev_status, tq_stream_t stream) {
    if (!good(weights)) return TQ_ERR_INVALID_ARG;
    return attend(p, q, dtype, B, Hq, Hkv, Nq, 0, cache_of(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), lens,
                  t_cap, cache_of(kcodes, ksigns, knorm, krnorm, vcodes, vnorm), scale, weights, out, scratch,
                  scratch_bytes, dev_status, stream);
}

static tq_status check_evict(const tq_params *p, int B, int Hkv, int64_t t_cap, int64_t budget) {
    const tq_status st = check_params(p);
    if (st != TQ_OK) return st;
    if (B < 1 || Hkv < 1 || t_cap < 1 || budget < 1 || budget > t_cap) return TQ_ERR_INVALID_ARG;
    if (t_cap > kMaxTokens || (int64_t)B * Hkv > kMaxRowsTotal) return TQ_ERR_UNSUPPORTED;
    return evict_chunks(budget) * B * Hkv <= INT32_MAX ? TQ_OK : TQ_ERR_UNSUPPORTED;
}

size_t tq_evict_scratch_bytes(const tq_params *p, int B, int Hkv, int64_t t_cap, int64_t budget) {
    if (check_evict(p, B, Hkv, t_cap, budget) != TQ_OK) return 0;
    return evict_scratch_bytes(B, Hkv);
}

tq_status tq_evict(const tq_params *p, int B, int Hkv, const int32_t *lens, int64_t t_cap, const uint32_t *kcodes,
                   const uint32_t *ksigns, const uint16_t *knorm, const uint16_t *krnorm, const uint32_t *vcodes,
                   const uint16_t *vnorm, const float *weights, int64_t budget, int64_t recent, int64_t out_cap,
                   uint32_t *out_kcodes, uint32_t *out_ksigns, uint16_t *out_knorm, uint16_t *out_krnorm,
                   uint32_t *out_vcodes, uint16_t *out_vnorm, float *out_weights, int32_t *kept,
                   int32_t *out_lens, void *scratch, size_t scratch_bytes, int32_t *dev_status,
                   tq_stream_t stream) {
    tq_status st = check_evict(p, B, Hkv, t_cap, budget);
    if (st != TQ_OK) return st;
    if (recent < 0 || recent > budget || out_cap < budget) return TQ_ERR_INVALID_ARG;
    if (out_cap > kMaxTokens) return TQ_ERR_UNSUPPORTED;
    if (!good(lens) || !good(out_lens) || !good(kept) || !good(scratch)) return TQ_ERR_INVALID_ARG;
    if (scratch_bytes < evict_scratch_bytes(B, Hkv)) return TQ_ERR_INVALID_ARG;
    const int d = p->dim;
    EvictCall c;
    memset(&c, 0, sizeof(c));
    const void *src[] = {kcodes, ksigns, knorm, krnorm, vcodes, vnorm, weights};
    void *dst[] = {out_kcodes, out_ksigns, out_knorm, out_krnorm, out_vcodes, out_vnorm, out_weights};
    const int bytes[] = {(p->bits - 1) * d / 8, p->proj_dim / 8, 2, 2, p->bits * d / 8, 2, 4};
    const int64_t n_src = (int64_t)B * Hkv * t_cap, n_dst = (int64_t)B * Hkv * out_cap;
    for (int i = 0; i < kEvictArrays; ++i) {
        if (!good(src[i]) || !good(dst[i])) return TQ_ERR_INVALID_ARG;
        c.src[i] = src[i];
        c.dst[i] = dst[i];
        c.bytes[i] = bytes[i];
    }
    // The copies run in no order and take the kept slots and counts from memory.
    Range read[kEvictArrays + 1], written[kEvictArrays + 4];
    for (int i = 0; i < kEvictArrays; ++i) {
        read[i] = {src[i], (size_t)n_src * bytes[i]};
        written[i] = {dst[i], (size_t)n_dst * bytes[i]};
    }
    read[kEvictArrays] = {lens, sizeof(int32_t) * (size_t)B};
    written[kEvictArrays] = {kept, sizeof(int32_t) * (size_t)(B * (int64_t)Hkv * budget)};
    written[kEvictArrays + 1] = {out_lens, sizeof(int32_t) * (size_t)B};
    written[kEvictArrays + 2] = {scratch, evict_scratch_bytes(B, Hkv)};
    written[kEvictArrays + 3] = {dev_status, sizeof(int32_t)};
    if (!apart(written, kEvictArrays + 4, read, kEvictArrays + 1)) return TQ_ERR_INVALID_ARG;
    c.B = B;
    c.Hkv = Hkv;
    c.lens = lens;
    c.t_cap = t_cap;
    c.budget = budget;
    c.recent = recent;
    c.out_cap = out_cap;
    c.kept = kept;
    c.out_lens = out_lens;
    c.counts = (int32_t *)scratch;
    c.dev_status = dev_status;
    return launch_evict(c, (cudaStream_t)stream) == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // extern "C"
