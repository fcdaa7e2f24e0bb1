// C ABI of the latent-space operators: host-side argument checks and the launch
// sequence of each entry point (conventions of dspark_capi.cu).
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>

#include "dspark_latent.cuh"

using namespace dspark;

namespace {

#define DSPARK_TRY(x)                          \
    do {                                       \
        dspark_status _s = (x);                \
        if (_s != DSPARK_OK) return _s;        \
    } while (0)

bool verbose() {
    static const bool v = getenv("DSPARK_VERBOSE") != nullptr;
    return v;
}

#define DSPARK_CUDA(x)                                                                             \
    do {                                                                                           \
        const cudaError_t _e = (x);                                                                \
        if (_e != cudaSuccess) {                                                                   \
            if (verbose()) fprintf(stderr, "dspark: %s failed: %s\n", #x, cudaGetErrorString(_e)); \
            return DSPARK_ERR_CUDA;                                                                \
        }                                                                                          \
    } while (0)

bool aligned(const void *x, uintptr_t n) { return ((uintptr_t)x & (n - 1)) == 0; }

dspark_status need(const void *ptr, size_t elems, uintptr_t align) {
    if (elems == 0) return DSPARK_OK;
    if (!ptr) return DSPARK_ERR_NULL;
    return aligned(ptr, align) ? DSPARK_OK : DSPARK_ERR_ALIGN;
}

bool good_base(double b) { return b > 0.0 && std::isfinite(b); }

dspark_status make_lat(const dspark_latent_problem *pp, Prob *out) {
    if (!pp) return DSPARK_ERR_NULL;
    const dspark_latent_problem &p = *pp;
    if (p.dtype != DSPARK_F32 && p.dtype != DSPARK_BF16) return DSPARK_ERR_DTYPE;
    if (p.reserved[0] != 0 || p.reserved[1] != 0 || p.B < 0 || p.n_h < 1 || p.S < 1 || p.N < 0 || p.W < 1 ||
        p.d_l < 1 || p.d_r < 0 || (p.d_r & 1) || !good_base(p.rope_base) || !(p.scale > 0.0) ||
        !std::isfinite(p.scale))
        return DSPARK_ERR_SHAPE;
    if (p.W > 4096 || p.N > 8192 || p.d_l > 512 || p.d_r > 128 || p.B > 65535) return DSPARK_ERR_UNSUPPORTED;
    const long long L = (long long)p.S + (long long)kBlock * p.N, R = (long long)kBlock * p.N;
    const long long lim = 1ll << 31;
    // (the products stay below 2^63: p.n_h < 2^31, R < 2^16, widths < 2^10)
    if (L * std::max(p.d_l, p.d_r) >= lim || R * p.n_h * (p.d_l + p.d_r) >= lim || (long long)p.S + 8 >= (1ll << 30) ||
        (long long)p.B * p.n_h * R >= lim)
        return DSPARK_ERR_UNSUPPORTED;
    Prob r{};
    r.B = p.B; r.n_h = p.n_h; r.S = p.S; r.N = p.N; r.W = p.W;
    r.d_c = r.d_v = p.d_l;
    r.d_r = p.d_r;
    r.dqk = p.d_l + p.d_r;
    r.R = (int)R;
    r.L = (int)L;
    r.P = p.S + 8;
    r.base = p.rope_base;
    r.dtype = p.dtype;
    r.scale = (float)p.scale;
    r.scale_log2 = (float)(p.scale * 1.4426950408889634);
    r.wait_ns = wait_limit_ns();
    *out = r;
    return DSPARK_OK;
}

dspark_status check_lat(const Prob &p, const void *q, const void *c, const void *kr, const int32_t *anchors,
                        const uint8_t *keep, void *ws, size_t bytes, bool bwd) {
    const LatWsLayout l = lat_layout(p);
    if (!ws || !aligned(ws, 256) || bytes < (bwd ? l.total : l.fwd_total)) return DSPARK_ERR_WORKSPACE;
    DSPARK_TRY(need(q, (size_t)p.B * p.n_h * p.R * p.dqk, 16));
    DSPARK_TRY(need(c, (size_t)p.B * p.L * p.d_c, 16));
    DSPARK_TRY(need(kr, (size_t)p.B * p.L * p.d_r, 16));
    if ((size_t)p.B * p.N && (!anchors || !keep)) return DSPARK_ERR_NULL;
    if ((size_t)p.B * p.N && !aligned(anchors, 4)) return DSPARK_ERR_ALIGN;
    return DSPARK_OK;
}

bool good_widths(int kind, int d_l, int d_r) {
    if (kind != DSPARK_CACHE_F32 && kind != DSPARK_CACHE_BF16 && kind != DSPARK_CACHE_FP8) return false;
    return d_l >= 8 && d_l <= 512 && d_l % (kind == DSPARK_CACHE_FP8 ? 128 : 8) == 0 && d_r >= 0 && d_r <= 128 &&
           d_r % 8 == 0;
}

dspark_status check_cache(const dspark_latent_cache *pp) {
    if (!pp) return DSPARK_ERR_NULL;
    if (pp->dtype != DSPARK_F32 && pp->dtype != DSPARK_BF16) return DSPARK_ERR_DTYPE;
    if (pp->kind != DSPARK_CACHE_F32 && pp->kind != DSPARK_CACHE_BF16 && pp->kind != DSPARK_CACHE_FP8)
        return DSPARK_ERR_DTYPE;
    if (pp->reserved != 0 || pp->T < 0 || pp->n_pages < 0 || pp->page_size < 1) return DSPARK_ERR_SHAPE;
    // (the last CTA's tokens are counted past T in 32 bits)
    if (pp->T > INT32_MAX - 63) return DSPARK_ERR_UNSUPPORTED;
    return good_widths(pp->kind, pp->d_l, pp->d_r) ? DSPARK_OK : DSPARK_ERR_UNSUPPORTED;
}

dspark_status make_paged(const dspark_latent_paged *pp, Paged *out) {
    if (!pp) return DSPARK_ERR_NULL;
    const dspark_latent_paged &p = *pp;
    if (p.kind != DSPARK_CACHE_F32 && p.kind != DSPARK_CACHE_BF16 && p.kind != DSPARK_CACHE_FP8)
        return DSPARK_ERR_DTYPE;
    if (p.dtype != (p.kind == DSPARK_CACHE_F32 ? DSPARK_F32 : DSPARK_BF16)) return DSPARK_ERR_DTYPE;
    if (p.reserved != 0 || p.n_seq < 0 || p.T < 0 || p.n_h < 1 || p.page_size < 1 || p.n_pages < 0 ||
        p.max_pages < 0 || p.max_kv_len < 0 || p.window < 0 || (p.causal != 0 && p.causal != 1) ||
        !good_base(p.rope_base) || !(p.scale > 0.0) || !std::isfinite(p.scale))
        return DSPARK_ERR_SHAPE;
    if (!good_widths(p.kind, p.d_l, p.d_r)) return DSPARK_ERR_UNSUPPORTED;
    const long long lim = 1ll << 31;
    if ((long long)p.T * p.n_h >= lim || (long long)p.max_pages * p.page_size >= lim || p.n_seq >= (1 << 24) ||
        (long long)p.n_pages * p.page_size >= lim)
        return DSPARK_ERR_UNSUPPORTED;
    Paged r{};
    r.n_seq = p.n_seq; r.T = p.T; r.n_h = p.n_h; r.d_l = p.d_l; r.d_r = p.d_r;
    r.page_size = p.page_size; r.n_pages = p.n_pages; r.max_pages = p.max_pages;
    const int cap = p.max_pages * p.page_size;
    r.max_kv = p.max_kv_len > 0 ? std::min(p.max_kv_len, cap) : cap;
    r.window = p.window; r.causal = p.causal; r.dtype = p.dtype; r.kind = p.kind;
    const int dk = p.d_l + p.d_r, per16 = p.dtype == DSPARK_F32 ? 4 : 8;
    r.q_ts = p.q_token_stride; r.q_hs = p.q_head_stride; r.o_ts = p.o_token_stride; r.o_hs = p.o_head_stride;
    if (r.q_ts == 0 && r.q_hs == 0) {
        r.q_ts = (long long)p.n_h * dk;
        r.q_hs = dk;
    }
    if (r.o_ts == 0 && r.o_hs == 0) {
        r.o_ts = (long long)p.n_h * p.d_l;
        r.o_hs = p.d_l;
    }
    if (r.q_ts < 0 || r.q_hs < 0 || r.o_ts < 0 || r.o_hs < 0 || (r.q_ts == 0 && p.T > 1) || (r.q_hs == 0 && p.n_h > 1))
        return DSPARK_ERR_SHAPE;
    if (r.q_ts % per16 || r.q_hs % per16 || r.o_ts % per16 || r.o_hs % per16) return DSPARK_ERR_ALIGN;
    // strides far outside any tensor would overflow the address arithmetic
    const long long far = 1ll << 39;
    if (r.q_ts >= far || r.q_hs >= far || r.o_ts >= far || r.o_hs >= far) return DSPARK_ERR_UNSUPPORTED;
    // output rows must not overlap: tokens apart by more than a token's heads reach, or the reverse
    const bool tok_major = (p.T <= 1 || r.o_ts >= (long long)(p.n_h - 1) * r.o_hs + p.d_l) &&
                           (p.n_h <= 1 || r.o_hs >= p.d_l);
    const bool head_major = (p.n_h <= 1 || r.o_hs >= (long long)(p.T - 1) * r.o_ts + p.d_l) &&
                            (p.T <= 1 || r.o_ts >= p.d_l);
    if (!tok_major && !head_major) return DSPARK_ERR_SHAPE;
    r.row_bytes = cache_row_bytes(p.kind, p.d_l, p.d_r);
    r.scale = (float)p.scale;
    r.scale_log2 = (float)(p.scale * 1.4426950408889634);
    r.wait_ns = wait_limit_ns();
    r.freq = rope_freq(p.d_r, p.rope_base);
    *out = r;
    return DSPARK_OK;
}

}  // namespace

extern "C" {

size_t dspark_latent_workspace_size(const dspark_latent_problem *pp) {
    Prob p;
    return make_lat(pp, &p) == DSPARK_OK ? lat_layout(p).total : 0;
}

dspark_status dspark_latent_attn_fwd(const dspark_latent_problem *pp, const void *q, const void *c, const void *kr,
                                     const int32_t *anchors, const uint8_t *keep, void *o, float *lse,
                                     void *workspace, size_t workspace_bytes, uint32_t flags, void *stream) {
    Prob p;
    DSPARK_TRY(make_lat(pp, &p));
    DSPARK_TRY(check_lat(p, q, c, kr, anchors, keep, workspace, workspace_bytes, false));
    DSPARK_TRY(need(o, (size_t)p.B * p.n_h * p.R * p.d_c, 16));
    DSPARK_TRY(need(lse, (size_t)p.B * p.n_h * p.R, 4));
    cudaStream_t st = (cudaStream_t)stream;
    const LatWs w = lat_view(p, workspace);
    if (!(flags & DSPARK_FLAG_REUSE_DESCRIPTOR)) DSPARK_CUDA(launch_build_descriptor(p, anchors, keep, w.base, st));
    const bool tc = lat_tc_supported(p);
    PadRows pad{};  // the tensor-core kernel leaves padding blocks' rows to the preparation
    pad.t[0] = o;
    pad.rows[0] = p.R;
    pad.width[0] = p.d_c;
    pad.lse = lse;
    DSPARK_CUDA(launch_lat_prep(p, kr, anchors, keep, tc ? &pad : nullptr, tc, false, nullptr, w, st));
    if (tc)
        DSPARK_CUDA(launch_lat_fwd_tc(p, q, c, o, lse, w, st));
    else
        DSPARK_CUDA(launch_lat_fwd_simt(p, q, c, anchors, keep, o, lse, w, st));
    return DSPARK_OK;
}

dspark_status dspark_latent_attn_bwd(const dspark_latent_problem *pp, const void *q, const void *c, const void *kr,
                                     const int32_t *anchors, const uint8_t *keep, const float *lse, const void *do_,
                                     void *dq, void *dc, void *dkr, void *workspace, size_t workspace_bytes,
                                     uint32_t flags, void *stream) {
    Prob p;
    DSPARK_TRY(make_lat(pp, &p));
    DSPARK_TRY(check_lat(p, q, c, kr, anchors, keep, workspace, workspace_bytes, true));
    DSPARK_TRY(need(lse, (size_t)p.B * p.n_h * p.R, 4));
    DSPARK_TRY(need(do_, (size_t)p.B * p.n_h * p.R * p.d_c, 16));
    DSPARK_TRY(need(dq, (size_t)p.B * p.n_h * p.R * p.dqk, 16));
    DSPARK_TRY(need(dc, (size_t)p.B * p.L * p.d_c, 16));
    DSPARK_TRY(need(dkr, (size_t)p.B * p.L * p.d_r, 16));
    cudaStream_t st = (cudaStream_t)stream;
    const LatWs w = lat_view(p, workspace);
    if (!(flags & DSPARK_FLAG_REUSE_DESCRIPTOR)) DSPARK_CUDA(launch_build_descriptor(p, anchors, keep, w.base, st));
    const bool tc = lat_bwd_tc_supported(p);
    PadRows pad{};
    pad.t[0] = dq;
    pad.rows[0] = p.R;
    pad.width[0] = p.dqk;
    DSPARK_CUDA(launch_lat_prep(p, kr, anchors, keep, tc ? &pad : nullptr, tc, tc, q, w, st));
    if (tc)
        DSPARK_CUDA(launch_lat_bwd_tc(p, q, c, anchors, lse, do_, dq, dc, dkr, w, st));
    else
        DSPARK_CUDA(launch_lat_bwd_simt(p, q, c, anchors, keep, lse, do_, dq, dc, dkr, w, st));
    return DSPARK_OK;
}

size_t dspark_latent_row_bytes(int32_t kind, int32_t d_l, int32_t d_r) {
    return good_widths(kind, d_l, d_r) ? cache_row_bytes(kind, d_l, d_r) : 0;
}

dspark_status dspark_latent_cache_write(const dspark_latent_cache *p, const void *c, const void *kr,
                                        const void *norm_weight, double eps, double rope_base,
                                        const int32_t *positions, const int64_t *slots, void *cache, void *stream) {
    DSPARK_TRY(check_cache(p));
    if (!(eps >= 0.0) || !std::isfinite(eps) || !good_base(rope_base)) return DSPARK_ERR_SHAPE;
    DSPARK_TRY(need(c, (size_t)p->T * p->d_l, 16));
    DSPARK_TRY(need(kr, (size_t)p->T * p->d_r, 16));
    if (norm_weight && !aligned(norm_weight, 16)) return DSPARK_ERR_ALIGN;
    DSPARK_TRY(need(positions, (size_t)p->T, 4));
    DSPARK_TRY(need(slots, (size_t)p->T, 8));
    DSPARK_TRY(need(cache, p->T > 0 ? (size_t)p->n_pages * p->page_size : 0, 16));
    DSPARK_CUDA(launch_cache_write(*p, c, kr, norm_weight, eps, rope_freq(p->d_r, rope_base), positions, slots, cache,
                                   (cudaStream_t)stream));
    return DSPARK_OK;
}

dspark_status dspark_latent_cache_read(const dspark_latent_cache *p, const void *cache, const int64_t *slots,
                                       void *c_out, void *kr_out, void *stream) {
    DSPARK_TRY(check_cache(p));
    DSPARK_TRY(need(c_out, (size_t)p->T * p->d_l, 16));
    if (kr_out && !aligned(kr_out, 16)) return DSPARK_ERR_ALIGN;
    DSPARK_TRY(need(slots, (size_t)p->T, 8));
    DSPARK_TRY(need(cache, p->T > 0 ? (size_t)p->n_pages * p->page_size : 0, 16));
    DSPARK_CUDA(launch_cache_read(*p, cache, slots, c_out, p->d_r ? kr_out : nullptr, (cudaStream_t)stream));
    return DSPARK_OK;
}

size_t dspark_latent_paged_workspace_size(const dspark_latent_paged *pp) {
    Paged p;
    return make_paged(pp, &p) == DSPARK_OK ? paged_workspace_size(p) : 0;
}

dspark_status dspark_latent_attn_paged(const dspark_latent_paged *pp, const void *q, const void *cache,
                                       const int32_t *block_table, const int32_t *q_start, const int32_t *kv_len,
                                       void *o, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    Paged p;
    DSPARK_TRY(make_paged(pp, &p));
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < paged_workspace_size(p))
        return DSPARK_ERR_WORKSPACE;
    const size_t rows = (size_t)p.T * p.n_h;
    DSPARK_TRY(need(q, rows, 16));
    DSPARK_TRY(need(o, rows, 16));
    DSPARK_TRY(need(lse, rows, 4));
    DSPARK_TRY(need(cache, (size_t)p.n_pages * p.page_size, 16));
    DSPARK_TRY(need(block_table, (size_t)p.n_seq * p.max_pages, 4));
    DSPARK_TRY(need(q_start, (size_t)p.n_seq, 4));
    DSPARK_TRY(need(kv_len, (size_t)p.n_seq, 4));
    p.q = q;
    p.cache = cache;
    p.table = block_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.o = o;
    p.lse = lse;
    DSPARK_CUDA(launch_paged(p, workspace, (cudaStream_t)stream));
    return DSPARK_OK;
}

}  // extern "C"
