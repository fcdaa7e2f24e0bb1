// Internal declarations of the latent-space operators: the problem views, the
// workspace layouts and the launch functions.
#pragma once

#include "../../include/dspark_latent.h"
#include <cuda_fp8.h>

#include "dspark_internal.cuh"

namespace dspark {

constexpr uint32_t kErrPage = 4u;  // error word bit: a page, kv_len or q_start out of range

// ---- training ----------------------------------------------------------------
// The Prob of dspark_internal.cuh with d_c = d_v = d_l, so that the mask
// descriptor and the rope-key rotation serve this family too.
struct LatWsLayout {
    size_t err, cnt, sorted_n, sorted_a, rope;  // as WsLayout
    size_t kr;     // turned rope keys [B, L, d_r]: fp32 (CUDA-core kernels) or bf16 hi, then bf16 lo
    size_t fwd_total;
    size_t dvec;   // float [B, n_h, 5N]: D = sum_k P dP (CUDA-core backward)
    size_t dacc;   // float [B, L, d_l + d_r]: key gradients (tensor-core backward)
    size_t q_rot;  // bf16 [B, n_h, 5N, 2 d_r]: turned rope queries, hi and lo (tensor-core backward)
    size_t total;
};

bool lat_tc_supported(const Prob &p);      // the tensor-core forward takes the problem
bool lat_bwd_tc_supported(const Prob &p);  // ... backward
uint64_t wait_limit_ns();  // limit of the pipeline waits in effect (dspark_set_wait_limit_ns)

inline LatWsLayout lat_layout(const Prob &p) {
    LatWsLayout w;
    size_t off = 0;
    w.err = off;       off = align256(off + 256);
    w.cnt = off;       off = align256(off + sizeof(int32_t) * (size_t)p.B);
    w.sorted_n = off;  off = align256(off + sizeof(int32_t) * (size_t)p.B * p.N);
    w.sorted_a = off;  off = align256(off + sizeof(int32_t) * (size_t)p.B * p.N);
    w.rope = off;      off = align256(off + sizeof(float2) * (size_t)p.P * (p.d_r / 2));
    w.kr = off;        off = align256(off + 4 * (size_t)p.B * p.L * p.d_r);
    w.fwd_total = off;
    const bool tc = lat_bwd_tc_supported(p);
    w.dvec = off;      off = align256(off + (tc ? 0 : sizeof(float) * (size_t)p.B * p.n_h * p.R));
    w.dacc = off;      off = align256(off + (tc ? sizeof(float) * (size_t)p.B * p.L * p.dqk : 0));
    w.q_rot = off;     off = align256(off + (tc ? 4 * (size_t)p.B * p.n_h * p.R * p.d_r : 0));
    w.total = off;
    return w;
}

struct LatWs {
    Ws base;  // err, cnt, sorted_n, sorted_a, rope
    float *kr_f32;
    __nv_bfloat16 *kr_hi, *kr_lo, *q_rot;
    float *dvec, *dacc;
};

inline LatWs lat_view(const Prob &p, void *ws) {
    const LatWsLayout l = lat_layout(p);
    char *c = (char *)ws;
    LatWs w{};
    w.base.err = (uint32_t *)(c + l.err);
    w.base.cnt = (int32_t *)(c + l.cnt);
    w.base.sorted_n = (int32_t *)(c + l.sorted_n);
    w.base.sorted_a = (int32_t *)(c + l.sorted_a);
    w.base.rope = (float2 *)(c + l.rope);
    w.kr_f32 = (float *)(c + l.kr);
    w.kr_hi = (__nv_bfloat16 *)(c + l.kr);
    w.kr_lo = w.kr_hi + (size_t)p.B * p.L * p.d_r;
    w.dvec = (float *)(c + l.dvec);
    w.dacc = (float *)(c + l.dacc);
    w.q_rot = (__nv_bfloat16 *)(c + l.q_rot);
    return w;
}

// What the tensor-core backward needs beside the turned rope keys.
constexpr int kTcDL = 512, kTcDR = 64;  // widths of the tensor-core kernels
struct BwdPrep {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;  // [rows, 2, 64]: turned rope slices, hi, lo
    float4 *acc;         // cleared
    size_t rows, acc4;
};

// turned rope keys; with pad != NULL, the padding blocks' rows of t[0] too; with
// bwd, BwdPrep for the queries q (tensor-core widths, bf16)
cudaError_t launch_lat_prep(const Prob &p, const void *kr, const int32_t *anchors, const uint8_t *keep,
                            const PadRows *pad, bool tc, bool bwd, const void *q, const LatWs &ws, cudaStream_t st);
cudaError_t launch_lat_fwd_tc(const Prob &p, const void *q, const void *c, void *o, float *lse, const LatWs &ws,
                              cudaStream_t st);
cudaError_t launch_lat_fwd_simt(const Prob &p, const void *q, const void *c, const int32_t *anchors,
                                const uint8_t *keep, void *o, float *lse, const LatWs &ws, cudaStream_t st);
cudaError_t launch_lat_bwd_tc(const Prob &p, const void *q, const void *c, const int32_t *anchors, const float *lse,
                              const void *dout, void *dq, void *dc, void *dkr, const LatWs &ws, cudaStream_t st);
cudaError_t launch_lat_bwd_simt(const Prob &p, const void *q, const void *c, const int32_t *anchors,
                                const uint8_t *keep, const float *lse, const void *dout, void *dq, void *dc,
                                void *dkr, const LatWs &ws, cudaStream_t st);

// ---- cache -------------------------------------------------------------------
// rope_base^(-2i/d_r), formed on the host
struct RopeFreq {
    double f[64];
};
RopeFreq rope_freq(int d_r, double base);

inline size_t cache_row_bytes(int kind, int d_l, int d_r) {
    if (kind == DSPARK_CACHE_FP8) return ((size_t)d_l + 2 * (size_t)d_r + 4 * (size_t)(d_l / 128) + 15) / 16 * 16;
    return (size_t)(d_l + d_r) * (kind == DSPARK_CACHE_F32 ? 4 : 2);
}

cudaError_t launch_cache_write(const dspark_latent_cache &p, const void *c, const void *kr, const void *w, double eps,
                               const RopeFreq &freq, const int32_t *pos, const int64_t *slots, void *cache,
                               cudaStream_t st);
cudaError_t launch_cache_read(const dspark_latent_cache &p, const void *cache, const int64_t *slots, void *c_out,
                              void *kr_out, cudaStream_t st);

// ---- attention over the paged cache --------------------------------------------
struct Paged {
    int n_seq, T, n_h, d_l, d_r, page_size, n_pages, max_pages, max_kv, window, causal, dtype, kind;
    long long q_ts, q_hs, o_ts, o_hs;  // strides in elements
    size_t row_bytes;
    float scale, scale_log2;
    uint64_t wait_ns;
    RopeFreq freq;
    const void *q, *cache;
    const int32_t *table, *q_start, *kv_len;
    void *o;
    float *lse;
    uint32_t *err;
};

size_t paged_workspace_size(const Paged &p);
cudaError_t launch_paged(const Paged &p, void *ws, cudaStream_t st);  // plan and attention

#ifdef __CUDACC__
// cos and sin of pos * f: the angle formed in 64 bits and brought into
// [-pi, pi] there (positions of a long cache times a frequency near 1 lose
// their fraction in 32 bits).
__device__ __forceinline__ float2 rope_cs(int pos, double f) {
    const double a = (double)pos * f;
    const double n = rint(a * 0.15915494309189535);
    const float r = (float)fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, a));
    float s, c;
    sincosf(r, &s, &c);
    return make_float2(c, s);
}

// A sequence's place and the keys a row of it sees, checked against the bounds
// that the host cannot see.
struct SeqView {
    int q0, q_len, kv;  // first token, new tokens, keys (0 when out of range)
    bool bad;
};
__device__ __forceinline__ SeqView seq_view(const Paged &p, int s) {
    SeqView v;
    const int a = p.q_start[s], b = p.q_start[s + 1];
    v.kv = p.kv_len[s];
    v.bad = false;
    v.q0 = a;
    v.q_len = b - a;
    if (a < 0 || b < a || b > p.T) {
        v.q0 = 0;
        v.q_len = 0;
        v.bad = true;
    }
    if (v.kv < 0 || (long long)v.kv > (long long)p.max_pages * p.page_size) {
        v.kv = 0;
        v.bad = true;
    }
    return v;
}
// keys [lo, hi) of token i of the sequence
__device__ __forceinline__ void seq_range(const Paged &p, const SeqView &v, int i, int *lo, int *hi) {
    const int ctx = v.kv - v.q_len;  // may be negative: tokens before position 0 see nothing
    const int t = ctx + i;
    *hi = p.causal ? min(t + 1, v.kv) : v.kv;
    const long long first = p.causal ? t : ctx;
    const long long l = p.window > 0 ? first - p.window + 1 : 0;
    *lo = l > 0 ? (int)l : 0;
    if (*hi < *lo) *hi = *lo;
}
#endif

}  // namespace dspark
