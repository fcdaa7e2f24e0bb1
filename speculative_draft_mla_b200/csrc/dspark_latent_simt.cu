// CUDA-core forward and backward of the latent draft attention, and the
// attention over the paged cache: the fp32 path and the path of every shape
// that the tensor-core kernels do not take (other widths, long windows).
//
// One warp owns one query row (forward, dq) or one key (dc, dkr); lane l holds
// dims l, l + 32, ... of the row in registers, a score is a 5-step butterfly
// sum, and a row's keys are taken four at a time so that their loads and
// butterflies overlap. Every output element has one writer and every sum a
// fixed order: no atomics. Bound: the butterfly latency (about 25 shuffles for
// four keys) and the L1 reads of the keys, which the heads of a block share.
#include <algorithm>

#include "dspark_latent_paged.cuh"

namespace dspark {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;  // warps per CTA

// Element d of the query row, rope slice turned to the row's position.
template <typename T>
__device__ __forceinline__ float q_elem(const T *row, int d, int d_l, int d_r, const float2 *cs) {
    if (d < d_l) return to_f(row[d]);
    const int r = d - d_l, i = r >> 1;
    if (r >= d_r) return 0.f;
    const float2 t = cs[i];
    const float x0 = to_f(row[d_l + 2 * i]), x1 = to_f(row[d_l + 2 * i + 1]);
    return (r & 1) ? x0 * t.y + x1 * t.x : x0 * t.x - x1 * t.y;
}

__device__ __forceinline__ bool live_block(const Prob &p, const int32_t *anchors, const uint8_t *keep, int b, int n,
                                           int *a) {
    *a = anchors[(size_t)b * p.N + n];
    return keep[(size_t)b * p.N + n] && *a >= 0 && *a <= p.S - 2;
}

// Keys of the training layout: element d of key position k of batch row b.
template <typename T> struct DenseKeys {
    const T *c;
    const float *krr;  // turned, fp32
    int d_l, d_r;
    __device__ __forceinline__ float at(size_t pos, int d) const {
        return d < d_l ? to_f(c[pos * d_l + d]) : (d < d_l + d_r ? krr[pos * d_r + d - d_l] : 0.f);
    }
};

// ---------------------------------------------------------------------------
// Forward, one warp per row: online softmax over four keys a step.
template <typename T, int NL>
__global__ void __launch_bounds__(kWarps * 32) k_lat_fwd_simt(Prob p, const T *__restrict__ q,
                                                              const T *__restrict__ c, const float *__restrict__ krr,
                                                              const int32_t *__restrict__ anchors,
                                                              const uint8_t *__restrict__ keep,
                                                              const float2 *__restrict__ tab, T *__restrict__ o,
                                                              float *__restrict__ lse) {
    const int lane = threadIdx.x & 31;
    const size_t row = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5);  // (b, h, 5n + j)
    if (row >= (size_t)p.B * p.n_h * p.R) return;
    const int r = (int)(row % p.R), n = r / kBlock, j = r % kBlock;
    const int b = (int)(row / ((size_t)p.R * p.n_h));
    int a;
    if (!live_block(p, anchors, keep, b, n, &a)) {
        for (int d = lane; d < p.d_c; d += 32) o[row * p.d_c + d] = from_f<T>(0.f);
        if (lane == 0) lse[row] = -INFINITY;
        return;
    }
    float qv[NL], acc[NL];
    const float2 *cs = tab + (size_t)(a + j) * (p.d_r / 2);
#pragma unroll
    for (int i = 0; i < NL; i++) {
        qv[i] = lane + 32 * i < p.dqk ? q_elem(q + row * p.dqk, lane + 32 * i, p.d_c, p.d_r, cs) : 0.f;
        acc[i] = 0.f;
    }
    const DenseKeys<T> keys{c, krr, p.d_c, p.d_r};
    const int lo = max(0, a - p.W + 1), nctx = a - lo, nk = nctx + kBlock;
    const size_t kb = (size_t)b * p.L;
    float m = -INFINITY, l = 0.f;
    for (int t = 0; t < nk; t += 4) {
        float s[4], kv[4][NL];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int tt = min(t + u, nk - 1);
            const size_t pos = kb + (tt < nctx ? lo + tt : p.S + kBlock * n + tt - nctx);
            s[u] = 0.f;
#pragma unroll
            for (int i = 0; i < NL; i++) {
                kv[u][i] = keys.at(pos, lane + 32 * i);
                s[u] = fmaf(qv[i], kv[u][i], s[u]);
            }
        }
        warp_sum_all(s);
        float mn = m;
#pragma unroll
        for (int u = 0; u < 4; u++) {
            s[u] = t + u < nk ? s[u] * p.scale_log2 : -INFINITY;
            mn = fmaxf(mn, s[u]);
        }
        const float mu = mn == -INFINITY ? 0.f : mn;  // (scores of -inf or NaN only)
        const float al = exp2f(m - mu);
        l *= al;
#pragma unroll
        for (int i = 0; i < NL; i++) acc[i] *= al;
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const float e = t + u < nk ? exp2f(s[u] - mu) : 0.f;
            l += e;
            if (t + u < nk) {
#pragma unroll
                for (int i = 0; i < NL; i++) acc[i] = fmaf(e, kv[u][i], acc[i]);
            }
        }
        m = mn;
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < NL; i++)
        if (lane + 32 * i < p.d_c) o[row * p.d_c + lane + 32 * i] = from_f<T>(acc[i] * inv);
    if (lane == 0) lse[row] = (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------------------
// dq and D = sum_k P_k dP_k (which is rowsum(dO o O)), one warp per row: a
// pass over the keys for D, a second one for dq = sum_k dS_k k.
template <typename T, int NL>
__global__ void __launch_bounds__(kWarps * 32) k_lat_bwd_q_simt(Prob p, const T *__restrict__ q,
                                                                const T *__restrict__ c, const float *__restrict__ krr,
                                                                const int32_t *__restrict__ anchors,
                                                                const uint8_t *__restrict__ keep,
                                                                const float2 *__restrict__ tab,
                                                                const float *__restrict__ lse,
                                                                const T *__restrict__ dout, T *__restrict__ dq,
                                                                float *__restrict__ dvec) {
    const int lane = threadIdx.x & 31;
    const size_t row = (size_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (size_t)p.B * p.n_h * p.R) return;
    const int r = (int)(row % p.R), n = r / kBlock, j = r % kBlock;
    const int b = (int)(row / ((size_t)p.R * p.n_h));
    int a;
    if (!live_block(p, anchors, keep, b, n, &a)) {
        for (int d = lane; d < p.dqk; d += 32) dq[row * p.dqk + d] = from_f<T>(0.f);
        if (lane == 0) dvec[row] = 0.f;
        return;
    }
    float qv[NL], gv[NL], acc[NL];
    const float2 *cs = tab + (size_t)(a + j) * (p.d_r / 2);
#pragma unroll
    for (int i = 0; i < NL; i++) {
        const int d = lane + 32 * i;
        qv[i] = d < p.dqk ? q_elem(q + row * p.dqk, d, p.d_c, p.d_r, cs) : 0.f;
        gv[i] = d < p.d_c ? to_f(dout[row * p.d_c + d]) : 0.f;
        acc[i] = 0.f;
    }
    const DenseKeys<T> keys{c, krr, p.d_c, p.d_r};
    const int lo = max(0, a - p.W + 1), nctx = a - lo, nk = nctx + kBlock;
    const size_t kb = (size_t)b * p.L;
    const float z = lse[row] * kLog2e;
    float D = 0.f;
    for (int pass = 0; pass < 2; pass++) {
        for (int t = 0; t < nk; t += 2) {
            float s[4], kv[2][NL];  // scores of two keys, then their dP
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int tt = min(t + u, nk - 1);
                const size_t pos = kb + (tt < nctx ? lo + tt : p.S + kBlock * n + tt - nctx);
                s[u] = s[2 + u] = 0.f;
#pragma unroll
                for (int i = 0; i < NL; i++) {
                    kv[u][i] = keys.at(pos, lane + 32 * i);
                    s[u] = fmaf(qv[i], kv[u][i], s[u]);
                    s[2 + u] = fmaf(gv[i], kv[u][i], s[2 + u]);
                }
            }
            warp_sum_all(s);
#pragma unroll
            for (int u = 0; u < 2; u++) {
                if (t + u >= nk) continue;
                const float pr = exp2f(fmaf(s[u], p.scale_log2, -z));
                if (pass == 0) {
                    D = fmaf(pr, s[2 + u], D);
                } else {
                    const float ds = pr * (s[2 + u] - D) * p.scale;
#pragma unroll
                    for (int i = 0; i < NL; i++) acc[i] = fmaf(ds, kv[u][i], acc[i]);
                }
            }
        }
    }
    if (lane == 0) dvec[row] = D;
    // the rope slice turned back: a pair's two elements are on neighbouring lanes
#pragma unroll
    for (int i = 0; i < NL; i++) {
        const int d = lane + 32 * i, rr = d - p.d_c;
        // d_c may be odd: the pair's other element is one lane up or down, or
        // in the next / last group of 32 dims
        const float up = __shfl_down_sync(0xffffffffu, acc[i], 1), dn = __shfl_up_sync(0xffffffffu, acc[i], 1);
        const float nx = i + 1 < NL ? __shfl_sync(0xffffffffu, acc[i + 1 < NL ? i + 1 : i], 0) : 0.f;
        const float pv = i > 0 ? __shfl_sync(0xffffffffu, acc[i > 0 ? i - 1 : 0], 31) : 0.f;
        float val = acc[i];
        if (rr >= 0 && d < p.dqk) {
            const float2 t = cs[rr >> 1];
            if (rr & 1) {
                const float x0 = lane == 0 ? pv : dn;
                val = acc[i] * t.x - x0 * t.y;
            } else {
                const float x1 = lane == 31 ? nx : up;
                val = acc[i] * t.x + x1 * t.y;
            }
        }
        if (d < p.dqk) dq[row * p.dqk + d] = from_f<T>(val);
    }
}

// ---------------------------------------------------------------------------
// dc and dkr: one CTA per key position; its warps take the rows that see the
// key in turn (every head and offset of the blocks whose window covers it, or
// of its own block for a draft key) and are summed in a fixed order.
template <typename T, int NL>
__global__ void __launch_bounds__(kWarps * 32) k_lat_bwd_k_simt(Prob p, const T *__restrict__ q,
                                                                const T *__restrict__ c, const float *__restrict__ krr,
                                                                const int32_t *__restrict__ anchors,
                                                                const uint8_t *__restrict__ keep,
                                                                const float2 *__restrict__ tab,
                                                                const float *__restrict__ lse,
                                                                const T *__restrict__ dout,
                                                                const float *__restrict__ dvec, T *__restrict__ dc,
                                                                T *__restrict__ dkr) {
    extern __shared__ float sm[];  // [kWarps][dqk]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int key = blockIdx.x, b = blockIdx.y;
    const size_t kpos = (size_t)b * p.L + key;
    float kv[NL], acc[NL];
    const DenseKeys<T> keys{c, krr, p.d_c, p.d_r};
#pragma unroll
    for (int i = 0; i < NL; i++) {
        kv[i] = keys.at(kpos, lane + 32 * i);
        acc[i] = 0.f;
    }
    int own = key >= p.S ? (key - p.S) / kBlock : -1, pos_of_key = key;
    const int n0 = own >= 0 ? own : 0, n1 = own >= 0 ? own + 1 : p.N;
    for (int n = n0; n < n1; n++) {
        int a;
        if (!live_block(p, anchors, keep, b, n, &a)) continue;
        if (own >= 0)
            pos_of_key = a + (key - p.S) % kBlock;
        else if (key >= a || key < a - p.W + 1)
            continue;
        for (int hj = warp; hj < p.n_h * kBlock; hj += kWarps) {
            const int j = hj % kBlock;
            const size_t row = ((size_t)b * p.n_h + hj / kBlock) * p.R + kBlock * n + j;
            const float2 *cs = tab + (size_t)(a + j) * (p.d_r / 2);
            float qv[NL], gv[NL], s[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NL; i++) {
                const int d = lane + 32 * i;
                qv[i] = d < p.dqk ? q_elem(q + row * p.dqk, d, p.d_c, p.d_r, cs) : 0.f;
                gv[i] = d < p.d_c ? to_f(dout[row * p.d_c + d]) : 0.f;
                s[0] = fmaf(qv[i], kv[i], s[0]);
                s[1] = fmaf(gv[i], kv[i], s[1]);
            }
            warp_sum_all(s);
            const float pr = exp2f(fmaf(s[0], p.scale_log2, -lse[row] * kLog2e));
            const float ds = pr * (s[1] - dvec[row]) * p.scale;
#pragma unroll
            for (int i = 0; i < NL; i++) acc[i] = fmaf(pr, gv[i], fmaf(ds, qv[i], acc[i]));
        }
    }
#pragma unroll
    for (int i = 0; i < NL; i++)
        if (lane + 32 * i < p.dqk) sm[warp * p.dqk + lane + 32 * i] = acc[i];
    __syncthreads();
    for (int d = threadIdx.x; d < p.dqk; d += blockDim.x) {
        float x = 0.f;
        for (int w = 0; w < kWarps; w++) x += sm[w * p.dqk + d];
        if (d < p.d_c) {
            dc[kpos * p.d_c + d] = from_f<T>(x);
        } else {
            const int rr = d - p.d_c, other = p.d_c + (rr ^ 1);
            float y = 0.f;
            for (int w = 0; w < kWarps; w++) y += sm[w * p.dqk + other];
            const float2 t = tab[(size_t)min(max(pos_of_key, 0), p.P - 1) * (p.d_r / 2) + (rr >> 1)];
            dkr[kpos * p.d_r + rr] = from_f<T>((rr & 1) ? x * t.x - y * t.y : x * t.x + y * t.y);
        }
    }
}

// ---------------------------------------------------------------------------
// Attention over the paged cache, one warp per (token, head).
template <typename T, int KIND, int NL>
__global__ void __launch_bounds__(kWarps * 32) k_paged_simt(const Paged p) {
    const int lane = threadIdx.x & 31;
    const long long id = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (id >= (long long)p.T * p.n_h) return;
    const int tok = (int)(id / p.n_h), h = (int)(id % p.n_h);
    // the sequence of the token: the warp scans the starts 32 at a time, and keeps the
    // last end before it (a sequence that begins before that attends nothing)
    int s = -1, before = 0;
    for (int s0 = 0; s0 < p.n_seq && s < 0; s0 += 32) {
        bool mine = false;
        int end = 0;
        if (s0 + lane < p.n_seq) {
            const SeqView v = seq_view(p, s0 + lane);
            mine = tok >= v.q0 && tok < v.q0 + v.q_len;
            if (v.q_len > 0) end = v.q0 + v.q_len;
        }
        const unsigned any = __ballot_sync(0xffffffffu, mine);
        if (any) s = s0 + __ffs(any) - 1;
        if (s < 0 || s0 + lane < s) before = max(before, end);
    }
    if (s < 0) return;  // behind the last sequence
    const SeqView sv = seq_view(p, s);
    if (__any_sync(0xffffffffu, sv.q0 < before)) return;
    int lo, hi;
    seq_range(p, sv, tok - sv.q0, &lo, &hi);
    const T *qrow = (const T *)p.q + (long long)tok * p.q_ts + (long long)h * p.q_hs;
    float acc[NL], m, l;
    const bool gone = paged_row<T, KIND, NL, 4>(p, s, qrow, sv.kv - sv.q_len + tok - sv.q0, lo, hi, acc, m, l);
    if (gone && lane == 0) atomicOr(p.err, kErrPage);
    const bool some = l != 0.f;  // (NaN counts)
    T *orow = (T *)p.o + (long long)tok * p.o_ts + (long long)h * p.o_hs;
#pragma unroll
    for (int i = 0; i < NL; i++)
        if (lane + 32 * i < p.d_l) orow[lane + 32 * i] = from_f<T>(some ? acc[i] / l : 0.f);
    if (lane == 0) p.lse[(size_t)tok * p.n_h + h] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <typename T, int NL>
cudaError_t fwd_t(const Prob &p, const void *q, const void *c, const int32_t *anchors, const uint8_t *keep, void *o,
                  float *lse, const LatWs &ws, cudaStream_t st) {
    const size_t rows = (size_t)p.B * p.n_h * p.R;
    if (rows == 0) return cudaSuccess;
    count_launch();
    k_lat_fwd_simt<T, NL><<<(unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(
        p, (const T *)q, (const T *)c, ws.kr_f32, anchors, keep, ws.base.rope, (T *)o, lse);
    return cudaGetLastError();
}

template <typename T, int NL>
cudaError_t bwd_t(const Prob &p, const void *q, const void *c, const int32_t *anchors, const uint8_t *keep,
                  const float *lse, const void *dout, void *dq, void *dc, void *dkr, const LatWs &ws,
                  cudaStream_t st) {
    const size_t rows = (size_t)p.B * p.n_h * p.R;
    if (rows) {
        count_launch();
        k_lat_bwd_q_simt<T, NL><<<(unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(
            p, (const T *)q, (const T *)c, ws.kr_f32, anchors, keep, ws.base.rope, lse,
            (const T *)dout, (T *)dq, ws.dvec);
    }
    if (p.B) {
        count_launch();
        k_lat_bwd_k_simt<T, NL><<<dim3(p.L, p.B), kWarps * 32, sizeof(float) * kWarps * p.dqk, st>>>(
            p, (const T *)q, (const T *)c, ws.kr_f32, anchors, keep, ws.base.rope, lse,
            (const T *)dout, ws.dvec, (T *)dc, (T *)dkr);
    }
    return cudaGetLastError();
}

template <typename T, int KIND> cudaError_t paged_t(const Paged &p, cudaStream_t st) {
    const unsigned grid = (unsigned)(((long long)p.T * p.n_h + kWarps - 1) / kWarps);
    count_launch();
    if (p.d_l + p.d_r <= 128)
        k_paged_simt<T, KIND, 4><<<grid, kWarps * 32, 0, st>>>(p);
    else
        k_paged_simt<T, KIND, 20><<<grid, kWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_lat_fwd_simt(const Prob &p, const void *q, const void *c, const int32_t *anchors,
                                const uint8_t *keep, void *o, float *lse, const LatWs &ws, cudaStream_t st) {
    if (p.dtype == DSPARK_F32)
        return p.dqk <= 128 ? fwd_t<float, 4>(p, q, c, anchors, keep, o, lse, ws, st)
                            : fwd_t<float, 20>(p, q, c, anchors, keep, o, lse, ws, st);
    return p.dqk <= 128 ? fwd_t<__nv_bfloat16, 4>(p, q, c, anchors, keep, o, lse, ws, st)
                        : fwd_t<__nv_bfloat16, 20>(p, q, c, anchors, keep, o, lse, ws, st);
}

cudaError_t launch_lat_bwd_simt(const Prob &p, const void *q, const void *c, const int32_t *anchors,
                                const uint8_t *keep, const float *lse, const void *dout, void *dq, void *dc,
                                void *dkr, const LatWs &ws, cudaStream_t st) {
    if (p.dtype == DSPARK_F32)
        return p.dqk <= 128 ? bwd_t<float, 4>(p, q, c, anchors, keep, lse, dout, dq, dc, dkr, ws, st)
                            : bwd_t<float, 20>(p, q, c, anchors, keep, lse, dout, dq, dc, dkr, ws, st);
    return p.dqk <= 128 ? bwd_t<__nv_bfloat16, 4>(p, q, c, anchors, keep, lse, dout, dq, dc, dkr, ws, st)
                        : bwd_t<__nv_bfloat16, 20>(p, q, c, anchors, keep, lse, dout, dq, dc, dkr, ws, st);
}

cudaError_t launch_paged_simt(const Paged &p, cudaStream_t st) {
    switch (p.kind) {
        case DSPARK_CACHE_F32: return paged_t<float, DSPARK_CACHE_F32>(p, st);
        case DSPARK_CACHE_BF16: return paged_t<__nv_bfloat16, DSPARK_CACHE_BF16>(p, st);
        default: return paged_t<__nv_bfloat16, DSPARK_CACHE_FP8>(p, st);
    }
}

}  // namespace dspark
