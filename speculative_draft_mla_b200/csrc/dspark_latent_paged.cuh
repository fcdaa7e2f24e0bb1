// The attention over the paged cache: plan, launch functions, and the
// CUDA-core evaluation of one row.
#pragma once

#include "dspark_latent.cuh"

namespace dspark {

constexpr int kPairs = 74;      // CTA pairs of the tensor-core kernel (two CTAs share a tile's value columns)
constexpr int kStepKeys = 64;   // keys of a step
constexpr int kShortKeys = 144; // keys that a sequence of the short kernel sees at most

struct PagedHead {
    long long total, per;  // steps of all tiles; steps of a pair
    int n_split;           // tiles that several pairs work on
    int n_short;           // sequences of the short kernel
    int n_tiles;
    int redo;              // whether a tile has rows to evaluate again
};
struct alignas(16) PagedTile {      // up to 128 (token, head) rows of a sequence
    int seq, i0, hc, q_len;  // first token within the sequence, chunk of 128 heads
    int q0, kv, lo, hi;      // the sequence's first token; keys; keys that some row sees
    long long start, steps;  // its steps in the list of all
    uint32_t redo[4];        // rows to evaluate again
};
struct PagedPlan {
    PagedHead *head;
    int *first;            // [kPairs] tile in which pair i begins
    int *split;            // [kPairs] tiles that several pairs work on
    PagedTile *tiles;
    int *short_seq;        // [n_seq] sequences of the short kernel
    float2 *tab;           // [T, 32] (cos, sin) of the tokens' positions
    float *part_lse, *part_o;  // [2 kPairs, 128], [2 kPairs, 128, 512]: results of parts of a tile
    int tpt, hchunks, max_tiles;  // tokens of a tile, its chunks of heads
};

bool paged_tc_supported(const Paged &p);
size_t paged_layout(const Paged &p, void *ws, PagedPlan *w);
cudaError_t launch_paged_simt(const Paged &p, cudaStream_t st);
// sequences whose tokens together see few keys (drafts, short windows)
cudaError_t launch_short_tc(const Paged &p, const PagedPlan &w, cudaStream_t st);
cudaError_t launch_paged_tc(const Paged &p, const PagedPlan &w, cudaStream_t st);

#ifdef __CUDACC__

// Keys [*lo, *hi) that some of the tokens [i0, i1) of a sequence see.
__device__ __forceinline__ void tile_range(const Paged &p, const SeqView &v, int i0, int i1, int *lo, int *hi) {
    int l1, h0;
    seq_range(p, v, i0, lo, &h0);
    seq_range(p, v, i1 - 1, &l1, hi);
    if (*hi < *lo) *hi = *lo;
}
__device__ __forceinline__ int tile_steps(const Paged &p, const SeqView &v, int i0, int i1) {
    int lo, hi;
    tile_range(p, v, i0, i1, &lo, &hi);
    // (the first step begins at a multiple of 8)
    return max(1, (int)(((long long)hi - (lo & ~7) + kStepKeys - 1) / kStepKeys));
}

// Slot of key of sequence s, or -1 where its page is out of range.
__device__ __forceinline__ long long key_slot(const Paged &p, int s, int key) {
    const int page = p.table[(size_t)s * p.max_pages + key / p.page_size];
    return page >= 0 && page < p.n_pages ? (long long)page * p.page_size + key % p.page_size : -1;
}

template <int N> __device__ __forceinline__ void warp_sum_all(float (&x)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; i++) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
}

template <int KIND> struct CacheRow;
template <> struct CacheRow<DSPARK_CACHE_F32> {
    static __device__ __forceinline__ float at(const uint8_t *row, int d, int d_l, int d_r) {
        return reinterpret_cast<const float *>(row)[d];
    }
};
template <> struct CacheRow<DSPARK_CACHE_BF16> {
    static __device__ __forceinline__ float at(const uint8_t *row, int d, int d_l, int d_r) {
        return to_f(reinterpret_cast<const __nv_bfloat16 *>(row)[d]);
    }
};
template <> struct CacheRow<DSPARK_CACHE_FP8> {
    static __device__ __forceinline__ float at(const uint8_t *row, int d, int d_l, int d_r) {
        if (d >= d_l) return to_f(reinterpret_cast<const __nv_bfloat16 *>(row + d_l)[d - d_l]);
        const float s = reinterpret_cast<const float *>(row + d_l + 2 * d_r)[d >> 7];
        __nv_fp8_e4m3 v;
        v.__x = row[d];
        return (float)v * s;
    }
};

// One row (token at position pos_q) over the keys [lo, hi) of sequence s, by a
// warp: lane l holds dims l, l + 32, .... U keys at a time, online softmax.
// acc = sum_k 2^(s_k - m) c_k, l the sum of the weights, m in log2 units;
// l = 0: no key. Returns whether a page was out of range.
template <typename T, int KIND, int NL, int U>
__device__ __forceinline__ bool paged_row(const Paged &p, int s, const T *qrow, int pos_q, int lo, int hi,
                                          float (&acc)[NL], float &m, float &l) {
    const int lane = threadIdx.x & 31, dk = p.d_l + p.d_r;
    float qv[NL];
#pragma unroll
    for (int i = 0; i < NL; i++) {
        const int d = lane + 32 * i;
        float val = 0.f;
        if (d < p.d_l) {
            val = to_f(qrow[d]);
        } else if (d < dk) {
            const int r = d - p.d_l;
            const float2 t = rope_cs(pos_q, p.freq.f[r >> 1]);
            const float x0 = to_f(qrow[p.d_l + (r & ~1)]), x1 = to_f(qrow[p.d_l + (r | 1)]);
            val = (r & 1) ? x0 * t.y + x1 * t.x : x0 * t.x - x1 * t.y;
        }
        qv[i] = val;
        acc[i] = 0.f;
    }
    m = -INFINITY;
    l = 0.f;
    bool gone = false;
    for (int k0 = lo; k0 < hi; k0 += U) {
        float sc[U], kv[U][NL];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int key = k0 + u;
            const long long slot = key < hi ? key_slot(p, s, key) : -1;
            ok[u] = slot >= 0;
            gone |= key < hi && !ok[u];
            sc[u] = 0.f;
            const uint8_t *krow = (const uint8_t *)p.cache + (size_t)(ok[u] ? slot : 0) * p.row_bytes;
#pragma unroll
            for (int i = 0; i < NL; i++) {
                const int d = lane + 32 * i;
                kv[u][i] = ok[u] && d < dk ? CacheRow<KIND>::at(krow, d, p.d_l, p.d_r) : 0.f;
                sc[u] = fmaf(qv[i], kv[u][i], sc[u]);
            }
        }
        warp_sum_all(sc);
        float mn = m;
#pragma unroll
        for (int u = 0; u < U; u++) {
            sc[u] = ok[u] ? sc[u] * p.scale_log2 : -INFINITY;
            mn = fmaxf(mn, sc[u]);
        }
        const float mu = mn == -INFINITY ? 0.f : mn;  // (scores of -inf or NaN only)
        const float al = exp2f(m - mu);
        l *= al;
#pragma unroll
        for (int i = 0; i < NL; i++) acc[i] *= al;
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (!ok[u]) continue;
            const float e = exp2f(sc[u] - mu);
            l += e;
#pragma unroll
            for (int i = 0; i < NL; i++) acc[i] = fmaf(e, kv[u][i], acc[i]);
        }
        m = mn;
    }
    return gone;
}

#endif

}  // namespace dspark
