// Attention of new tokens over the paged latent cache: the plan of a call and
// the choice of kernels.
#include <algorithm>

#include "dspark_latent_paged.cuh"

namespace dspark {

namespace {

// One launch ahead of the attention. CTA 0 writes the error word (the page bit
// for a q_start or kv_len out of range, else 0; pages are checked by the
// kernels that read them) and, for the tensor-core kernels, the list of short
// sequences and the list of row tiles: tile r is up to 128 (token, head) rows of
// one sequence and takes its steps of 64 keys, at least one. The CTA pairs of the
// attention share all steps evenly, wherever tiles begin and end; first[i] is
// the tile that pair i begins in. The other CTAs fill the tokens' (cos, sin).
//
// A sequence that begins before the end of an earlier one (of any whose own two
// entries are in order, refused or not) attends nothing. So those that attend
// share no token: no row has two writers, the first sequence that holds a token
// is its only one (what the search below and the CUDA-core kernel rely on), and
// their tiles, fewer than 2^26 as T * n_h < 2^31, fit the list.
__global__ void __launch_bounds__(1024) k_paged_plan(const Paged p, const PagedPlan w, int tc, int shorts, int tab_ctas) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x > 0) {
        // one warp per token: its sequence by a search over the starts, 32 at a time
        const int lane = threadIdx.x & 31;
        for (int tok = (blockIdx.x - 1) * 32 + (threadIdx.x >> 5); tok < p.T; tok += tab_ctas * 32) {
            int s = -1;
            for (int s0 = 0; s0 < p.n_seq && s < 0; s0 += 32) {
                bool mine = false;
                if (s0 + lane < p.n_seq) {
                    const SeqView v = seq_view(p, s0 + lane);
                    mine = tok >= v.q0 && tok < v.q0 + v.q_len;
                }
                const unsigned any = __ballot_sync(0xffffffffu, mine);
                if (any) s = s0 + __ffs(any) - 1;
            }
            if (s < 0) continue;
            const SeqView v = seq_view(p, s);
            w.tab[(size_t)tok * 32 + lane] = rope_cs(v.kv - v.q_len + tok - v.q0, p.freq.f[lane]);
        }
        return;
    }
    __shared__ long long wsteps[32], carry_steps;
    __shared__ int wtiles[32], wends[32], carry_tiles, carry_end, bad, n_split, n_short;
    if (threadIdx.x == 0) {
        bad = 0;
        n_split = 0;
        n_short = 0;
        carry_steps = 0;
        carry_tiles = 0;
        carry_end = 0;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int disorder = 0;
    for (int s0 = 0; s0 < p.n_seq; s0 += blockDim.x) {
        const int s = s0 + threadIdx.x;
        SeqView v{};
        int nt = 0;
        long long ns = 0;
        if (s < p.n_seq) v = seq_view(p, s);
        // (in order so far: none begins before an earlier one's end)
        disorder |= __syncthreads_or(v.bad);
        if (disorder) {
            const int end = v.q_len > 0 ? v.q0 + v.q_len : 0;
            int upto = end;  // the last end of the sequences up to this one
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto = max(upto, a);
            }
            if (lane == 31) wends[warp] = upto;
            const int last = __shfl_up_sync(0xffffffffu, upto, 1);
            __syncthreads();
            int before = max(carry_end, lane > 0 ? last : 0);
            for (int k = 0; k < warp; k++) before = max(before, wends[k]);
            __syncthreads();
            if (threadIdx.x == blockDim.x - 1) carry_end = max(before, end);
            if (v.q_len > 0 && v.q0 < before) {
                v.q_len = 0;
                v.bad = true;
            }
        } else if (threadIdx.x == 0 && s0 + (int)blockDim.x < p.n_seq) {
            const int next = p.q_start[s0 + blockDim.x];
            carry_end = next > p.q_start[0] ? next : 0;
        }
        if (s < p.n_seq) {
            if (v.bad) bad = 1;
            bool brief = false;
            if (shorts && v.q_len > 0) {
                int lo, hi;
                tile_range(p, v, 0, v.q_len, &lo, &hi);
                brief = hi - lo <= kShortKeys;
            }
            if (brief) {
                w.short_seq[atomicAdd(&n_short, 1)] = s;
            } else if (tc) {
                nt = (v.q_len + w.tpt - 1) / w.tpt;
                for (int t = 0; t < nt; t++) ns += tile_steps(p, v, t * w.tpt, min(v.q_len, (t + 1) * w.tpt));
                nt *= w.hchunks;
                ns *= w.hchunks;
            }
        }
        // inclusive sums over the block
        int it = nt;
        long long is = ns;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, it, o);
            const long long b = __shfl_up_sync(0xffffffffu, is, o);
            if (lane >= o) {
                it += a;
                is += b;
            }
        }
        if (lane == 31) {
            wtiles[warp] = it;
            wsteps[warp] = is;
        }
        __syncthreads();
        int bt = carry_tiles + it - nt;
        long long bs = carry_steps + is - ns;
        for (int k = 0; k < warp; k++) {
            bt += wtiles[k];
            bs += wsteps[k];
        }
        __syncthreads();
        if (threadIdx.x == blockDim.x - 1) {
            carry_tiles = bt + nt;
            carry_steps = bs + ns;
        }
        for (int t = 0; t < nt; t++) {
            const int hc = t % w.hchunks, i0 = t / w.hchunks * w.tpt;
            PagedTile o{};
            o.seq = s;
            o.i0 = i0;
            o.hc = hc;
            o.q_len = v.q_len;
            o.q0 = v.q0;
            o.kv = v.kv;
            tile_range(p, v, i0, min(v.q_len, i0 + w.tpt), &o.lo, &o.hi);
            o.start = bs;
            o.steps = tile_steps(p, v, i0, min(v.q_len, i0 + w.tpt));
            w.tiles[bt + t] = o;
            bs += o.steps;
        }
        __syncthreads();
    }
    __syncthreads();
    if (tc) {
        const int n = carry_tiles;
        const long long total = carry_steps;
        const long long X = (total + kPairs - 1) / kPairs;
        if (threadIdx.x == 0) {
            w.head->total = total;
            w.head->per = X;
            w.head->n_short = n_short;
            w.head->n_tiles = n;
            w.head->redo = 0;
        }
        __syncthreads();
        if (total)
            for (int r = threadIdx.x; r < n; r += blockDim.x) {
                const long long a = w.tiles[r].start, b = a + w.tiles[r].steps;
                for (long long i = (a + X - 1) / X; i < kPairs && i * X < b; i++) w.first[i] = r;
                if (a / X != (b - 1) / X) w.split[atomicAdd(&n_split, 1)] = r;  // (at most one for each end of a pair)
            }
        __syncthreads();
        if (threadIdx.x == 0) w.head->n_split = n_split;
    }
    if (threadIdx.x == 0) *p.err = bad ? kErrPage : 0u;
}

}  // namespace

bool paged_tc_supported(const Paged &p) {
    return p.d_l == 512 && p.d_r == 64 && (p.kind == DSPARK_CACHE_BF16 || p.kind == DSPARK_CACHE_FP8);
}

size_t paged_layout(const Paged &p, void *ws, PagedPlan *w) {
    PagedPlan r{};
    char *c = (char *)ws;
    size_t off = 256;
    const bool tc = paged_tc_supported(p);
    r.head = (PagedHead *)(c + 128);
    r.tpt = p.n_h <= 128 ? 128 / p.n_h : 1;
    r.hchunks = (p.n_h + 127) / 128;
    r.max_tiles = tc ? (int)std::min<long long>(((long long)p.T / r.tpt + p.n_seq) * r.hchunks, 1ll << 30) : 0;
    auto take = [&](size_t n) {
        char *at = c + off;
        off = align256(off + (tc ? n : 0));
        return (void *)at;
    };
    r.first = (int *)take(sizeof(int) * kPairs);
    r.split = (int *)take(sizeof(int) * kPairs);
    r.tiles = (PagedTile *)take(sizeof(PagedTile) * (size_t)r.max_tiles);
    r.short_seq = (int *)take(sizeof(int) * (size_t)p.n_seq);
    r.tab = (float2 *)take(sizeof(float2) * 32 * (size_t)p.T);
    r.part_lse = (float *)take(sizeof(float) * 2 * kPairs * 128);
    r.part_o = (float *)take(sizeof(float) * 2 * kPairs * 128 * 512);
    if (w) *w = r;
    return off;
}

size_t paged_workspace_size(const Paged &p) { return paged_layout(p, nullptr, nullptr); }

cudaError_t launch_paged(const Paged &pp, void *ws, cudaStream_t st) {
    Paged p = pp;
    p.err = (uint32_t *)ws;
    PagedPlan w;
    paged_layout(p, ws, &w);
    const bool run = p.T > 0 && p.n_seq > 0, tc = run && paged_tc_supported(p) && p.n_pages > 0;
    const int tab_ctas = tc ? std::min((p.T + 31) / 32, 296) : 0;
    // Sequences whose tokens see up to 144 keys together go to the short kernel
    // (calls with drafts of 5 tokens, 128 sequences, 8-bit rows: a window of 140, the
    // last that it takes, 49 us, of 141, 156; bf16 rows 48 and 117. 128 tokens over up
    // to 144 keys each, no window: 21 us, and 47 without it; one token: 17 and 18.5).
    // It is launched where the window or the bound of kv_len makes such sequences
    // likely, and alone where no sequence can see more.
    const auto at_most = [](long long n) { return n <= kShortKeys; };
    const bool shorts = tc && ((p.window > 0 && at_most(p.window)) || at_most(p.max_kv)) &&
                        (long long)p.n_seq * w.hchunks < (1 << 23);
    const bool all_short = shorts && ((p.window > 0 && at_most((long long)p.window - 1 + p.T)) ||
                                      at_most((long long)p.max_pages * p.page_size));
    count_launch();
    cudaError_t e = launch_pdl(k_paged_plan, dim3(1 + tab_ctas), dim3(1024), 0, st, p, w, tc ? 1 : 0, shorts ? 1 : 0,
                               tab_ctas);
    if (e != cudaSuccess || !run) return e;
    if (!tc) return launch_paged_simt(p, st);
    if (shorts && (e = launch_short_tc(p, w, st)) != cudaSuccess) return e;
    return all_short ? cudaSuccess : launch_paged_tc(p, w, st);
}

}  // namespace dspark
