// Tensor-core attention of new tokens over the paged latent cache where a
// sequence's tokens together see at most 144 keys: drafts and short windows
// (512-wide latents, 64-wide rope keys; bf16 and 8-bit rows).
//
// As in the draft attention's forward, S = Q K^T of 128 rows over all keys is one
// accumulator of 144 columns: one softmax without a running maximum, the keys
// loaded once for all of a sequence's rows, O in eight 64-column products through
// two accumulators. (The kernel for long contexts takes three steps of 64 keys for
// 132, forms S twice and reloads Q for each half of the values: 5 token drafts of
// 128 sequences over a window of 128 took it 170 us.)
//
// Item: a sequence, a chunk of 128 heads, a run of its tiles of 128 (token, head)
// rows. Keys are gathered row by row (slots of no key are zero); 8-bit rows become
// bf16 on the way. Q comes in 64-column slices through a ring of three. The turned
// rope slice of the queries is hi + lo of two bf16; P is rounded once to bf16 as an
// operand (2^-8 of each weight, as of the rounded O). A row whose product met a key
// that is not finite and not its own (0 x NaN) is evaluated again by its warp, over
// the keys in shared memory.
//
// 128 sequences of 5 tokens, 64 heads, window 128, 8-bit rows: 43 us of the call's 50, one
// item to an SM, so that the latency of the keys and of the first tile is in the open, and that
// of code not yet in the instruction cache: loops over keys that were unrolled more
// made it 60.
// What bounds it beyond: Q in (1152 B a row) and O out (1024 B); per tile 40 products of
// 144 keys (80 cycles; 32 of the latents, 8 of the rope slice's hi and lo) and 72 of 64
// columns (50).
//
// TMEM: S 0..143 / 144..287 (P over its own S columns), rope query hi, lo
// 288..351, O 352..415 / 416..479.
// Warps: 0-3 and 4-7 softmax and output of even and odd tiles (thread = row);
// 8-11 keys (of a CTA's first item 0-11), and the queries' rope slices; 12 loads Q slices, 13 and 14 issue the
// products of S and of O. Every wait is bounded.
#include <algorithm>

#include "dspark_latent_paged.cuh"
#include "dspark_latent_tc.cuh"

namespace dspark {

namespace {

using namespace tc;

constexpr int kDL = 512, kDR = 64, kSlices = 8, kKeys = kShortKeys;
constexpr int kKSlice = kKeys * 128, kQSlot = 128 * 128, kQSlots = 3;
constexpr int oQ = 9 * kKSlice, oBar = oQ + kQSlots * kQSlot;
constexpr int kSmem = oBar + 512 + 1024;
static_assert(kSmem <= 232448 && kKSlice % 1024 == 0, "shared memory");
constexpr uint32_t kColS = 0, kColR = 2 * kKeys, kColO = kColR + 64;
constexpr int kLoaders = 12, kWarpA = 8, kWarpQ = 12, kWarpM = 13, kThreads = 15 * 32;
constexpr float kLn2 = 0.6931471805599453f;

// An item's sequence and tiles.
struct Item {
    int seq, q0, q_len, kv, lo, hi, hc, t0, t1, ncol;
};
__device__ __forceinline__ bool item_at(const Paged &p, const PagedPlan &w, int parts, int i, Item &o) {
    const int s = i / (parts * w.hchunks);
    if (s >= w.head->n_short) return false;
    const int part = i % parts;
    o.hc = i / parts % w.hchunks;
    o.seq = w.short_seq[s];
    const SeqView v = seq_view(p, o.seq);
    o.q0 = v.q0;
    o.q_len = v.q_len;
    o.kv = v.kv;
    tile_range(p, v, 0, v.q_len, &o.lo, &o.hi);
    const int tiles = (v.q_len + w.tpt - 1) / w.tpt, per = (tiles + parts - 1) / parts;
    o.t0 = min(tiles, part * per);
    o.t1 = min(tiles, o.t0 + per);
    o.ncol = max(16, (o.hi - o.lo + 15) & ~15);
    return true;
}
// Row r of tile t of an item.
struct RowOf {
    int i, h;  // token within the sequence, head
    bool live;
    __device__ __forceinline__ RowOf(const Paged &p, const PagedPlan &w, const Item &o, int t, int r) {
        const int ti = w.tpt > 1 || p.n_h == 128 ? r / p.n_h : 0;
        i = t * w.tpt + ti;
        h = o.hc * 128 + r - ti * p.n_h;
        live = ti < w.tpt && i < o.q_len && h < p.n_h && (ti == 0 || w.hchunks == 1);
    }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ uint32_t fp8x2_bf16(uint32_t w, float s) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16x2(f.x * s, f.y * s);
}

// A row once more, by a warp, over the keys in shared memory that it sees (slots
// [lo, hi)): its product met a key that is not finite and not its own. Lane l takes
// the scores of keys l, l + 32, .., then 16 columns of O. 32 rows over 128 keys,
// 0.75 ms; from the cache, a key at a time, 4.2 (8-bit rows: 16).
__device__ __noinline__ void redo_row(const Paged &p, const PagedPlan &w, const Item &it, const uint8_t *sm,
                                      const volatile uint32_t *kmask, int i, int h, int lo, int hi) {
    constexpr int kPer = (kKeys + 31) / 32;
    const int lane = threadIdx.x & 31, tok = it.q0 + i;
    const uint4 *q =
        reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)p.q + (long long)tok * p.q_ts + (long long)h * p.q_hs);
    const float4 *tab = reinterpret_cast<const float4 *>(w.tab + (size_t)tok * 32);
    const auto pair = [](uint32_t x) { return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)); };
    float s[kPer];
#pragma unroll
    for (int j = 0; j < kPer; j++) s[j] = 0.f;
#pragma unroll 1
    for (int u = 0; u < (kDL + kDR) / 8; u++) {
        const uint4 x = __ldg(q + u);
        float2 v[4] = {pair(x.x), pair(x.y), pair(x.z), pair(x.w)};
        if (u >= kDL / 8) {
            const float4 c0 = __ldg(tab + 2 * (u - kDL / 8)), c1 = __ldg(tab + 2 * (u - kDL / 8) + 1);
            const float2 cs[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
#pragma unroll
            for (int e = 0; e < 4; e++)
                v[e] = make_float2(v[e].x * cs[e].x - v[e].y * cs[e].y, v[e].x * cs[e].y + v[e].y * cs[e].x);
        }
#pragma unroll
        for (int j = 0; j < kPer; j++) {
            const int slot = min(lane + 32 * j, kKeys - 1);
            const uint4 k = *reinterpret_cast<const uint4 *>(sm + (u >> 3) * kKSlice + sw128(slot, u & 7));
            const float2 c[4] = {pair(k.x), pair(k.y), pair(k.z), pair(k.w)};
#pragma unroll
            for (int e = 0; e < 4; e++) s[j] = fmaf(v[e].x, c[e].x, fmaf(v[e].y, c[e].y, s[j]));
        }
    }
    uint32_t in[kPer];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        in[j] = slot_mask(lo - 32 * j, hi - 32 * j) & kmask[j];
        s[j] *= p.scale_log2;
        if ((in[j] >> lane) & 1) m = fmaxf(m, s[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mu = m == -INFINITY ? 0.f : m;  // (scores of -inf only)
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        s[j] = (in[j] >> lane) & 1 ? ex2(s[j] - mu) : 0.f;
        l += s[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l != 0.f ? 1.f / l : 0.f;
    if (lane == 0) p.lse[(size_t)tok * p.n_h + h] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    // columns 8 lane .., 256 + 8 lane ..
    float2 acc[2][4];
#pragma unroll
    for (int y = 0; y < 2; y++)
#pragma unroll
        for (int e = 0; e < 4; e++) acc[y][e] = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kPer; j++)
#pragma unroll 1
        for (uint32_t x = in[j]; x; x &= x - 1) {
            const int k = __ffs(x) - 1;
            const float f = __shfl_sync(0xffffffffu, s[j], k);
#pragma unroll
            for (int y = 0; y < 2; y++) {
                const uint4 c = *reinterpret_cast<const uint4 *>(sm + (4 * y + (lane >> 3)) * kKSlice +
                                                                 sw128(32 * j + k, lane & 7));
                const float2 v[4] = {pair(c.x), pair(c.y), pair(c.z), pair(c.w)};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    acc[y][e].x = fmaf(f, v[e].x, acc[y][e].x);
                    acc[y][e].y = fmaf(f, v[e].y, acc[y][e].y);
                }
            }
        }
    __nv_bfloat16 *out = (__nv_bfloat16 *)p.o + (long long)tok * p.o_ts + (long long)h * p.o_hs;
#pragma unroll
    for (int y = 0; y < 2; y++) {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; e++) x[e] = l != 0.f ? pack_bf16x2(acc[y][e].x * inv, acc[y][e].y * inv) : 0u;
        reinterpret_cast<uint4 *>(out)[lane + 32 * y] = make_uint4(x[0], x[1], x[2], x[3]);
    }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    k_short_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ Paged p,
               const __grid_constant__ PagedPlan w, const int parts) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *kfull = reinterpret_cast<uint64_t *>(sm + oBar), *kempty = kfull + 1;
    uint64_t *qfull = kfull + 2, *qempty = qfull + kQSlots;
    uint64_t *sfull = qempty + kQSlots, *pready = sfull + 2, *pvdone = sfull + 4, *ofull = sfull + 6, *ofree = ofull + 4;
    uint64_t *rready = ofree + 2, *rfree = rready + 1, *drain = rready + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(drain + 3);
    volatile uint32_t *kmask = reinterpret_cast<volatile uint32_t *>(drain + 4);  // 32 slots' validity each
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = gridDim.x;
    const uint64_t wlim = p.wait_ns;

    if (threadIdx.x == 0) {
        mbar_init(kfull, kLoaders);
        mbar_init(kempty, 1 + kWarpA);  // the last product of O, the softmax warps
        for (int i = 0; i < 2 * kQSlots; i++) mbar_init(&qfull[i], 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pready[i], 4);
            mbar_init(&pvdone[i], 1);
            mbar_init(&ofull[i], 1);  // of even tiles; 2, 3 of odd ones
            mbar_init(&ofull[2 + i], 1);
            mbar_init(&ofree[i], 4);
            mbar_init(&drain[i], 1);
        }
        mbar_init(rready, 4);
        mbar_init(rfree, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kWarpM) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    uint32_t issued_q = 0;
    Item it;

    // An item's keys, by some of warps: groups first, first + warps, ... of 8 slots, two at a time.
    const uint8_t *cache = (const uint8_t *)p.cache;
    const auto load_keys = [&](const Item &it, int first, int warps) {
        for (int g0 = first; g0 < it.ncol / 8; g0 += 2 * warps) {
            long long off[2];
#pragma unroll
            for (int y = 0; y < 2; y++) {
                const int slot = 8 * (g0 + warps * y) + (lane & 7), key = it.lo + slot;
                long long at = -1;
                if (slot < it.ncol && key < it.hi) {
                    at = key_slot(p, it.seq, key);
                    if (at < 0 && lane < 8) atomicOr(p.err, kErrPage);
                }
                const uint32_t valid = __ballot_sync(0xffffffffu, at >= 0) & 0xffu;
                if (lane == 0 && slot < it.ncol) reinterpret_cast<volatile uint8_t *>(kmask)[g0 + warps * y] = (uint8_t)valid;
                off[y] = at >= 0 ? at * (long long)p.row_bytes : -1;
            }
            if constexpr (KIND == DSPARK_CACHE_BF16) {
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    if (8 * (g0 + warps * y) >= it.ncol) continue;
#pragma unroll
                    for (int e = 0; e < 18; e++) {
                        const int x = lane + 32 * e, row = x / 72, ch = x % 72;
                        const long long o = __shfl_sync(0xffffffffu, off[y], row);
                        cp16(smem_u32(sm) + (ch >> 3) * kKSlice + sw128(8 * (g0 + warps * y) + row, ch & 7),
                             cache + (o >= 0 ? o + ch * 16 : 0), o >= 0);
                    }
                }
            } else {
                uint4 x[2][8];
                float4 sc[2];
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    if (8 * (g0 + warps * y) >= it.ncol) continue;
#pragma unroll
                    for (int e = 0; e < 2; e++) {  // the rope slice as it is
                        const int row = 4 * e + (lane >> 3), ch = lane & 7;
                        const long long o = __shfl_sync(0xffffffffu, off[y], row);
                        cp16(smem_u32(sm) + 8 * kKSlice + sw128(8 * (g0 + warps * y) + row, ch),
                             cache + (o >= 0 ? o + kDL + ch * 16 : 0), o >= 0);
                    }
                    const long long o = __shfl_sync(0xffffffffu, off[y], lane >> 2);
                    const uint8_t *row = cache + (o >= 0 ? o : 0);
                    sc[y] = o >= 0 ? __ldg(reinterpret_cast<const float4 *>(row + kDL + 2 * kDR))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int s = 0; s < 8; s++)
                        x[y][s] = o >= 0 ? __ldg(reinterpret_cast<const uint4 *>(row + 64 * s + 16 * (lane & 3)))
                                         : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    if (8 * (g0 + warps * y) >= it.ncol) continue;
                    const int row = 8 * (g0 + warps * y) + (lane >> 2);
#pragma unroll
                    for (int s = 0; s < 8; s++) {
                        const float f = s < 2 ? sc[y].x : s < 4 ? sc[y].y : s < 6 ? sc[y].z : sc[y].w;
                        const uint4 v = x[y][s];
                        *reinterpret_cast<uint4 *>(sm + s * kKSlice + sw128(row, 2 * (lane & 3))) =
                            make_uint4(fp8x2_bf16(v.x, f), fp8x2_bf16(v.x >> 16, f), fp8x2_bf16(v.y, f),
                                       fp8x2_bf16(v.y >> 16, f));
                        *reinterpret_cast<uint4 *>(sm + s * kKSlice + sw128(row, 2 * (lane & 3) + 1)) =
                            make_uint4(fp8x2_bf16(v.z, f), fp8x2_bf16(v.z >> 16, f), fp8x2_bf16(v.w, f),
                                       fp8x2_bf16(v.w >> 16, f));
                    }
                }
            }
        }
        cp_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
    };
    // The first item's keys by the warps that would wait for them too (128 sequences
    // of 5 tokens, 8-bit rows: 43.5 us with four warps, 40.7).
    if (warp < kLoaders && item_at(p, w, parts, blockIdx.x, it) && it.t0 < it.t1) {
        load_keys(it, warp, kLoaders);
        if (lane == 0) mbar_arrive(kfull);
    }

    if (warp == kWarpQ) {
        // ------------------------------------------------------ Q slices
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            const uint32_t bytes = 128u * min(p.n_h, 128) * w.tpt;
            uint32_t &g = issued_q;
            bool ok = true;
            for (int i = blockIdx.x; ok && item_at(p, w, parts, i, it); i += G)
                for (int t = it.t0; ok && t < it.t1; t++)
                    for (int c = 0; c < kSlices; c++, g++) {
                        const uint32_t s = g % kQSlots;
                        if (g >= kQSlots && !mbar_wait(&qempty[s], (g / kQSlots - 1) & 1, abort_flag, wlim)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&qfull[s], bytes);
                        tma_load_3d(sm + oQ + s * kQSlot, &tm_q, &qfull[s], 64 * c, it.hc * 128, it.q0 + t * w.tpt);
                    }
        }
    } else if (warp >= kWarpA && warp < kWarpQ) {
        // ------------------------------ keys; rope slices of the queries -> TMEM
        const int wr = warp - kWarpA, r = wr * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(wr * 32) << 16) + kColR;
        uint32_t k = 0, n = 0;  // items, tiles
        bool ok = true;
        for (int i = blockIdx.x; ok && item_at(p, w, parts, i, it); i += G) {
            if (it.t0 == it.t1) continue;
            if (k > 0) ok = warp_all(mbar_wait(kempty, (k - 1) & 1, abort_flag, wlim));
            if (!ok) break;
            if (i != (int)blockIdx.x) {
                load_keys(it, wr, 4);
                if (lane < kLoaders / 4) mbar_arrive(kfull);
            }
            k++;
            for (int t = it.t0; ok && t < it.t1; t++, n++) {
                const RowOf o(p, w, it, t, r);
                const int tok = it.q0 + (o.live ? o.i : t * w.tpt);
                const uint4 *src = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)p.q + (long long)tok * p.q_ts +
                                                                   (o.live ? o.h : 0) * p.q_hs + kDL);
                const float4 *tab = reinterpret_cast<const float4 *>(w.tab + (size_t)tok * 32);
                uint32_t x[32], lo[32];
#pragma unroll
                for (int u = 0; u < 8; u++) {
                    const uint4 v = o.live ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
                    const float4 c0 = __ldg(tab + 2 * u), c1 = __ldg(tab + 2 * u + 1);
                    const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
                    const float2 cs[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float a = __uint_as_float(wv[e] << 16), b = __uint_as_float(wv[e] & 0xffff0000u);
                        split_bf16x2(a * cs[e].x - b * cs[e].y, a * cs[e].y + b * cs[e].x, x[4 * u + e], lo[4 * u + e]);
                    }
                }
                if (n > 0) ok = warp_all(mbar_wait(rfree, (n - 1) & 1, abort_flag, wlim));
                if (!ok) break;
                tc_fence_after();
                tmem_st32u(trow, x);
                tmem_st32u(trow + 32, lo);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(rready);
            }
        }
        cp_wait_all();
    } else if (warp == kWarpM) {
        // ------------------------------------------------------ S = Q K^T
        if (lane == 0) {
            uint32_t n = 0, g = 0, k = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = ok && mbar_wait(bar, parity, abort_flag, wlim); };
            for (int i = blockIdx.x; ok && item_at(p, w, parts, i, it); i += G) {
                if (it.t0 == it.t1) continue;
                if (!wait(kfull, k++ & 1)) break;
                const uint32_t idS = idesc_bf16(128, it.ncol, 0);
                for (int t = it.t0; ok && t < it.t1; t++, n++) {
                    if (n >= 2 && !wait(&pvdone[n & 1], ((n >> 1) - 1) & 1)) break;
                    const uint32_t dS = tmem + kColS + (n & 1) * kKeys;
#pragma unroll 1
                    for (int c = 0; c < kSlices; c++, g++) {
                        const uint32_t s = g % kQSlots;
                        if (!wait(&qfull[s], (g / kQSlots) & 1)) break;
                        tc_fence_after();
                        const SDesc qd = sdesc_split(sdesc_sw128(smem_u32(sm + oQ + s * kQSlot), 16, 1024));
                        const SDesc kd = sdesc_split(sdesc_sw128(smem_u32(sm + c * kKSlice), 16, 1024));
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            mma_bf16_ss(dS, qd.at(2 * u), kd.at(2 * u), idS, (c | u) != 0 ? 1u : 0u);
                        mma_commit(&qempty[s]);
                    }
                    if (!wait(rready, n & 1)) break;
                    tc_fence_after();
                    const SDesc hd = sdesc_split(sdesc_sw128(smem_u32(sm + kSlices * kKSlice), 16, 1024));
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        mma_bf16_ts(dS, tmem + kColR + 8 * u, hd.at(2 * u), idS, 1u);
                        mma_bf16_ts(dS, tmem + kColR + 32 + 8 * u, hd.at(2 * u), idS, 1u);
                    }
                    mma_commit(rfree);
                    mma_commit(&sfull[n & 1]);
                }
            }
        }
    } else if (warp == kWarpM + 1) {
        // ------------------------------------------------------- O = P V
        if (lane == 0) {
            const uint32_t idO = idesc_bf16(128, 64, 1);
            uint32_t n = 0, g = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = ok && mbar_wait(bar, parity, abort_flag, wlim); };
            for (int i = blockIdx.x; ok && item_at(p, w, parts, i, it); i += G)
                for (int t = it.t0; ok && t < it.t1; t++, n++) {
                    if (!wait(&pready[n & 1], (n >> 1) & 1)) break;
                    const uint32_t pa = tmem + kColS + (n & 1) * kKeys;
                    const int ksteps = it.ncol / 16;
#pragma unroll 1
                    for (int d = 0; d < kSlices; d++, g++) {
                        const uint32_t s = g & 1, dO = tmem + kColO + 64 * s;
                        if (g >= 2 && !wait(&ofree[s], ((g >> 1) - 1) & 1)) break;
                        tc_fence_after();
                        const SDesc vd = sdesc_split(sdesc_sw128(smem_u32(sm + d * kKSlice), kKSlice, 1024));
#pragma unroll
                        for (int u = 0; u < kKeys / 16; u++)
                            if (u < ksteps) mma_bf16_ts(dO, pa + 8 * u, vd.at(128 * u), idO, u > 0 ? 1u : 0u);
                        if (d == kSlices - 1) {
                            if (t + 1 == it.t1) mma_commit(kempty);
                            mma_commit(&pvdone[n & 1]);
                        }
                        mma_commit(&ofull[2 * (n & 1) + s]);
                    }
                }
        }
    } else if (warp < kWarpA) {
        // ------------------------------------------- softmax and output
        const int wg = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16), tS = trow + kColS + wg * kKeys;
        uint32_t n = 0, k = 0;  // tiles, items
        bool ok = true;
        for (int i = blockIdx.x; ok && item_at(p, w, parts, i, it); i += G) {
            if (it.t0 == it.t1) continue;
            // The keys stay until every warp has seen that it needs them for no row again: at its
            // last tile of the item, or here, where the only one is the other warps' (then after the
            // item before: an arrival must not count for that one).
            if (it.t1 - it.t0 == 1 && (int)(n & 1) != wg) {
                if (k > 0) ok = warp_all(mbar_wait(kempty, (k - 1) & 1, abort_flag, wlim));
                if (ok && lane == 0) mbar_arrive(kempty);
            }
            k++;
            for (int t = it.t0; ok && t < it.t1; t++, n++) {
                if ((int)(n & 1) != wg) continue;
                const bool last = t + 2 >= it.t1;  // of this warp's tiles of the item
                const RowOf o(p, w, it, t, r);
                const SeqView v{it.q0, it.q_len, it.kv, false};
                int lo = 0, hi = 0;
                if (o.live) seq_range(p, v, o.i, &lo, &hi);
                ok = warp_all(mbar_wait(&sfull[wg], (n >> 1) & 1, abort_flag, wlim));
                if (!ok) break;
                tc_fence_after();
                float far = 0.f;  // of keys that the row does not see: 0, or NaN (0 x NaN, 0 x infinity)
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                for (int c = 0; c < it.ncol; c += 16) {
                    float s[16];
                    tmem_ld16(tS + c, s);
                    tmem_wait_ld();
                    const uint32_t in = slot_mask(lo - it.lo - c, hi - it.lo - c) & (kmask[c >> 5] >> (c & 16));
                    if (warp_all((in & 0xffffu) == 0xffffu)) {
#pragma unroll
                        for (int e = 0; e < 16; e++) m[e & 3] = fmaxf(m[e & 3], s[e]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; e++) {
                            const bool mine = (in >> e) & 1;
                            far = mine ? far : fmaf(0.f, s[e], far);
                            m[e & 3] = fmaxf(m[e & 3], mine ? s[e] : -INFINITY);
                        }
                    }
                }
                const float mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * p.scale_log2;
                const float neg = mx == -INFINITY ? 0.f : -mx;
                float l[4] = {0.f, 0.f, 0.f, 0.f};
                // P, bf16, over the S columns already read (two to a column)
                for (int c = 0; c < it.ncol; c += 16) {
                    float s[16];
                    tmem_ld16(tS + c, s);
                    tmem_wait_ld();
                    const uint32_t in = slot_mask(lo - it.lo - c, hi - it.lo - c) & (kmask[c >> 5] >> (c & 16));
                    uint32_t pw[8];
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        s[e] = (in >> e) & 1 ? ex2(fmaf(s[e], p.scale_log2, neg)) : 0.f;
                        l[e & 3] += s[e];
                    }
#pragma unroll
                    for (int e = 0; e < 8; e++) pw[e] = pack_bf16x2(s[2 * e], s[2 * e + 1]);
                    tmem_st8u(tS + c / 2, pw);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pready[wg]);
                const float ls = (l[0] + l[1]) + (l[2] + l[3]);
                // rows beside a key that is not finite and not theirs
                const uint32_t redo = __ballot_sync(0xffffffffu, o.live && far != 0.f && ls == ls);
                if (last && !redo && lane == 0) mbar_arrive(kempty);
                const float inv = ls > 0.f ? 1.f / ls : 0.f;
                // of a row that sees no key, or NaN
                const uint32_t none = ls != ls ? 0x7fff7fffu : 0u;
                const int tok = it.q0 + (o.live ? o.i : 0);
                __nv_bfloat16 *dst = (__nv_bfloat16 *)p.o + (long long)tok * p.o_ts + (long long)(o.live ? o.h : 0) * p.o_hs;
                const bool wide = ((uintptr_t)dst & 31) == 0;
                if (o.live) p.lse[(size_t)tok * p.n_h + o.h] = ls > 0.f ? (mx + log2f(ls)) * kLn2 : ls != ls ? ls : -INFINITY;
#pragma unroll 1
                for (int c = 0; c < kSlices; c++) {
                    const uint32_t g = n * kSlices + c, s = g & 1;
                    ok = warp_all(mbar_wait(&ofull[2 * wg + s], (c >> 1) & 1, abort_flag, wlim));
                    if (!ok) break;
                    tc_fence_after();
                    float v0[32], v1[32];
                    tmem_ld32(trow + kColO + 64 * s, v0);
                    tmem_ld32(trow + kColO + 64 * s + 32, v1);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ofree[s]);
                    if (o.live) {
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            uint32_t x[8];
#pragma unroll
                            for (int e = 0; e < 8; e++) {
                                const float a = u < 2 ? v0[16 * (u & 1) + 2 * e] : v1[16 * (u & 1) + 2 * e];
                                const float b = u < 2 ? v0[16 * (u & 1) + 2 * e + 1] : v1[16 * (u & 1) + 2 * e + 1];
                                x[e] = ls > 0.f ? pack_bf16x2(a * inv, b * inv) : none;
                            }
                            st_global_32B(reinterpret_cast<uint8_t *>(dst) + 128 * c + 32 * u, x, wide);
                        }
                    }
                }
                if (!ok) break;
                if (redo) {
                    // (the keys have long landed: for their writers' view of shared memory)
                    ok = warp_all(mbar_wait(kfull, (k - 1) & 1, abort_flag, wlim));
                    if (!ok) break;
                    for (uint32_t rows = redo; rows; rows &= rows - 1) {
                        const int who = __ffs(rows) - 1;
                        redo_row(p, w, it, sm, kmask, __shfl_sync(0xffffffffu, o.i, who), __shfl_sync(0xffffffffu, o.h, who),
                                 __shfl_sync(0xffffffffu, lo, who) - it.lo, __shfl_sync(0xffffffffu, hi, who) - it.lo);
                    }
                    __syncwarp();
                    if (last && lane == 0) mbar_arrive(kempty);
                }
            }
        }
    }

    // ---------------------------------------------------------- teardown
    __syncthreads();
    if (*abort_flag && lane == 0) {
        volatile int never = 0;
        if (warp == kWarpQ)
            for (uint32_t g = issued_q > kQSlots ? issued_q - kQSlots : 0; g < issued_q; g++)
                mbar_wait(&qfull[g % kQSlots], (g / kQSlots) & 1, &never);
        if (warp >= kWarpM) {
            mma_commit(&drain[warp - kWarpM]);
            mbar_wait(&drain[warp - kWarpM], 0, &never);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpM) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, kErrTimeout);
}

template <int KIND> cudaError_t launch_t(const CUtensorMap &mq, const Paged &p, const PagedPlan &w, int parts, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_short_tc<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    count_launch();
    const long long items = (long long)p.n_seq * w.hchunks * parts;
    return launch_pdl(k_short_tc<KIND>, dim3((unsigned)std::min<long long>(items, 2 * kPairs)), dim3(kThreads), kSmem, st, mq,
                      p, w, parts);
}

}  // namespace

cudaError_t launch_short_tc(const Paged &p, const PagedPlan &w, cudaStream_t st) {
    CUtensorMap mq{};
    if (!make_q_map(&mq, p, w)) return cudaErrorInvalidValue;
    // few sequences: a sequence's tiles are spread over the SMs (at most a part for each of its tiles)
    const long long tiles = (p.T + w.tpt - 1) / w.tpt, most = 2 * kPairs / ((long long)p.n_seq * w.hchunks);
    const int parts = (int)std::max<long long>(1, std::min<long long>(tiles, most));
    return p.kind == DSPARK_CACHE_BF16 ? launch_t<DSPARK_CACHE_BF16>(mq, p, w, parts, st)
                                       : launch_t<DSPARK_CACHE_FP8>(mq, p, w, parts, st);
}

}  // namespace dspark
