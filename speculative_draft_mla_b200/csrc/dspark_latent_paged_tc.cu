// Tensor-core attention of new tokens over the paged latent cache (512-wide
// latents, 64-wide rope keys; bf16 and 8-bit rows), any length and mask.
//
// Row tile: 128 (token, head) rows of one sequence, which share the keys. The
// fp32 output of 128 rows x 512 values would fill tensor memory by itself, so
// two CTAs (a pair) take 256 value columns each and both form the scores: 1.5
// times the tensor work of one, but no exchange, and the second read of a key
// comes from L2. The steps (64 keys of a tile) of all tiles are one list that
// the 74 pairs share evenly, wherever tiles begin and end; a tile that several
// pairs work on leaves partial results (output and log-sum-exp, fp32), which
// the last launch joins. So one token over a long context and a batch of ragged
// chunks keep all SMs equally busy.
//
// Step: S = Q K^T (128 x 64) in TMEM; softmax with a running maximum (the
// output is rescaled only when it grows by more than 2^8); P, bf16, through
// shared memory; O += P V, V the same key rows read MN-major. bf16 keys come by
// TMA in groups of 8 rows where the tile sees all 8 and pages hold whole groups,
// else row by row (TMA gathers of 4 rows x 64 columns, which need no groups, took
// 64 cycles each and were twice as slow); 8-bit rows through registers, where they
// become bf16 (exact: a scale is a power of two). Slots of keys that no row of the
// tile sees are zero, and a row's weight of a key outside its own range is zero. A
// row that sees NaN or +inf is NaN; one whose tile holds a key that is not finite
// and that it does not see has met 0 x NaN, and the last launch evaluates it again.
//
// A CTA holds two steps of keys; the five slices that only S needs (the other
// half's values, the rope keys) are free for the step after next once S is formed,
// the other four once O is.
//
// What bounds it: long contexts (16 sequences of 6 tokens over up to 16384 keys,
// 243 us), the issue and the tensor work of a step, 3000 of its 4000 cycles (40
// products of 64 keys, 50 cycles each where nothing else runs, 4 of 256 columns,
// 134; issued by one lane, 268 us), and the way from S to the softmax and
// back; few keys, the latency of the launches, of Q and of a step (one token over
// 8192 keys, 32.5 us: plan 6, this kernel 13, join 8).
//
// The query's turned rope slice is split as hi + lo of two bf16 (the cache's
// rope keys are exact bf16 operands), so scores and LSE keep 2^-16. P is rounded once
// to bf16 as an operand (2^-8 of each weight, as of the rounded O).
//
// TMEM: O 0..255, S 256..319, Q 320..511 (latent slices 0 - 3, rope hi, rope
// lo). Shared: Q slices 4 - 7, two key stages, P.
// Warps: 0-7 softmax (warps w and w + 4 share 32 rows and take 32 keys and 128
// output columns each); bf16: 8-11 Q, 12 keys, 13 and 14 issue the products of S
// and of O; 8 bits: 8-11 keys of even steps and Q, 12-15 keys of odd steps, 16 and
// 17 the products. Every wait is bounded.
#include <algorithm>

#include "dspark_latent_paged.cuh"
#include "dspark_latent_tc.cuh"

namespace dspark {

namespace {

using namespace tc;

constexpr int kDL = 512, kDR = 64;
// A stage: per group of 8 keys 1 KB (8 rows of 128 swizzled bytes) for each slice
// of 64 columns; first the five slices that only S reads (the other half's, the
// rope slice), group by group, then the CTA's own four.
constexpr int kGroupA = 5 * 1024, kGroupB = 4 * 1024, oPartB = 8 * kGroupA, kStage = oPartB + 8 * kGroupB;
constexpr int oQ = 2 * kStage, oP = oQ + 4 * 128 * 128;
constexpr int oX = oP + 128 * 128;  // pair exchange [2][2][128]: maximum of a step, row sums of a segment
constexpr int oBar = oX + 4 * 512;
constexpr int kSmem = oBar + 304;
static_assert(kSmem <= 232448, "shared memory");
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320, kColR = kColQ + 4 * 32;
constexpr int kSoft = 8, kWarpQ = 8, kWarpKeys = 12;
constexpr int issuer_warp(int kind) { return kind == DSPARK_CACHE_BF16 ? 13 : 16; }  // of S; O's is the next
constexpr int threads_of(int kind) { return (issuer_warp(kind) + 2) * 32; }
constexpr float kGrow = 8.0f;  // log2 units
constexpr float kLn2 = 0.6931471805599453f;

// A part of a tile that a pair works on: steps [s0, s1) of it.
struct Seg {
    int seq, i0, n_tok, hc;       // tokens i0 .. i0 + n_tok of the sequence
    int tok0, kv, q_len, lo, hi;  // first token of q; keys; the tile's key range
    int base;                     // key of the first step's first slot
    int s0, s1, slot;             // slot >= 0: a partial result
};
struct SegCursor {
    long long at, end, per;
    int r, pair;
    __device__ __forceinline__ void begin(const PagedPlan &w) {
        pair = blockIdx.x >> 1;
        r = w.first[pair];  // (not written where the pair has no steps)
        per = w.head->per;
        at = per * pair;
        end = min(at + per, w.head->total);
    }
    __device__ __forceinline__ bool next(const Paged &p, const PagedPlan &w, Seg &g) {
        if (at >= end) return false;
        const PagedTile t = w.tiles[r];
        g.seq = t.seq;
        g.i0 = t.i0;
        g.hc = t.hc;
        g.n_tok = min(w.tpt, t.q_len - t.i0);
        g.tok0 = t.q0 + t.i0;
        g.kv = t.kv;
        g.q_len = t.q_len;
        g.lo = t.lo;
        g.hi = t.hi;
        g.base = t.lo & ~7;
        g.s0 = (int)(at - t.start);
        const long long b = t.start + t.steps, e = min(end, b);
        g.s1 = (int)(e - t.start);
        g.slot = g.s0 == 0 && e == b ? -1 : 2 * pair + (g.s0 == 0 ? 1 : 0);
        at = e;
        r++;
        return true;
    }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Two e4m3 codes (low half of w) times s as a bf16 pair.
__device__ __forceinline__ uint32_t fp8x2_bf16(uint32_t w, float s) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16x2(f.x * s, f.y * s);
}

// The (token, head) of a tile's row.
struct RowOf {
    int ti, h;
    bool live;
    __device__ __forceinline__ RowOf(const Paged &p, const PagedPlan &w, const Seg &g, int r) {
        ti = w.tpt > 1 || p.n_h == 128 ? r / p.n_h : 0;
        h = g.hc * 128 + r - ti * p.n_h;
        live = ti < g.n_tok && h < p.n_h && (ti == 0 || w.hchunks == 1);
    }
};

// A segment's queries, by four warps (thread = row r of 128). TMA brings latent
// slices 0 - 3 into Q's shared memory (rows one to a lane would cost a request
// each), from where they go to tensor memory; then slices 4 - 7 come to stay. The
// rope slice is turned on its way to tensor memory. land: both copies' barrier.
__device__ __forceinline__ bool load_q(const Paged &p, const PagedPlan &w, const Seg &sg, const CUtensorMap *tm, uint8_t *sm,
                                       uint32_t tmem, int wr, uint32_t bytes, uint64_t *land, uint64_t *read, uint64_t *ready,
                                       uint32_t k, uint32_t &armed, volatile int *abort_flag, uint64_t wlim) {
    const int lane = threadIdx.x & 31, r = wr * 32 + lane, h0 = sg.hc * 128;
    const uint32_t trow = tmem + ((uint32_t)(wr * 32) << 16);
    if (wr == 0 && lane == 0) {
        mbar_arrive_expect_tx(land, 4 * bytes);
        armed++;
        for (int c = 0; c < 4; c++) tma_load_3d(sm + oQ + c * 16384, tm, land, 64 * c, h0, sg.tok0);
    }
    __syncwarp();
    const RowOf o(p, w, sg, r);
    const int tok = sg.tok0 + (o.live ? o.ti : 0);
    const uint4 *src = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)p.q + (long long)tok * p.q_ts +
                                                       (o.live ? o.h : 0) * p.q_hs + kDL);
    const float4 *tab = reinterpret_cast<const float4 *>(w.tab + (size_t)tok * 32);
    tc_fence_after();
    uint32_t x[32], lo[32];
#pragma unroll
    for (int u = 0; u < 8; u++) {
        const uint4 v = o.live ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
        const float4 c0 = __ldg(tab + 2 * u), c1 = __ldg(tab + 2 * u + 1);
        const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
        const float2 cs[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a = __uint_as_float(wv[i] << 16), b = __uint_as_float(wv[i] & 0xffff0000u);
            split_bf16x2(a * cs[i].x - b * cs[i].y, a * cs[i].y + b * cs[i].x, x[4 * u + i], lo[4 * u + i]);
        }
    }
    tmem_st32u(trow + kColR, x);
    tmem_st32u(trow + kColR + 32, lo);
    if (!warp_all(mbar_wait(land, 0, abort_flag, wlim))) {  // (its even phase)
        tmem_wait_st();  // tensor memory is about to be released
        return false;
    }
#pragma unroll
    for (int c = 0; c < 4; c++) {
#pragma unroll
        for (int u = 0; u < 8; u++) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sm + oQ + c * 16384 + sw128(r, u));
            x[4 * u] = v.x;
            x[4 * u + 1] = v.y;
            x[4 * u + 2] = v.z;
            x[4 * u + 3] = v.w;
        }
        tmem_st32u(trow + kColQ + 32 * c, x);
    }
    tmem_wait_st();
    tc_fence_before();
    fence_proxy_async_smem();  // the reads come before the next copies' writes
    __syncwarp();
    if (lane == 0) {
        mbar_arrive(read);
        mbar_arrive(ready);
    }
    bool ok = true;
    if (wr == 0 && lane == 0) {
        ok = mbar_wait(read, k & 1, abort_flag, wlim);
        if (ok) {
            mbar_arrive_expect_tx(land, 4 * bytes);
            armed++;
            for (int c = 0; c < 4; c++) tma_load_3d(sm + oQ + c * 16384, tm, land, 64 * (4 + c), h0, sg.tok0);
        }
    }
    return warp_all(ok);
}

template <int KIND>
__global__ void __launch_bounds__(threads_of(KIND), 1)
    k_paged_tc(const __grid_constant__ CUtensorMap tm_k4, const __grid_constant__ CUtensorMap tm_k1,
               const __grid_constant__ CUtensorMap tm_q, const Paged p, const PagedPlan w) {
    constexpr int kWarpM = issuer_warp(KIND), kThreads = threads_of(KIND);
    constexpr int kFull = KIND == DSPARK_CACHE_BF16 ? 2 : 4;  // arrivals for a part of a stage
    extern __shared__ __align__(1024) uint8_t sm[];  // swizzle atoms: no room for slack
    // of stage s: part 2 s the slices that only S reads, part 2 s + 1 those that O reads too
    uint64_t *kfull = reinterpret_cast<uint64_t *>(sm + oBar), *kempty = kfull + 4;
    uint64_t *sfull = kempty + 4, *sfree = sfull + 1, *pready = sfull + 2, *pvdone = sfull + 3;
    uint64_t *qready = sfull + 4, *qfree = sfull + 5, *ofree = sfull + 6, *drain = sfull + 7;
    uint64_t *qland = sfull + 9, *qread = sfull + 10, *xbar = sfull + 11, *lbar = xbar + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(lbar + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(lbar + 4) + 1;
    // [4][4]: 16 keys' validity each, of step g at g % 4 (a stage's first part is
    // free before the softmax has read them)
    volatile uint16_t *kmask = reinterpret_cast<volatile uint16_t *>(lbar + 5);
    float *xm = reinterpret_cast<float *>(sm + oX);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = blockIdx.x & 1;
    const uint64_t wlim = p.wait_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; i++) {
            mbar_init(&kfull[i], kFull);
            mbar_init(&kempty[i], 1);
        }
        mbar_init(sfull, 1);
        mbar_init(sfree, kSoft);
        mbar_init(pready, kSoft);
        mbar_init(pvdone, 1);
        mbar_init(qready, 4);
        mbar_init(qland, 1);
        mbar_init(qread, 4);
        mbar_init(qfree, 1);
        mbar_init(ofree, kSoft);
        mbar_init(&drain[0], 1);
        mbar_init(&drain[1], 1);
        for (int i = 0; i < 8; i++) mbar_init(&xbar[i], 2);
        for (int i = 0; i < 4; i++) mbar_init(&lbar[i], 2);
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
    if (w.head->total == 0) {  // all sequences went to the short kernel
        if (warp == kWarpM) tmem_dealloc(tmem, 512);
        return;
    }
    SegCursor cur;
    cur.begin(w);
    Seg sg;
    uint32_t issued = 0, q_issued = 0;  // the loaders' parts of steps; copies of Q
    const uint32_t q_bytes = 128u * min(p.n_h, 128) * w.tpt;  // of a slice

    if (KIND == DSPARK_CACHE_BF16 && warp == kWarpKeys) {
        // ------------------------------------------------- bf16 keys -> stages
        if (lane == 0) tma_prefetch_desc(&tm_k4);
        const bool groups = p.page_size % 8 == 0;
        const uint8_t *cache = (const uint8_t *)p.cache;
        bool ok = true;
        uint32_t g = 0;
        while (ok && cur.next(p, w, sg))
            for (int t = sg.s0; ok && t < sg.s1; t++, g++) {
                const int st = g & 1;
                // lane l: the slots of keys l and l + 32 of the step
                int row[2];
                uint32_t valid[2];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const int key = sg.base + t * kStepKeys + lane + 32 * i;
                    long long slot = -1;
                    if (key >= sg.lo && key < sg.hi) {
                        slot = key_slot(p, sg.seq, key);
                        if (slot < 0) atomicOr(p.err, kErrPage);
                    }
                    valid[i] = __ballot_sync(0xffffffffu, slot >= 0);
                    row[i] = (int)slot;
                }
                // lane l < 8: whether group l is whole, and its first slot
                const int ga = __shfl_sync(0xffffffffu, row[0], 8 * (lane & 3));
                const int gb = __shfl_sync(0xffffffffu, row[1], 8 * (lane & 3));
                const int gslot = lane & 4 ? gb : ga;
                const bool whole = groups && ((lane & 4 ? valid[1] : valid[0]) >> (8 * (lane & 3)) & 0xffu) == 0xffu;
                const uint32_t wholes = __ballot_sync(0xffffffffu, whole) & 0xffu;
#pragma unroll
                for (int part = 0; part < 2; part++) {
                    if (g >= 2) ok = warp_all(mbar_wait(&kempty[2 * st + part], ((g >> 1) - 1) & 1, abort_flag, wlim));
                    if (!ok) break;
                    uint64_t *full = &kfull[2 * st + part];
                    uint8_t *dst = sm + st * kStage + (part ? oPartB : 0);
                    if (lane == 0) {
                        if (part == 0) {
                            kmask[(g & 3) * 4] = (uint16_t)valid[0];
                            kmask[(g & 3) * 4 + 1] = (uint16_t)(valid[0] >> 16);
                            kmask[(g & 3) * 4 + 2] = (uint16_t)valid[1];
                            kmask[(g & 3) * 4 + 3] = (uint16_t)(valid[1] >> 16);
                        }
                        mbar_arrive_expect_tx(full, __popc(wholes) * (part ? kGroupB : kGroupA));
                    }
                    __syncwarp();
                    issued = 2 * g + part + 1;
                    if (lane < 8 && whole) {
                        if (part == 0) {
                            tma_load_3d(dst + lane * kGroupA, &tm_k4, full, 0, gslot, 4 * (half ^ 1));
                            tma_load_3d(dst + lane * kGroupA + 4096, &tm_k1, full, 0, gslot, 8);
                        } else {
                            tma_load_3d(dst + lane * kGroupB, &tm_k4, full, 0, gslot, 4 * half);
                        }
                    }
                    if (wholes != 0xffu) {
                        // the other groups row by row: lane's row of a group, every fourth 16 bytes
                        for (int gr = 0; gr < 8; gr++) {
                            if ((wholes >> gr) & 1) continue;
                            const int key = 8 * gr + (lane >> 2);
                            const int a = __shfl_sync(0xffffffffu, row[0], key & 31);
                            const int b = __shfl_sync(0xffffffffu, row[1], key & 31);
                            const int slot = gr >= 4 ? b : a;
                            const uint8_t *src = cache + (slot >= 0 ? (size_t)slot * p.row_bytes : 0);
#pragma unroll
                            for (int i = 0; i < 10; i++) {
                                const int u = 4 * i + (lane & 3), n = u >> 3;  // unit of the part; its slice
                                if (part == 1 && n >= 4) continue;
                                const int c = part ? 4 * half + n : n == 4 ? 8 : 4 * (half ^ 1) + n;
                                cp16(smem_u32(dst) + gr * (part ? kGroupB : kGroupA) + n * 1024 + sw128(lane >> 2, u & 7),
                                     src + c * 128 + (u & 7) * 16, slot >= 0);
                            }
                        }
                        cp_wait_all();
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) mbar_arrive(full);
                }
            }
    } else if (KIND == DSPARK_CACHE_FP8 && warp >= kWarpQ && warp < kWarpM) {
        // -------------------------------------- 8-bit keys -> bf16 stages; Q
        const int gp = (warp - kWarpQ) >> 2, wr = (warp - kWarpQ) & 3;  // stage; 16 rows from 16 wr
        uint32_t g = 0, k = 0;
        bool ok = true;
        for (; ok && cur.next(p, w, sg); k++) {
            if (gp == 0) {
                if (k > 0) ok = warp_all(mbar_wait(qfree, (k - 1) & 1, abort_flag, wlim));
                if (!ok) break;
                ok = load_q(p, w, sg, &tm_q, sm, tmem, wr, q_bytes, qland, qread, qready, k, q_issued, abort_flag, wlim);
                if (!ok) break;
            }
            for (int t = sg.s0; ok && t < sg.s1; t++, g++) {
                if ((int)(g & 1) != gp) continue;
                // lane l < 16: the slot of key 16 wr + l of the step
                const int key = sg.base + t * kStepKeys + 16 * wr + (lane & 15);
                long long slot = -1;
                if (key >= sg.lo && key < sg.hi) {
                    slot = key_slot(p, sg.seq, key);
                    if (slot < 0 && lane < 16) atomicOr(p.err, kErrPage);
                }
                const uint32_t valid = __ballot_sync(0xffffffffu, slot >= 0) & 0xffffu;
                const uint8_t *cache = (const uint8_t *)p.cache;
                const long long off = slot >= 0 ? slot * (long long)p.row_bytes : -1;
                // lane: rows 8 rb + lane / 4, 16 codes of each slice; x[.][0 .. 3] of the
                // other half, x[.][4 .. 7] of the own
                uint4 x[2][8];
                float2 sc[2][2];
#pragma unroll
                for (int rb = 0; rb < 2; rb++) {
                    const long long o = __shfl_sync(0xffffffffu, off, 8 * rb + (lane >> 2));
                    const uint8_t *row = cache + (o >= 0 ? o : 0);
#pragma unroll
                    for (int part = 0; part < 2; part++) {
                        const int up = half ^ part ^ 1;
                        sc[rb][part] = o >= 0 ? __ldg(reinterpret_cast<const float2 *>(row + kDL + 2 * kDR) + up)
                                              : make_float2(0.f, 0.f);
#pragma unroll
                        for (int n = 0; n < 4; n++)
                            x[rb][4 * part + n] =
                                o >= 0 ? __ldg(reinterpret_cast<const uint4 *>(row + 256 * up + 64 * n + 16 * (lane & 3)))
                                       : make_uint4(0, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int part = 0; part < 2; part++) {
                    if (g >= 2) ok = warp_all(mbar_wait(&kempty[2 * gp + part], ((g >> 1) - 1) & 1, abort_flag, wlim));
                    if (!ok) break;
                    if (part == 0) {
                        if (lane == 0) kmask[(g & 3) * 4 + wr] = (uint16_t)valid;
                        // the rope slice as it is
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int row = 4 * i + (lane >> 3), ch = lane & 7;
                            const long long o = __shfl_sync(0xffffffffu, off, row);
                            cp16(smem_u32(sm) + gp * kStage + (2 * wr + (row >> 3)) * kGroupA + 4096 + sw128(row & 7, ch),
                                 cache + (o >= 0 ? o + kDL + ch * 16 : 0), o >= 0);
                        }
                    }
#pragma unroll
                    for (int rb = 0; rb < 2; rb++) {
                        uint8_t *dst = sm + gp * kStage + (part ? oPartB + (2 * wr + rb) * kGroupB : (2 * wr + rb) * kGroupA);
#pragma unroll
                        for (int n = 0; n < 4; n++) {
                            const float f = n < 2 ? sc[rb][part].x : sc[rb][part].y;
                            const uint4 v = x[rb][4 * part + n];
                            *reinterpret_cast<uint4 *>(dst + n * 1024 + sw128(lane >> 2, 2 * (lane & 3))) =
                                make_uint4(fp8x2_bf16(v.x, f), fp8x2_bf16(v.x >> 16, f), fp8x2_bf16(v.y, f),
                                           fp8x2_bf16(v.y >> 16, f));
                            *reinterpret_cast<uint4 *>(dst + n * 1024 + sw128(lane >> 2, 2 * (lane & 3) + 1)) =
                                make_uint4(fp8x2_bf16(v.z, f), fp8x2_bf16(v.z >> 16, f), fp8x2_bf16(v.w, f),
                                           fp8x2_bf16(v.w >> 16, f));
                        }
                    }
                    if (part == 0) cp_wait_all();
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kfull[2 * gp + part]);
                }
            }
        }
        cp_wait_all();
    } else if (KIND == DSPARK_CACHE_BF16 && warp >= kWarpQ && warp < kWarpKeys) {
        // -------------------------------------- Q -> shared and tensor memory
        uint32_t k = 0;  // segments
        bool ok = true;
        int before = 0;  // steps of the segment before
        for (; ok && cur.next(p, w, sg); k++) {
            // (the one wait that lasts as long as a segment: a limit for each 2048 steps, 5 ms)
            if (k > 0) ok = warp_all(mbar_wait(qfree, (k - 1) & 1, abort_flag, wlim * (1 + (before >> 11))));
            if (!ok) break;
            before = sg.s1 - sg.s0;
            ok = load_q(p, w, sg, &tm_q, sm, tmem, warp - kWarpQ, q_bytes, qland, qread, qready, k, q_issued, abort_flag, wlim);
        }
    } else if (warp == kWarpM) {
        // ------------------------------------------------------ S = Q K^T
        const uint32_t idS = idesc_bf16(128, kStepKeys, 0), tm = uniform(tmem), dS = tm + kColS;
        const SDesc qd = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oQ), 16, 1024)));
        uint32_t g = 0, k = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return ok = ok && warp_all(mbar_wait(bar, parity, abort_flag, wlim));
        };
        // latent slices 0 - 3 (Q in tensor memory) or 4 - 7 (Q in shared memory); kd: the first of the four
        auto four = [&](const SDesc &kd, bool upper, bool first) {
            if (upper) {
#pragma unroll
                for (int n = 0; n < 16; n++)
                    mma_bf16_ss_warp(dS, qd.at((n >> 2) * 1024 + 2 * (n & 3)), kd.at((n >> 2) * 64 + 2 * (n & 3)), idS,
                                !first || n > 0);
            } else {
#pragma unroll
                for (int n = 0; n < 16; n++)
                    mma_bf16_ts_warp(dS, tm + kColQ + 8 * n, kd.at((n >> 2) * 64 + 2 * (n & 3)), idS, !first || n > 0);
            }
        };
        for (; ok && cur.next(p, w, sg); k++)
            for (int t = sg.s0; t < sg.s1; t++, g++) {
                const int st = g & 1;
                // (Q in tensor memory, then in shared memory: its barrier's odd phase)
                if (t == sg.s0 && (!wait(qready, k & 1) || !wait(qland, 1))) break;
                if (g > 0 && !wait(sfree, (g - 1) & 1)) break;
                if (!wait(&kfull[2 * st], (g >> 1) & 1)) break;
                tc_fence_after();
                const SDesc kd = uniform(sdesc_split(sdesc_sw128(smem_u32(sm) + st * kStage, 16, kGroupA)));
                four(kd, half == 0, true);
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const uint64_t b = kd.at(4 * 64 + 2 * u);
                    mma_bf16_ts_warp(dS, tm + kColR + 8 * u, b, idS, 1u);
                    mma_bf16_ts_warp(dS, tm + kColR + 32 + 8 * u, b, idS, 1u);
                }
                mma_commit_warp(&kempty[2 * st]);
                if (!wait(&kfull[2 * st + 1], (g >> 1) & 1)) break;
                tc_fence_after();
                four(uniform(sdesc_split(sdesc_sw128(smem_u32(sm) + st * kStage + oPartB, 16, kGroupB))), half != 0,
                     false);
                if (t + 1 == sg.s1) mma_commit_warp(qfree);
                mma_commit_warp(sfull);
            }
    } else if (warp == kWarpM + 1) {
        // ------------------------------------------------------- O += P V
        const uint32_t idO = idesc_bf16(128, 256, 1), tm = uniform(tmem);
        const SDesc pd = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oP), 16, 1024)));
        uint32_t g = 0, k = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return ok = ok && warp_all(mbar_wait(bar, parity, abort_flag, wlim));
        };
        for (; ok && cur.next(p, w, sg); k++)
            for (int t = sg.s0; t < sg.s1; t++, g++) {
                const int st = g & 1;
                if (!wait(pready, g & 1) || (t == sg.s0 && k > 0 && !wait(ofree, (k - 1) & 1))) break;
                tc_fence_after();
                const SDesc vd = uniform(sdesc_split(sdesc_sw128(smem_u32(sm) + st * kStage + oPartB, 1024, kGroupB)));
#pragma unroll
                for (int u = 0; u < 4; u++)
                    mma_bf16_ss_warp(tm + kColO, pd.at(2 * u), vd.at(2 * (kGroupB / 16) * u), idO,
                                     t != sg.s0 || u > 0 ? 1u : 0u);
                mma_commit_warp(&kempty[2 * st + 1]);
                mma_commit_warp(pvdone);
            }
    } else {
        // -------------------------------------------------------- softmax
        const int q4 = warp & 3, hf = warp >> 2, r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        uint32_t g = 0, sk = 0;
        bool ok = true;
        for (; ok && cur.next(p, w, sg); sk++) {
            const RowOf row(p, w, sg, r);
            const int ti = row.ti, h = row.h;
            const bool live = row.live;
            const SeqView v{sg.tok0 - sg.i0, sg.q_len, sg.kv, false};
            int lo = 0, hi = 0;
            if (live) seq_range(p, v, sg.i0 + ti, &lo, &hi);
            float m = -INFINITY, l = 0.f;
            bool bad = false;  // a key outside the row's range is not finite
            for (int t = sg.s0; t < sg.s1; t++, g++) {
                ok = warp_all(mbar_wait(sfull, g & 1, abort_flag, wlim));
                if (!ok) break;
                tc_fence_after();
                float s[32];
                tmem_ld32(trow + kColS + 32 * hf, s);
                const uint32_t km = kmask[(g & 3) * 4 + 2 * hf] | ((uint32_t)kmask[(g & 3) * 4 + 2 * hf + 1] << 16);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sfree);
                const int k0 = sg.base + t * kStepKeys + 32 * hf;
                const int c0 = max(lo - k0, 0), c1 = min(hi - k0, 32);
                uint32_t rm = c1 > c0 ? (c1 >= 32 ? 0xffffffffu : (1u << c1) - 1u) & ~((1u << (c0 & 31)) - 1u) : 0u;
                rm &= km;
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (!warp_all(rm == 0xffffffffu)) {
                    float far = 0.f;  // 0, or NaN (0 x NaN, 0 x infinity)
#pragma unroll
                    for (int c = 0; c < 32; c++) {
                        const bool in = (rm >> c) & 1;
                        far = in ? far : fmaf(0.f, s[c], far);
                        s[c] = in ? s[c] : -INFINITY;
                    }
                    bad |= far != 0.f;
                }
#pragma unroll
                for (int c = 0; c < 32; c++) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
                const float mh = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (t == sg.s0 && sk > 0) {  // the other warp has read the last segment's sums from here
                    ok = warp_all(mbar_wait(&lbar[q4], 1, abort_flag, wlim));
                    if (!ok) break;
                }
                xm[((g & 1) * 2 + hf) * 128 + r] = mh;
                __syncwarp();
                if (lane == 0) mbar_arrive(&xbar[2 * q4 + (g & 1)]);
                ok = warp_all(mbar_wait(&xbar[2 * q4 + (g & 1)], (g >> 1) & 1, abort_flag, wlim));
                if (!ok) break;
                const float mt = fmaxf(mh, xm[((g & 1) * 2 + (hf ^ 1)) * 128 + r]) * p.scale_log2;
                bool resc = false;
                float alpha = 1.f;
                if (mt > m + kGrow || (m == -INFINITY && mt > m)) {
                    if (m != -INFINITY) {
                        resc = true;
                        alpha = ex2(m - mt);
                    }
                    m = mt;
                }
                const bool some = m != -INFINITY;
                const float neg = some ? -m : 0.f;
                float ps[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t pw[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float e0 = ex2(fmaf(s[c], p.scale_log2, neg)), e1 = ex2(fmaf(s[c + 1], p.scale_log2, neg));
                    ps[c & 3] += e0;
                    ps[(c + 1) & 3] += e1;
                    pw[c / 2] = pack_bf16x2(e0, e1);
                }
                l = l * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
                if (g > 0) {  // P and O are free once the product before has completed
                    ok = warp_all(mbar_wait(pvdone, (g - 1) & 1, abort_flag, wlim));
                    if (!ok) break;
                }
                if (__any_sync(0xffffffffu, resc)) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 128 * hf; c < 128 * hf + 128; c += 32) {
                        float o[32];
                        tmem_ld32(trow + kColO + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i++) o[i] *= alpha;
                        tmem_st32(trow + kColO + c, o);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                }
#pragma unroll
                for (int u = 0; u < 4; u++)
                    *reinterpret_cast<uint4 *>(sm + oP + sw128(r, 4 * hf + u)) =
                        make_uint4(pw[4 * u], pw[4 * u + 1], pw[4 * u + 2], pw[4 * u + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(pready);
            }
            if (!ok) break;
            // A row's share of the sums: NaN where a key of its own is not finite; else
            // -1 where one that it does not see is not: its product with that key was not
            // zero (0 x NaN), and it is left to the last launch.
            const float mine = bad && l == l ? -1.f : l;
            xm[((g & 1) * 2 + hf) * 128 + r] = mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(&lbar[q4]);
            ok = warp_all(mbar_wait(pvdone, (g - 1) & 1, abort_flag, wlim)) &&
                 warp_all(mbar_wait(&lbar[q4], 0, abort_flag, wlim));
            if (!ok) break;
            tc_fence_after();
            const float theirs = xm[((g & 1) * 2 + (hf ^ 1)) * 128 + r];
            __syncwarp();
            if (lane == 0) mbar_arrive(&lbar[q4]);
            const float lt = mine + theirs;
            const uint32_t redo = __ballot_sync(0xffffffffu, live && lt == lt && (mine < 0.f || theirs < 0.f));
            if (redo && lane == 0) {
                atomicOr(&w.tiles[cur.r - 1].redo[q4], redo);
                w.head->redo = 1;
            }
            const int tok = sg.tok0 + ti, col0 = 256 * half + 128 * hf;
            const float none = lt != lt ? lt : 0.f;  // of a row that sees no key, or NaN
            const float lse2 = lt > 0.f ? m + log2f(lt) : lt != lt ? lt : -INFINITY;
            uint8_t *dst = nullptr;
            float *pdst = nullptr;
            if (sg.slot >= 0) {
                pdst = w.part_o + ((size_t)sg.slot * 128 + r) * kDL + col0;
                if (half == 0 && hf == 0) w.part_lse[sg.slot * 128 + r] = lse2;
            } else if (live) {
                dst = (uint8_t *)((__nv_bfloat16 *)p.o + (long long)tok * p.o_ts + (long long)h * p.o_hs + col0);
                if (half == 0 && hf == 0) p.lse[(size_t)tok * p.n_h + h] = lse2 * kLn2;
            }
            const float f = lt > 0.f ? 1.f / lt : 0.f;
            const bool wide = ((uintptr_t)dst & 31) == 0;
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                float o[32];
                tmem_ld32(trow + kColO + 128 * hf + c, o);
                tmem_wait_ld();
                // (a row that sees no key may hold what was there before)
#pragma unroll
                for (int i = 0; i < 32; i++) o[i] = lt > 0.f ? o[i] * f : none;
                if (pdst && live) {
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        uint32_t x[8];
#pragma unroll
                        for (int i = 0; i < 8; i++) x[i] = __float_as_uint(o[8 * u + i]);
                        st_global_32B(pdst + c + 8 * u, x, true);
                    }
                } else if (dst) {
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        uint32_t x[8];
#pragma unroll
                        for (int i = 0; i < 8; i++) x[i] = pack_bf16x2(o[16 * u + 2 * i], o[16 * u + 2 * i + 1]);
                        st_global_32B(dst + 2 * c + 32 * u, x, wide);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ofree);
        }
    }

    // ---------------------------------------------------------- teardown
    __syncthreads();
    if (*abort_flag && warp >= kWarpM) mma_commit_warp(&drain[warp - kWarpM]);
    if (*abort_flag && lane == 0) {
        volatile int never = 0;
        if (KIND == DSPARK_CACHE_BF16 && warp == kWarpKeys)
            for (uint32_t n = issued > 4 ? issued - 4 : 0; n < issued; n++)  // part n % 2 of step n / 2
                mbar_wait(&kfull[n & 3], (n >> 2) & 1, &never);
        if (warp == kWarpQ && q_issued) mbar_wait(qland, (q_issued - 1) & 1, &never);
        if (warp >= kWarpM) mbar_wait(&drain[warp - kWarpM], 0, &never);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpM) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, kErrTimeout);
}

// The last launch joins the parts of the tiles that pairs shared, and evaluates
// rows again that met a foreign value that is not finite. Part k of a tile is pair
// p0 + k's, in its slot 1 for the tile's beginning, 0 after it.
__device__ __forceinline__ size_t part_row(int p0, int k, int row) {
    return (size_t)(2 * (p0 + k) + (k == 0)) * 128 + row;
}
// Tiles of up to kFew parts go a row to a warp (16 columns to a lane), others a
// row to a CTA: four groups of 128 threads take every fourth part, four columns
// to a thread.
constexpr int kFew = 8;
constexpr int kJoinSmem = 3 * 128 * 16;

// Evaluates rows again whose product met a key that is not finite and that they do
// not see: over their own keys, a row to a CTA, its keys in 16 runs, one to a warp.
// Here, after the attention, no wait of that kernel stands on it (in its softmax
// warps a NaN beside 6 tokens over 16384 keys took 80 - 280 ms, and time-outs were
// near), and all SMs share the rows.
template <int KIND> __device__ __forceinline__ void redo_rows(const Paged &p, const PagedPlan &w, uint8_t *smem) {
    constexpr int kAtOnce = 64;  // tiles whose masks are looked at together
    uint4 *masks = reinterpret_cast<uint4 *>(smem);
    float *qs = reinterpret_cast<float *>(masks + kAtOnce), *col = qs + kDL + kDR, *pm = col + kDL, *pl = pm + 16;
    static_assert(kAtOnce * 16 + (2 * kDL + kDR + 32) * 4 <= kJoinSmem, "shared memory");
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = w.head->n_tiles;
    uint32_t seen = 0;  // rows so far: they are dealt to the CTAs in turn
    for (int t0 = 0; t0 < n; t0 += kAtOnce) {
        uint4 mine = make_uint4(0, 0, 0, 0);
        if (threadIdx.x < kAtOnce && t0 + (int)threadIdx.x < n) {
            mine = *reinterpret_cast<const uint4 *>(w.tiles[t0 + threadIdx.x].redo);
            masks[threadIdx.x] = mine;
        }
        const bool some_tile = __syncthreads_or((mine.x | mine.y | mine.z | mine.w) != 0);
        for (int t = t0; some_tile && t < min(n, t0 + kAtOnce); t++)
            for (int q4 = 0; q4 < 4; q4++)
                for (uint32_t rows = reinterpret_cast<const uint32_t *>(&masks[t - t0])[q4]; rows; rows &= rows - 1) {
                    if (seen++ % gridDim.x != blockIdx.x) continue;
                    const PagedTile &tl = w.tiles[t];
                    const int row = 32 * q4 + __ffs(rows) - 1;
                    const int ti = w.tpt > 1 || p.n_h == 128 ? row / p.n_h : 0, h = tl.hc * 128 + row - ti * p.n_h;
                    const int i = tl.i0 + ti, tok = tl.q0 + i;
                    const SeqView v{tl.q0, tl.q_len, tl.kv, false};
                    int lo, hi;
                    seq_range(p, v, i, &lo, &hi);
                    // the query, its rope slice turned, for all warps
                    const __nv_bfloat16 *qrow =
                        (const __nv_bfloat16 *)p.q + (long long)tok * p.q_ts + (long long)h * p.q_hs;
                    __syncthreads();  // the row before is done
                    qs[threadIdx.x] = to_f(qrow[threadIdx.x]);
                    if (threadIdx.x < kDR / 2) {
                        const float2 t = w.tab[(size_t)tok * 32 + threadIdx.x];
                        const float x0 = to_f(qrow[kDL + 2 * threadIdx.x]), x1 = to_f(qrow[kDL + 2 * threadIdx.x + 1]);
                        qs[kDL + 2 * threadIdx.x] = x0 * t.x - x1 * t.y;
                        qs[kDL + 2 * threadIdx.x + 1] = x0 * t.y + x1 * t.x;
                    }
                    __syncthreads();
                    // the warp's run of keys: acc = sum 2^(s - m) c, l the sum of the weights
                    float acc[kDL / 32], m = -INFINITY, l = 0.f;
#pragma unroll
                    for (int e = 0; e < kDL / 32; e++) acc[e] = 0.f;
                    const int run = (hi - lo + 15) / 16, k0 = min(hi, lo + warp * run), k1 = min(hi, k0 + run);
                    for (int key = k0; key < k1; key++) {
                        const long long slot = key_slot(p, tl.seq, key);
                        if (slot < 0) continue;  // (a page out of range, reported by the attention)
                        const uint8_t *krow = (const uint8_t *)p.cache + (size_t)slot * p.row_bytes;
                        float c[kDL / 32], x[1] = {0.f};
#pragma unroll
                        for (int e = 0; e < kDR / 32; e++)
                            x[0] = fmaf(qs[kDL + lane + 32 * e], CacheRow<KIND>::at(krow, kDL + lane + 32 * e, kDL, kDR), x[0]);
#pragma unroll
                        for (int e = 0; e < kDL / 32; e++) {
                            c[e] = CacheRow<KIND>::at(krow, lane + 32 * e, kDL, kDR);
                            x[0] = fmaf(qs[lane + 32 * e], c[e], x[0]);
                        }
                        warp_sum_all(x);
                        const float sc = x[0] * p.scale_log2, mn = fmaxf(m, sc);
                        const float mu = mn == -INFINITY ? 0.f : mn;  // (scores of -inf or NaN only)
                        const float old = exp2f(m - mu), f = exp2f(sc - mu);
                        l = fmaf(l, old, f);
#pragma unroll
                        for (int e = 0; e < kDL / 32; e++) acc[e] = fmaf(acc[e], old, f * c[e]);
                        m = mn;
                    }
                    if (lane == 0) {
                        pm[warp] = m;
                        pl[warp] = l;
                    }
                    col[threadIdx.x] = 0.f;
                    __syncthreads();
                    float mx = -INFINITY, sum = 0.f;
                    for (int k = 0; k < 16; k++) mx = fmaxf(mx, pm[k]);
                    // (a run of no key, or of scores of -inf or NaN: its l is 0 or NaN)
                    const auto weight = [&](float x) { return x == -INFINITY ? 1.f : exp2f(x - mx); };
                    for (int k = 0; k < 16; k++) {
                        sum = fmaf(weight(pm[k]), pl[k], sum);
                        if (warp == k) {
                            const float f = weight(m);
#pragma unroll
                            for (int e = 0; e < kDL / 32; e++) col[lane + 32 * e] = fmaf(f, acc[e], col[lane + 32 * e]);
                        }
                        __syncthreads();
                    }
                    const bool some = sum != 0.f;
                    ((__nv_bfloat16 *)p.o)[(long long)tok * p.o_ts + (long long)h * p.o_hs + threadIdx.x] =
                        __float2bfloat16_rn(some ? col[threadIdx.x] / sum : 0.f);
                    if (threadIdx.x == 0) p.lse[(size_t)tok * p.n_h + h] = some ? (mx + log2f(sum)) * kLn2 : -INFINITY;
                }
        __syncthreads();  // (masks)
    }
}

template <int KIND>
__global__ void __launch_bounds__(512, 2)
    k_paged_join(const __grid_constant__ Paged p, const __grid_constant__ PagedPlan w) {
    static_assert(kDL == 512, "a column to a thread");
    __shared__ float wt[kPairs + 1];
    __shared__ float4 sum[3][128];
    static_assert(sizeof(sum) == kJoinSmem, "shared memory");
    pdl_wait();
    const long long per = w.head->per;
    const int n_split = w.head->n_split, redo = w.head->redo, lane = threadIdx.x & 31;
    const auto again = [&](int u) {  // row u & 127 of split tile u >> 7 is left to redo_rows
        return redo && ((w.tiles[w.split[u >> 7]].redo[(u & 127) >> 5] >> (u & 31)) & 1);
    };
    const int grp = threadIdx.x >> 7, c = threadIdx.x & 127;
    bool many = false;
    for (int t = 0; t < n_split; t++) {
        const PagedTile &tl = w.tiles[w.split[t]];
        many |= (int)((tl.start + tl.steps - 1) / per - tl.start / per) + 1 > kFew;
    }
    if (many) {
        for (int u = blockIdx.x; u < n_split * 128; u += gridDim.x) {
            const PagedTile tl = w.tiles[w.split[u >> 7]];
            const int row = u & 127, p0 = (int)(tl.start / per), n = (int)((tl.start + tl.steps - 1) / per) - p0 + 1;
            const int ti = w.tpt > 1 || p.n_h == 128 ? row / p.n_h : 0, h = tl.hc * 128 + row - ti * p.n_h;
            if (n <= kFew || ti >= min(w.tpt, tl.q_len - tl.i0) || h >= p.n_h || (ti > 0 && w.hchunks > 1) || again(u))
                continue;
            __syncthreads();
            if (threadIdx.x < n) wt[threadIdx.x] = w.part_lse[part_row(p0, threadIdx.x, row)];
            __syncthreads();
            float m = -INFINITY, l = 0.f;
            for (int k = 0; k < n; k++) m = wt[k] != wt[k] || m != m ? NAN : fmaxf(m, wt[k]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (m != -INFINITY) {
                for (int k = 0; k < n; k++) l += exp2f(wt[k] - m);
#pragma unroll 8
                for (int k = grp; k < n; k += 4) {
                    const float4 x = __ldg(reinterpret_cast<const float4 *>(w.part_o + part_row(p0, k, row) * kDL) + c);
                    const float f = exp2f(wt[k] - m) / l;
                    acc.x = fmaf(f, x.x, acc.x);
                    acc.y = fmaf(f, x.y, acc.y);
                    acc.z = fmaf(f, x.z, acc.z);
                    acc.w = fmaf(f, x.w, acc.w);
                }
            }
            if (grp) sum[grp - 1][c] = acc;
            __syncthreads();
            if (grp == 0) {
#pragma unroll
                for (int k = 0; k < 3; k++) {
                    acc.x += sum[k][c].x;
                    acc.y += sum[k][c].y;
                    acc.z += sum[k][c].z;
                    acc.w += sum[k][c].w;
                }
                const int tok = tl.q0 + tl.i0 + ti;
                *reinterpret_cast<uint2 *>((__nv_bfloat16 *)p.o + (long long)tok * p.o_ts + (long long)h * p.o_hs + 4 * c) =
                    make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
                if (c == 0) p.lse[(size_t)tok * p.n_h + h] = m == -INFINITY ? m : (m + log2f(l)) * kLn2;
            }
        }
    }
    for (int u = blockIdx.x * 16 + (threadIdx.x >> 5); u < n_split * 128; u += gridDim.x * 16) {
        const PagedTile tl = w.tiles[w.split[u >> 7]];
        const int row = u & 127, p0 = (int)(tl.start / per), n = (int)((tl.start + tl.steps - 1) / per) - p0 + 1;
        const int ti = w.tpt > 1 || p.n_h == 128 ? row / p.n_h : 0, h = tl.hc * 128 + row - ti * p.n_h;
        if (n > kFew || ti >= min(w.tpt, tl.q_len - tl.i0) || h >= p.n_h || (ti > 0 && w.hchunks > 1) || again(u))
            continue;
        const float mine = lane < n ? w.part_lse[part_row(p0, lane, row)] : -INFINITY;
        const bool nan = __any_sync(0xffffffffu, mine != mine);
        float m = mine;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = nan ? NAN : __shfl_sync(0xffffffffu, m, 0);
        float f = m == -INFINITY || lane >= n ? 0.f : exp2f(mine - m), l = f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        l = __shfl_sync(0xffffffffu, l, 0);
        f = l != 0.f ? f / l : 0.f;
        float4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; i++) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int k = 0; k < n; k++) {
            const float g = __shfl_sync(0xffffffffu, f, k);
            const float4 *src = reinterpret_cast<const float4 *>(w.part_o + part_row(p0, k, row) * kDL);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float4 x = __ldg(src + lane + 32 * i);
                acc[i].x = fmaf(g, x.x, acc[i].x);
                acc[i].y = fmaf(g, x.y, acc[i].y);
                acc[i].z = fmaf(g, x.z, acc[i].z);
                acc[i].w = fmaf(g, x.w, acc[i].w);
            }
        }
        const int tok = tl.q0 + tl.i0 + ti;
        uint2 *dst = reinterpret_cast<uint2 *>((__nv_bfloat16 *)p.o + (long long)tok * p.o_ts + (long long)h * p.o_hs);
#pragma unroll
        for (int i = 0; i < 4; i++)
            dst[lane + 32 * i] = make_uint2(pack_bf16x2(acc[i].x, acc[i].y), pack_bf16x2(acc[i].z, acc[i].w));
        if (lane == 0) p.lse[(size_t)tok * p.n_h + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    if (redo) redo_rows<KIND>(p, w, reinterpret_cast<uint8_t *>(sum));
}

template <int KIND>
cudaError_t launch_t(const CUtensorMap &m4, const CUtensorMap &m1, const CUtensorMap &mq, const Paged &p,
                     const PagedPlan &w, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_paged_tc<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    count_launch();
    e = launch_pdl(k_paged_tc<KIND>, dim3(2 * kPairs), dim3(threads_of(KIND)), kSmem, st, m4, m1, mq, p, w);
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_pdl(k_paged_join<KIND>, dim3(296), dim3(512), 0, st, p, w);
}

}  // namespace

cudaError_t launch_paged_tc(const Paged &p, const PagedPlan &w, cudaStream_t st) {
    // 64 columns, slots, slices of 64 columns
    CUtensorMap m4{}, m1{};
    const uint64_t dims[3] = {64, (uint64_t)p.n_pages * p.page_size, 9}, strides[2] = {(kDL + kDR) * 2, 128};
    const uint32_t b4[3] = {64, 8, 4}, b1[3] = {64, 8, 1};
    if (p.kind == DSPARK_CACHE_BF16 &&
        (!make_map_nd(&m4, p.cache, 3, dims, strides, b4) || !make_map_nd(&m1, p.cache, 3, dims, strides, b1)))
        return cudaErrorInvalidValue;
    CUtensorMap mq{};
    if (!make_q_map(&mq, p, w)) return cudaErrorInvalidValue;
    return p.kind == DSPARK_CACHE_BF16 ? launch_t<DSPARK_CACHE_BF16>(m4, m1, mq, p, w, st)
                                       : launch_t<DSPARK_CACHE_FP8>(m4, m1, mq, p, w, st);
}

}  // namespace dspark
