// Tensor-core (tcgen05 / TMEM / TMA) forward of the latent draft attention:
// bf16, 512-wide latents, 64-wide rope keys, windows of at most 128.
//
// A block's 5 offsets and all its heads see the same keys, at most 127 context
// positions and 5 draft keys: S = Q K^T of 128 query rows over all of them is
// one accumulator of 144 columns, so the softmax is done in one go, without a
// running maximum, and the keys are loaded once per block and stay in shared
// memory, as keys and as values (K-major and MN-major reads of the same bytes).
// Work item: a kept block (or some of its head tiles, when there are few
// blocks); tile: up to 22 heads x 5 rows of it.
//
// What bounds it is the stream of Q in (1152 B a row) and O out (1024 B a row):
// at S = 8192, N = 512, B = 2 they are 0.71 GB of the 0.74 GB that have to move,
// 113 us at the measured copy rate, against 58 us of tensor work; measured 207 us with
// inputs that change from call to call, 177 with the same ones (S = 2048, N = 128, B = 1:
// 35.5, of which 32 are one round of 2 or 3 tiles). So Q comes
// in 64-column slices through a ring of three, feeding S = Q K^T slice by
// slice, and O leaves in eight 64-column products P V through two accumulators;
// S is double-buffered, so the loads of one tile go on while the tile before it
// is in its softmax and its stores.
//
// RoPE: the turned slices of queries and keys are split as hi + lo of two bf16
// each and their product formed as hi hi + lo hi + hi lo, which keeps the scores
// and the fp32 LSE to 2^-16 (one bf16 each would leave 2^-8 of the rope part). P is
// rounded once to bf16 as an operand: 2^-8 of each weight, as of the rounded O.
//
// TMEM: S 0..143 / 144..287 (P, bf16, over its own S columns), rope query hi, lo
// 288..351, O 352..415 / 416..479.
// Warps: 0-3 and 4-7 softmax and output of even and odd tiles (thread = row);
// 8-11 turn the query's rope slice, global -> TMEM; 12 loads Q slices, 13 loads
// keys, 14 issues the products of S, 15 those of O (one thread each).
// Keys of a block: context slot i is position A - W + 1 + i (before the
// sequence's start: zero fill by TMA), then, at the next multiple of 32, the 5
// draft keys; no other row of memory is ever read into a slot, the slots
// between stay zero, so nothing outside the mask can reach a result.
// Every wait is bounded: on time-out the CTA raises its abort flag, all roles
// leave, loads and MMAs in flight are waited for (bounded), TMEM is freed and
// the error word gets kErrTimeout.
#include <algorithm>

#include "dspark_latent_tc.cuh"

namespace dspark {

namespace {

using namespace tc;

constexpr int kDL = 512, kDR = 64, kDK = kDL + kDR;
constexpr int kSlices = kDL / 64;
constexpr int kKeys = 144;                 // key slots: up to 128 context, 16 for the draft keys
constexpr int kKSlice = kKeys * 128;       // one 64-column slice of the keys
constexpr int kKSlices = kSlices + 2;      // the latent's, rope hi, rope lo
constexpr int kHeads = 22;                 // heads per tile at most: 110 rows, so that three Q slices fit
constexpr int kQSlot = 14 * 1024, kQSlots = 3;
constexpr int oQ = kKSlices * kKSlice;
constexpr int oBar = oQ + kQSlots * kQSlot;
// an MMA reads 128 rows from a Q slot: the last one's read ends inside the allocation
constexpr int kSmem = oQ + (kQSlots - 1) * kQSlot + 128 * 128 + 1024;
static_assert(kHeads * kBlock * 128 <= kQSlot && oBar + 512 + 1024 <= kSmem && kSmem <= 232448, "shared memory");
static_assert(kKSlice % 1024 == 0 && kQSlot % 1024 == 0, "swizzle atoms");

constexpr uint32_t kColS = 0, kColR = 2 * kKeys, kColO = kColR + 64;
constexpr int kWarpR = 8, kWarpQ = 12, kWarpK = 13, kWarpM = 14;
constexpr int kThreads = 16 * 32;
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
    int n_h, S, N, W, R, B;
    int ctxpad;          // key slots of the context: W - 1 rounded up to 32
    int hp;              // heads per tile
    int nsplit, tiles, per, n_work;
    float scale_log2;
    const __nv_bfloat16 *q;
    const int32_t *cnt, *sorted_n, *sorted_a;
    const float2 *tab;
    __nv_bfloat16 *o;
    float *lse;
    uint32_t *err;
    uint64_t wait_ns;
    bool wide;  // o is 32-byte aligned
};

__global__ void __launch_bounds__(kThreads, 1)
    k_lat_fwd_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c,
                 const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_l,
                 const __grid_constant__ CUtensorMap tm_c5, const __grid_constant__ CUtensorMap tm_h5,
                 const __grid_constant__ CUtensorMap tm_l5, const Args p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *kfull = reinterpret_cast<uint64_t *>(sm + oBar), *kempty = kfull + kKSlices;
    uint64_t *qfull = kempty + kKSlices, *qempty = qfull + kQSlots;
    uint64_t *sfull = qempty + kQSlots, *pready = sfull + 2, *ofull = pready + 2, *ofree = ofull + 4;
    uint64_t *pvdone = ofree + 2, *rready = pvdone + 2, *rfree = rready + 1, *drain = rready + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(drain + 3);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t wlim = p.wait_ns;

    for (int e = threadIdx.x; e < oQ / 16; e += kThreads) reinterpret_cast<uint4 *>(sm)[e] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kKSlices; i++) mbar_init(&kfull[i], 1);
        for (int i = 0; i < 2 * kQSlots; i++) mbar_init(&qfull[i], 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pready[i], 4);
            mbar_init(&ofull[i], 1);  // of even tiles; 2, 3 of odd ones, whose reader is the other warps
            mbar_init(&ofull[2 + i], 1);
            mbar_init(&ofree[i], 4);
        }
        mbar_init(rready, 4);
        mbar_init(rfree, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&pvdone[i], 1);
            mbar_init(&drain[i], 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kWarpM) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    pdl_wait();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    DraftCursor cur{p.cnt, p.sorted_n, p.sorted_a, p.B, p.N, p.nsplit, p.tiles, p.per};
    DraftItem it;
    const int G = gridDim.x;
    uint32_t issued_q = 0, issued_k[2] = {0, 0};  // the loaders' copies: Q slices; items in full, slices of the next

    if (warp == kWarpQ) {
        // ------------------------------------------------------ Q slices
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            uint32_t &g = issued_q;
            bool ok = true;
            for (int w = blockIdx.x; ok && w < p.n_work && cur.at(w, it); w += G)
                for (int t = it.t0; ok && t < it.t1; t++)
                    for (int c = 0; c < kSlices; c++, g++) {
                        const uint32_t s = g % kQSlots;
                        if (g >= kQSlots && !mbar_wait(&qempty[s], (g / kQSlots - 1) & 1, abort_flag, wlim)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&qfull[s], p.hp * kBlock * 128);
                        tma_load_4d(sm + oQ + s * kQSlot, &tm_q, &qfull[s], 64 * c, kBlock * it.n, t * p.hp, it.b);
                    }
        }
    } else if (warp == kWarpK) {
        // ------------------------------------------------------ keys
        if (lane == 0) {
            const uint32_t bytes = (p.W - 1 + kBlock) * 128;
            uint32_t &k = issued_k[0];
            bool ok = true;
            for (int w = blockIdx.x; ok && w < p.n_work && cur.at(w, it); w += G) {
                for (int c = 0; c < kKSlices; c++) {
                    if (k && !mbar_wait(&kempty[c], (k - 1) & 1, abort_flag, wlim)) {
                        ok = false;
                        break;
                    }
                    uint8_t *dst = sm + c * kKSlice;
                    const CUtensorMap *m = c < kSlices ? &tm_c : c == kSlices ? &tm_h : &tm_l;
                    const CUtensorMap *m5 = c < kSlices ? &tm_c5 : c == kSlices ? &tm_h5 : &tm_l5;
                    const int x = c < kSlices ? 64 * c : 0;
                    mbar_arrive_expect_tx(&kfull[c], bytes);
                    if (p.W > 1) tma_load_3d(dst, m, &kfull[c], x, it.a - (p.W - 1), it.b);
                    tma_load_3d(dst + p.ctxpad * 128, m5, &kfull[c], x, p.S + kBlock * it.n, it.b);
                    issued_k[1]++;
                }
                if (ok) {
                    k++;
                    issued_k[1] = 0;
                }
            }
        }
    } else if (warp == kWarpM) {
        // ------------------------------------------------- S = Q K^T
        if (lane == 0) {
            const uint32_t idS = idesc_bf16(128, p.ctxpad + 16, 0);
            uint32_t i = 0, g = 0, k = 0;  // tiles, slices, items
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = ok && mbar_wait(bar, parity, abort_flag, wlim); };
            for (int w = blockIdx.x; ok && w < p.n_work && cur.at(w, it); w += G, k++)
                for (int t = it.t0; ok && t < it.t1; t++, i++) {
                    if (i >= 2 && !wait(&pvdone[i & 1], ((i >> 1) - 1) & 1)) break;
                    const uint32_t dS = tmem + kColS + (i & 1) * kKeys;
#pragma unroll 1
                    for (int c = 0; c < kSlices; c++, g++) {
                        const uint32_t s = g % kQSlots;
                        if ((t == it.t0 && !wait(&kfull[c], k & 1)) || !wait(&qfull[s], (g / kQSlots) & 1)) break;
                        tc_fence_after();
                        const SDesc qd = sdesc_split(sdesc_sw128(smem_u32(sm + oQ + s * kQSlot), 16, 1024));
                        const SDesc kd = sdesc_split(sdesc_sw128(smem_u32(sm + c * kKSlice), 16, 1024));
#pragma unroll
                        for (int u = 0; u < 4; u++)
                            mma_bf16_ss(dS, qd.at(2 * u), kd.at(2 * u), idS, (c | u) != 0 ? 1u : 0u);
                        mma_commit(&qempty[s]);
                    }
                    if (t == it.t0 && (!wait(&kfull[kSlices], k & 1) || !wait(&kfull[kSlices + 1], k & 1))) break;
                    if (!wait(rready, i & 1)) break;
                    tc_fence_after();
                    const SDesc hd = sdesc_split(sdesc_sw128(smem_u32(sm + kSlices * kKSlice), 16, 1024));
                    const SDesc ld = sdesc_split(sdesc_sw128(smem_u32(sm + (kSlices + 1) * kKSlice), 16, 1024));
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        mma_bf16_ts(dS, tmem + kColR + 8 * u, hd.at(2 * u), idS, 1u);
                        mma_bf16_ts(dS, tmem + kColR + 32 + 8 * u, hd.at(2 * u), idS, 1u);
                        mma_bf16_ts(dS, tmem + kColR + 8 * u, ld.at(2 * u), idS, 1u);
                    }
                    mma_commit(rfree);
                    if (t + 1 == it.t1) {
                        mma_commit(&kempty[kSlices]);
                        mma_commit(&kempty[kSlices + 1]);
                    }
                    mma_commit(&sfull[i & 1]);  // (last: nothing is in flight once its reader has it)
                }
        }
    } else if (warp == kWarpM + 1) {
        // ------------------------------------------------- O = P V
        // (an issuer of its own: one thread issuing both was the bound, at twice
        // the time of the products)
        if (lane == 0) {
            const uint32_t idO = idesc_bf16(128, 64, 1);
            const int ksteps = p.ctxpad / 16 + 1;
            uint32_t j = 0, g = 0;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = ok && mbar_wait(bar, parity, abort_flag, wlim); };
            for (int w = blockIdx.x; ok && w < p.n_work && cur.at(w, it); w += G)
                for (int t = it.t0; ok && t < it.t1; t++, j++) {
                    if (!wait(&pready[j & 1], (j >> 1) & 1)) break;
                    const uint32_t pa = tmem + kColS + (j & 1) * kKeys;
#pragma unroll 1
                    for (int d = 0; d < kSlices; d++, g++) {
                        const uint32_t s = g & 1, dO = tmem + kColO + 64 * s;
                        if (g >= 2 && !wait(&ofree[s], ((g >> 1) - 1) & 1)) break;
                        tc_fence_after();
                        const SDesc vd = sdesc_split(sdesc_sw128(smem_u32(sm + d * kKSlice), kKSlice, 1024));
                        // (unrolled: a product of 64 columns takes 50 cycles, a step of a rolled loop 90)
#pragma unroll
                        for (int u = 0; u < kKeys / 16; u++)
                            if (u < ksteps) mma_bf16_ts(dO, pa + 8 * u, vd.at(128 * u), idO, u > 0 ? 1u : 0u);
                        if (t + 1 == it.t1) mma_commit(&kempty[d]);
                        if (d == kSlices - 1) mma_commit(&pvdone[j & 1]);
                        mma_commit(&ofull[2 * (j & 1) + s]);  // (last)
                    }
                }
        }
    } else if (warp >= kWarpR) {
        // ------------------------------- rope slice of the queries -> TMEM
        const int r = (warp - kWarpR) * 32 + lane, j = r % kBlock, hl = r / kBlock;
        const uint32_t trow = tmem + ((uint32_t)((warp - kWarpR) * 32) << 16) + kColR;
        uint32_t i = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < p.n_work && cur.at(w, it); w += G)
            for (int t = it.t0; ok && t < it.t1; t++, i++) {
                const int h = t * p.hp + hl;
                const bool live = hl < p.hp && h < p.n_h;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    p.q + (((size_t)it.b * p.n_h + (live ? h : 0)) * p.R + (size_t)kBlock * it.n + j) * kDK + kDL);
                const float4 *tab = reinterpret_cast<const float4 *>(p.tab + (size_t)(it.a + j) * (kDR / 2));
                uint32_t x[32];
#pragma unroll
                for (int u = 0; u < 8; u++) {
                    const uint4 v = live ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
                    x[4 * u] = v.x;
                    x[4 * u + 1] = v.y;
                    x[4 * u + 2] = v.z;
                    x[4 * u + 3] = v.w;
                }
                uint32_t lo[32];
#pragma unroll
                for (int u = 0; u < 16; u++) {
                    const float4 cs = __ldg(tab + u);  // (cos, sin) of pairs 2 u, 2 u + 1
                    const uint32_t w0 = x[2 * u], w1 = x[2 * u + 1];
                    const float a0 = __uint_as_float(w0 << 16), a1 = __uint_as_float(w0 & 0xffff0000u);
                    const float b0 = __uint_as_float(w1 << 16), b1 = __uint_as_float(w1 & 0xffff0000u);
                    split_bf16x2(a0 * cs.x - a1 * cs.y, a0 * cs.y + a1 * cs.x, x[2 * u], lo[2 * u]);
                    split_bf16x2(b0 * cs.z - b1 * cs.w, b0 * cs.w + b1 * cs.z, x[2 * u + 1], lo[2 * u + 1]);
                }
                if (i > 0) ok = warp_all(mbar_wait(rfree, (i - 1) & 1, abort_flag, wlim));
                if (!ok) break;
                tc_fence_after();
                tmem_st32u(trow, x);
                tmem_st32u(trow + 32, lo);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(rready);
            }
    } else {
        // ------------------------------------------- softmax and output
        const int wg = warp >> 2, q4 = warp & 3, r = q4 * 32 + lane, j = r % kBlock, hl = r / kBlock;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t tS = trow + kColS + wg * kKeys;
        uint32_t i = 0;
        bool ok = true;
        for (int w = blockIdx.x; ok && w < p.n_work && cur.at(w, it); w += G)
            for (int t = it.t0; ok && t < it.t1; t++, i++) {
                if ((int)(i & 1) != wg) continue;
                ok = warp_all(mbar_wait(&sfull[wg], (i >> 1) & 1, abort_flag, wlim));
                if (!ok) break;
                tc_fence_after();
                // the block's keys: context slots [lo, W - 1), draft slots 0 .. 4
                const int lo = max(0, p.W - 1 - it.a), hi = p.W - 1;
                // (chunks of 32 slots that are visible throughout take no tests)
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                for (int c = 0; c < p.ctxpad; c += 32) {
                    float s[32];
                    tmem_ld32(tS + c, s);
                    tmem_wait_ld();
                    if (c >= lo && c + 32 <= hi) {
#pragma unroll
                        for (int k = 0; k < 32; k++) m[k & 3] = fmaxf(m[k & 3], s[k]);
                    } else {
                        const uint32_t in = slot_mask(lo - c, hi - c);
#pragma unroll
                        for (int k = 0; k < 32; k++) m[k & 3] = fmaxf(m[k & 3], (in >> k) & 1 ? s[k] : -INFINITY);
                    }
                }
                float sd[8];
                tmem_ld8(tS + p.ctxpad, sd);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < kBlock; k++) m[k & 3] = fmaxf(m[k & 3], sd[k]);
                const float mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * p.scale_log2;
                const float neg = mx == -INFINITY ? 0.f : -mx;
                float l[4] = {0.f, 0.f, 0.f, 0.f};
                // P, bf16, over the S columns already read (two to a column)
                for (int c = 0; c < p.ctxpad; c += 32) {
                    float s[32];
                    tmem_ld32(tS + c, s);
                    tmem_wait_ld();
                    if (!(c >= lo && c + 32 <= hi)) {
                        const uint32_t in = slot_mask(lo - c, hi - c);
#pragma unroll
                        for (int k = 0; k < 32; k++) s[k] = (in >> k) & 1 ? s[k] : -INFINITY;
                    }
                    uint32_t pw[16];
#pragma unroll
                    for (int k = 0; k < 32; k++) {
                        s[k] = ex2(fmaf(s[k], p.scale_log2, neg));
                        l[k & 3] += s[k];
                    }
#pragma unroll
                    for (int k = 0; k < 16; k++) pw[k] = pack_bf16x2(s[2 * k], s[2 * k + 1]);
                    tmem_st16u(tS + c / 2, pw);
                }
                uint32_t pd[8];
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    sd[k] = k < kBlock ? ex2(fmaf(sd[k], p.scale_log2, neg)) : 0.f;
                    l[k & 3] += sd[k];
                }
#pragma unroll
                for (int k = 0; k < 8; k++) pd[k] = k < 4 ? pack_bf16x2(sd[(2 * k) & 7], sd[(2 * k + 1) & 7]) : 0u;
                tmem_st8u(tS + p.ctxpad / 2, pd);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pready[wg]);
                const float ls = (l[0] + l[1]) + (l[2] + l[3]);
                const float inv = ls > 0.f ? 1.f / ls : 0.f;
                const int h = t * p.hp + hl;
                const bool live = hl < p.hp && h < p.n_h;
                const size_t row = ((size_t)it.b * p.n_h + (live ? h : 0)) * p.R + (size_t)kBlock * it.n + j;
                if (live) p.lse[row] = (mx + log2f(ls)) * kLn2;
                uint8_t *dst = reinterpret_cast<uint8_t *>(p.o + row * kDL);
#pragma unroll 1
                for (int c = 0; c < kSlices; c++) {
                    const uint32_t g = i * kSlices + c, s = g & 1;
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
                    if (live) {
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            uint32_t x[8];
#pragma unroll
                            for (int k = 0; k < 8; k++)
                                x[k] = u < 2 ? pack_bf16x2(v0[16 * (u & 1) + 2 * k] * inv, v0[16 * (u & 1) + 2 * k + 1] * inv)
                                             : pack_bf16x2(v1[16 * (u & 1) + 2 * k] * inv, v1[16 * (u & 1) + 2 * k + 1] * inv);
                            st_global_32B(dst + 128 * c + 32 * u, x, p.wide);
                        }
                    }
                }
            }
    }

    // ---------------------------------------------------------- teardown
    __syncthreads();
    if (*abort_flag && lane == 0) {
        // what is in flight lands before shared and tensor memory go away; each wait is bounded on its own
        volatile int never = 0;
        if (warp == kWarpQ)
            for (uint32_t g = issued_q > kQSlots ? issued_q - kQSlots : 0; g < issued_q; g++)
                mbar_wait(&qfull[g % kQSlots], (g / kQSlots) & 1, &never);
        if (warp == kWarpK)
            for (uint32_t c = 0; c < kKSlices; c++) {
                const uint32_t n = issued_k[0] + (c < issued_k[1] ? 1u : 0u);
                if (n) mbar_wait(&kfull[c], (n - 1) & 1, &never);
            }
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

}  // namespace

bool lat_tc_supported(const Prob &p) {
    return p.dtype == DSPARK_BF16 && p.d_c == kDL && p.d_r == kDR && p.W <= 128;
}

cudaError_t launch_lat_fwd_tc(const Prob &p, const void *q, const void *c, void *o, float *lse, const LatWs &ws,
                              cudaStream_t st) {
    // (padding blocks' rows are written by the preparation)
    if (p.B == 0 || p.N == 0) return cudaSuccess;
    int dev = 0, nsm = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    Args a{};
    a.n_h = p.n_h; a.S = p.S; a.N = p.N; a.W = p.W; a.R = p.R; a.B = p.B;
    a.ctxpad = (p.W - 1 + 31) / 32 * 32;
    a.tiles = (p.n_h + kHeads - 1) / kHeads;
    a.hp = (p.n_h + a.tiles - 1) / a.tiles;
    // few blocks: their tiles spread over the SMs
    const long long blocks = (long long)p.B * p.N;
    a.nsplit = (int)std::max<long long>(1, std::min<long long>(a.tiles, nsm / blocks));
    a.per = (a.tiles + a.nsplit - 1) / a.nsplit;
    a.nsplit = (a.tiles + a.per - 1) / a.per;
    if (blocks * a.nsplit >= (1ll << 31) - 4096) return cudaErrorInvalidValue;
    a.n_work = (int)(blocks * a.nsplit);
    a.scale_log2 = p.scale_log2;
    a.q = (const __nv_bfloat16 *)q;
    a.cnt = ws.base.cnt;
    a.sorted_n = ws.base.sorted_n;
    a.sorted_a = ws.base.sorted_a;
    a.tab = ws.base.rope;
    a.o = (__nv_bfloat16 *)o;
    a.lse = lse;
    a.err = ws.base.err;
    a.wait_ns = p.wait_ns;
    a.wide = ((uintptr_t)o & 31) == 0;
    CUtensorMap mq, mc, mh, ml, mc5, mh5, ml5;
    const uint64_t L = p.L, B = p.B;
    const uint64_t qd[4] = {kDK, (uint64_t)p.R, (uint64_t)p.n_h, B};
    const uint64_t qs[3] = {kDK * 2, (uint64_t)p.R * kDK * 2, (uint64_t)p.n_h * p.R * kDK * 2};
    const uint32_t qb[4] = {64, kBlock, (uint32_t)a.hp, 1};
    const uint64_t cd[3] = {kDL, L, B}, cs[2] = {kDL * 2, L * kDL * 2};
    const uint64_t rd[3] = {kDR, L, B}, rs[2] = {kDR * 2, L * kDR * 2};
    const uint32_t wb[3] = {64, (uint32_t)std::max(p.W - 1, 1), 1}, db[3] = {64, kBlock, 1};
    if (!make_map_nd(&mq, q, 4, qd, qs, qb) || !make_map_nd(&mc, c, 3, cd, cs, wb) ||
        !make_map_nd(&mh, ws.kr_hi, 3, rd, rs, wb) || !make_map_nd(&ml, ws.kr_lo, 3, rd, rs, wb) ||
        !make_map_nd(&mc5, c, 3, cd, cs, db) || !make_map_nd(&mh5, ws.kr_hi, 3, rd, rs, db) ||
        !make_map_nd(&ml5, ws.kr_lo, 3, rd, rs, db))
        return cudaErrorInvalidValue;
    e = cudaFuncSetAttribute(k_lat_fwd_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_pdl(k_lat_fwd_tc, dim3(std::min(a.n_work, nsm)), dim3(kThreads), kSmem, st, mq, mc, mh, ml, mc5, mh5,
                      ml5, a);
}

}  // namespace dspark
