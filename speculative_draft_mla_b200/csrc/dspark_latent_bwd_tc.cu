// Tensor-core (tcgen05 / TMEM / TMA) backward of the latent draft attention:
// bf16, 512-wide latents, 64-wide rope keys, windows of at most 128.
//
// Tile: up to 22 heads x 5 rows of one kept block, whose rows all see the same
// keys (up to 127 context and 5 draft). Recomputed: S = Q K^T and dP = dO C^T
// over all of them, P = exp(S - LSE), D = sum_k P dP (the row is whole, so the
// forward's O is not needed), dS = scale P (dP - D). Then per 64 columns c:
//   dq_c = dS K_c                       rows x columns
//   dk_c = dS^T Q_c + P^T dO_c          context keys x columns
//   dd_c = Q_c^T dS_d, dO_c^T P_d       columns x draft keys (one product: the two
//                                       column sets are its 128 rows, the two key
//                                       sets its 32 columns)
// P and dS go through shared memory, where rows-by-keys tiles are read transposed
// (dS^T Q), and dS, for dS K, to tensor memory besides. Key gradients of all heads and of the blocks
// whose windows overlap meet in an fp32 accumulator [B, L, 576] by
// reductions; the last launch turns its rope part back and rounds.
//
// The 132 x 576 fp32 key gradients of a block (304 KB) fit neither tensor
// memory nor shared memory beside the keys, so a tile's share leaves the SM as
// it is formed, and keys, Q and dO come in 64-column slices through two rings,
// twice per tile: for S and dP, and, from L2, for the gradients. (Gradients of a
// tile interleaved with S and dP of the next share the keys' slices, but need
// two slots of Q and dO a slice, and with the three that fit the copies' latency
// is exposed: 4500 cycles a slice against 2700.)
//
// What bounds it (S = 4096, N = 512, B = 4, a tenth padding: 1090 - 1115 us with its
// preparation where inputs change from call to call, 1010 - 1080 with the same ones, as
// in the comparisons below; 42000 cycles a tile): the gradients, 26000, whose 30 short products a
// slice take 1500 cycles by their shared-memory operands beside 1100 of copies in
// and results out; S and dP, 15000, by the latency of copies that three slots
// hide in part; the softmax between, 4400. DRAM moves little more than it must
// (1.53 GB read, 0.74 GB written; L2 serves the second reads).
//
// Sums of key gradients are fp32 in whatever order the tiles finish: two runs
// may differ in the last bits before the rounding to bf16. P and dS are bf16
// operands (an error of half a step each, as of the rounded results). The turned
// rope slices of Q and K are hi + lo of two bf16 in S, as in the forward, and Q's
// in its product with dS: one bf16 would nearly double the error of dkr. The rope
// part of dq is formed with the keys' hi alone, one rounding more than its latent part.
//
// TMEM: S 0..143 (then dS, bf16), dP 144..287, dq 288..351, dk 352..415 / 416..479, dd 480..511.
// Warps 0-7 softmax (warps w and w + 4 share 32 rows, 64 context keys each);
// 0-3 then take dq and dd, 4-7 dk; 8 loads keys, 9 Q and dO, 10 - 12 issue the
// MMAs (as whole warps: 1010 us, one lane of each 1084), 13 stores dq. Every wait
// is bounded.
#include <algorithm>

#include "dspark_latent_tc.cuh"

namespace dspark {

namespace {

using namespace tc;

constexpr int kDL = 512, kDR = 64, kDK = kDL + kDR;
constexpr int kSlices = 9;
constexpr int kKeys = 144, kKSlot = kKeys * 128, kKSlots = 2;
constexpr int kHeads = 22, kRows = 112;            // rows of a tile, padded to the K steps of 16
// Q and dO slices of the same columns; last, hi and lo of Q's rope slice
constexpr int kSlot = kRows * 128, kPair = 2 * kSlot, kPairs2 = 3;
constexpr int oK = 0, oPair = kKSlots * kKSlot;
constexpr int oDS = oPair + kPairs2 * kPair;       // dS, context keys: two slices of 64 keys
constexpr int oPr = oDS + 2 * kSlot;               // P
constexpr int oDD = oPr + 2 * kSlot;               // draft keys: [2 x 64 rows][16 dS, 16 P][128 B]
constexpr int oT = oDD + 2 * 32 * 128;             // 4 KB of each reducing warp: 32 rows x 32 columns of dk
constexpr int oO = oT + 4 * 4096;                  // dq on its way out: rows x 64 columns
constexpr int oX = oO + kSlot;                     // D halves [2][128]
constexpr int oBar = oX + 1024;
constexpr int kSmem = oBar + 512 + 1024;
static_assert(kHeads * kBlock <= kRows && kSmem <= 232448, "shared memory");
static_assert(kSlot % 1024 == 0 && oDD % 1024 == 0 && oT % 1024 == 0, "swizzle atoms");
constexpr uint32_t kColS = 0, kColP = kKeys, kColC = 2 * kKeys, kColD = kColC + 3 * 64;
constexpr int kWarpK = 8, kWarpQ = 9, kWarpM = 10, kWarpO = 13, kThreads = 14 * 32;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    int n_h, S, N, W, R, B, L;
    int ctxpad, hp, nsplit, tiles, per, n_work;
    float scale, scale_log2;
    const int32_t *cnt, *sorted_n, *sorted_a;
    const float2 *tab;
    const float *lse;
    float *dacc;
    uint32_t *err;
    uint64_t wait_ns;
};

__device__ __forceinline__ void red4(float *a, float x, float y, float z, float w) {
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
// A box of shared memory added to fp32 rows.
__device__ __forceinline__ void tma_red_3d(const CUtensorMap *m, const void *src, int x, int y, int z) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     (uint64_t)m),
                 "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void red1(float *a, float x) {
    asm volatile("red.global.add.f32 [%0], %1;" ::"l"(a), "f"(x) : "memory");
}
// The CTA's tiles in order, over its items: blocks are dealt out in turn, so that
// the accumulators of the keys at work at one time are a few MB (with a run of
// neighbouring blocks to a CTA they are all of them, and thrash L2 beside the
// stream of Q, dO and dq: 1220 us against 1020 at S = 4096, N = 512, B = 4).
struct Tile {
    int b, n, a, h0, nh;
};
struct TileCursor {
    DraftCursor cur;
    DraftItem it;
    int w, t;
    bool open;
    __device__ __forceinline__ TileCursor(const Args &p)
        : cur{p.cnt, p.sorted_n, p.sorted_a, p.B, p.N, p.nsplit, p.tiles, p.per}, w(blockIdx.x), t(0), open(false) {}
    __device__ __forceinline__ bool next(const Args &p, Tile &o) {
        if (!open) {
            if (w >= p.n_work || !cur.at(w, it)) return false;
            t = it.t0;
            open = true;
        }
        o.b = it.b;
        o.n = it.n;
        o.a = it.a;
        o.h0 = t * p.hp;
        o.nh = min(p.hp, p.n_h - o.h0);
        if (++t == it.t1) {
            open = false;
            w += gridDim.x;
        }
        return true;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    k_lat_bwd_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_g,
                 const __grid_constant__ CUtensorMap tm_qr, const __grid_constant__ CUtensorMap tm_c,
                 const __grid_constant__ CUtensorMap tm_h, const __grid_constant__ CUtensorMap tm_l,
                 const __grid_constant__ CUtensorMap tm_c5, const __grid_constant__ CUtensorMap tm_h5,
                 const __grid_constant__ CUtensorMap tm_l5, const __grid_constant__ CUtensorMap tm_dq,
                 const __grid_constant__ CUtensorMap tm_acc, const Args p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    // a slot's full barriers: [0] of copies for the gradients, [1] of those for the scores
    uint64_t *kfull = reinterpret_cast<uint64_t *>(sm + oBar), *kempty = kfull + 2 * kKSlots;
    uint64_t *qfull = kempty + kKSlots, *qempty = qfull + 2 * kPairs2;
    uint64_t *sfull = qempty + kPairs2, *pds = sfull + 1, *drain = sfull + 2;
    uint64_t *qcfull = sfull + 5, *qcfree = qcfull + 1, *kcfull = qcfull + 2, *kcfree = kcfull + 2;
    uint64_t *dfull = kcfree + 2, *dfree = dfull + 1, *done = dfull + 2, *lbar = done + 2;
    uint64_t *ofull = lbar + 4, *ofree = ofull + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ofree + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ofree + 2);
    float *xd = reinterpret_cast<float *>(sm + oX);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t wlim = p.wait_ns;

    // slots of keys and rows that no copy ever writes, and P, dS, stay or start zero
    for (int e = threadIdx.x; e < oX / 16; e += kThreads) reinterpret_cast<uint4 *>(sm)[e] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKSlots; i++) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kfull[kKSlots + i], 1);
            mbar_init(&kempty[i], 1);
        }
        for (int i = 0; i < 3 * kPairs2; i++) mbar_init(&qfull[i], 1);
        mbar_init(sfull, 1);
        mbar_init(pds, 8);
        for (int i = 0; i < 3; i++) mbar_init(&drain[i], 1);
        mbar_init(qcfull, 1);  // dq's buffer
        mbar_init(qcfree, 4);
        for (int i = 0; i < 2; i++) {
            mbar_init(&kcfull[i], 1);  // dk's two
            mbar_init(&kcfree[i], 4);
            mbar_init(&done[i], 1);  // the gradients of a tile
        }
        mbar_init(ofull, 4);
        mbar_init(ofree, 1);
        mbar_init(dfull, 1);
        mbar_init(dfree, 4);
        for (int i = 0; i < 4; i++) mbar_init(&lbar[i], 2);
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
    // the loaders' copies; by kind, the slots' next phases and whether a slot was used
    uint32_t n_issued = 0, n_phase[2] = {0, 0}, n_used[2] = {0, 0};

    // Per tile the slices for S and dP, then those for the gradients.
    if (warp == kWarpK) {
        // -------------------------------------------------------- keys
        if (lane == 0) {
            TileCursor cu(p);
            Tile cur;
            const uint32_t bytes = (p.W - 1 + kBlock) * 128;
            bool ok = true;
            auto load = [&](const Tile &t, int c, int kind) {
                const uint32_t s = n_issued % kKSlots;
                uint64_t *full = &kfull[kind * kKSlots + s];
                if (n_issued >= kKSlots && !mbar_wait(&kempty[s], (n_issued / kKSlots - 1) & 1, abort_flag, wlim))
                    return false;
                uint8_t *dst = sm + oK + s * kKSlot;
                const int x = c < 8 ? 64 * c : 0;
                mbar_arrive_expect_tx(full, bytes);
                if (p.W > 1) tma_load_3d(dst, c < 8 ? &tm_c : c == 8 ? &tm_h : &tm_l, full, x, t.a - (p.W - 1), t.b);
                tma_load_3d(dst + p.ctxpad * 128, c < 8 ? &tm_c5 : c == 8 ? &tm_h5 : &tm_l5, full, x,
                            p.S + kBlock * t.n, t.b);
                n_issued++;
                n_phase[kind] ^= 1u << s;
                n_used[kind] |= 1u << s;
                return true;
            };
            while (ok && cu.next(p, cur)) {
                for (int c = 0; ok && c <= kSlices; c++) ok = load(cur, c, 1);  // (9: the rope keys' lo)
                for (int c = 0; ok && c < kSlices; c++) ok = load(cur, c, 0);
            }
        }
    } else if (warp == kWarpQ) {
        // ---------------------------------------------------- Q and dO
        if (lane == 0) {
            TileCursor cu(p);
            Tile cur;
            bool ok = true;
            const uint32_t bytes = p.hp * kBlock * 128;
            auto load = [&](const Tile &t, int c, int kind) {
                const uint32_t s = n_issued % kPairs2;
                uint64_t *full = &qfull[kind * kPairs2 + s];
                if (n_issued >= kPairs2 && !mbar_wait(&qempty[s], (n_issued / kPairs2 - 1) & 1, abort_flag, wlim))
                    return false;
                uint8_t *dst = sm + oPair + s * kPair;
                mbar_arrive_expect_tx(full, 2 * bytes);
                if (c < 8) {
                    tma_load_4d(dst, &tm_q, full, 64 * c, kBlock * t.n, t.h0, t.b);
                    tma_load_4d(dst + kSlot, &tm_g, full, 64 * c, kBlock * t.n, t.h0, t.b);
                } else {
                    tma_load_4d(dst, &tm_qr, full, 0, kBlock * t.n, t.h0, t.b);
                    tma_load_4d(dst + kSlot, &tm_qr, full, 64, kBlock * t.n, t.h0, t.b);
                }
                n_issued++;
                n_phase[kind] ^= 1u << s;
                n_used[kind] |= 1u << s;
                return true;
            };
            while (ok && cu.next(p, cur))
                for (int kind = 1; kind >= 0; kind--)
                    for (int c = 0; ok && c < kSlices; c++) ok = load(cur, c, kind);
        }
    } else if (warp == kWarpO) {
        // ---------------------------------------------------- dq -> memory
        if (lane == 0) {
            TileCursor cu(p);
            Tile cur;
            uint32_t i = 0;
            bool ok = true;
            while (ok && cu.next(p, cur))
                for (int c = 0; c < kSlices; c++, i++) {
                    if (!(ok = mbar_wait(ofull, i & 1, abort_flag, wlim))) break;
                    tma_store_4d(&tm_dq, sm + oO, 64 * c, kBlock * cur.n, cur.h0, cur.b);
                    bulk_commit();
                    bulk_wait_read_all();
                    mbar_arrive(ofree);
                }
            bulk_wait_all();
        }
    } else if (warp >= kWarpM) {
        // -------------------------------------------------------- MMAs
        // Three issuers, as one issuing all products was slower than the products: 0 S
        // and dP, 1 dq, 2 dk and dd (four, dd apart: 1141 us against 1058).
        const int who = (int)uniform((uint32_t)(warp - kWarpM));
        const uint32_t tm = uniform(tmem);
        const uint32_t idS = idesc_bf16(128, p.ctxpad + 16, 0), idQ = idesc_bf16(128, 64, 1);
        const uint32_t idK = idesc_bf16_ab(128, 64, 1, 1), idD = idesc_bf16_ab(128, 32, 1, 0);
        const int ksc = p.ctxpad / 16, ksr = (p.hp * kBlock + 15) / 16;
        const SDesc dst = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oDS), kSlot, 1024)));      // keys x rows
        const SDesc pt = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oPr), kSlot, 1024)));
        const SDesc ddb = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oDD), 16, 1024)));         // draft keys x rows
        // slots of keys, and of Q and dO, as rows x columns and transposed
        const SDesc sk = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oK), 16, 1024)));
        const SDesc vk = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oK), kKSlot, 1024)));
        const SDesc sq = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oPair), 16, 1024)));
        const SDesc vq = uniform(sdesc_split(sdesc_sw128(smem_u32(sm + oPair), kSlot, 1024)));
        TileCursor cu(p);
        Tile cur;
        bool ok = true;
        uint32_t i = 0, k = 0;  // slices of gradients; tiles
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return ok = ok && warp_all(mbar_wait(bar, parity, abort_flag, wlim));
        };
        // Copy n of a ring, of a kind: its slot, once it has landed. A parity tells a
        // barrier's phase from the one before only, so copies for the scores and for
        // the gradients, which have other users, have barriers of their own (a user
        // that skipped a copy on a shared one could pass a phase early).
        uint32_t kph = 0, qph = 0;
        auto take_k = [&](int kind, uint32_t n) {
            const uint32_t s = n % kKSlots;
            wait(&kfull[kind * kKSlots + s], (kph >> s) & 1);
            kph ^= 1u << s;
            return s;
        };
        auto take_q = [&](int kind, uint32_t n) {
            const uint32_t s = n % kPairs2;
            wait(&qfull[kind * kPairs2 + s], (qph >> s) & 1);
            qph ^= 1u << s;
            return s;
        };
        for (; ok && cu.next(p, cur); k++) {
            const uint32_t kn = k * (2 * kSlices + 1), qn = k * 2 * kSlices;  // the tile's first copies
            if (who == 0) {
                // S and dP of the tile before are read, and dS, over S, by the products of dq
                if (k > 0 && (!wait(pds, (k - 1) & 1) || !wait(&done[0], (k - 1) & 1))) break;
#pragma unroll 1
                for (int c = 0; c < kSlices; c++) {
                    const uint32_t ks = take_k(1, kn + c), qs = take_q(1, qn + c);
                    if (!ok) break;
                    tc_fence_after();
                    const SDesc kd = sdesc_plus(sk, ks * kKSlot);
                    const SDesc qd = sdesc_plus(sq, qs * kPair);
                    const SDesc gd = sdesc_plus(sq, qs * kPair + kSlot);
                    // the second product: dP; of the rope slice, S again with Q's lo
                    const uint32_t d2 = tm + (c < 8 ? kColP : kColS);
#pragma unroll
                    for (int s = 0; s < 4; s++) mma_bf16_ss_warp(tm + kColS, qd.at(2 * s), kd.at(2 * s), idS, (c | s) != 0);
#pragma unroll
                    for (int s = 0; s < 4; s++) mma_bf16_ss_warp(d2, gd.at(2 * s), kd.at(2 * s), idS, (c | s) != 0);
                    mma_commit_warp(&kempty[ks]);
                    if (c == kSlices - 1) {  // Q's hi with the keys' lo
                        const uint32_t kl = take_k(1, kn + kSlices);
                        if (!ok) break;
                        tc_fence_after();
                        const SDesc ld = sdesc_plus(sk, kl * kKSlot);
#pragma unroll
                        for (int s = 0; s < 4; s++) mma_bf16_ss_warp(tm + kColS, qd.at(2 * s), ld.at(2 * s), idS, 1u);
                        mma_commit_warp(&kempty[kl]);
                    }
                    mma_commit_warp(&qempty[qs]);
                }
                if (ok) mma_commit_warp(sfull);
                continue;
            }
            if (!wait(pds, k & 1)) break;  // P and dS are written
#pragma unroll 1
            for (int c = 0; c < kSlices; c++, i++) {
                if (who == 1) {
                    const uint32_t ks = take_k(0, kn + kSlices + 1 + c);
                    if (!ok || (i > 0 && !wait(qcfree, (i - 1) & 1))) break;
                    tc_fence_after();
                    const uint32_t d = tm + kColC;
                    const SDesc kv = sdesc_plus(vk, ks * kKSlot);
                    // (unrolled: a product of 64 columns takes 50 cycles, a step of a rolled loop 90)
#pragma unroll
                    for (int s = 0; s < 8; s++)
                        if (s < ksc) mma_bf16_ts_warp(d, tm + kColS + 8 * s, kv.at(128 * s), idQ, s > 0);
                    mma_bf16_ts_warp(d, tm + kColS + p.ctxpad / 2, kv.at(p.ctxpad * 8), idQ, ksc > 0);
                    mma_commit_warp(&kempty[ks]);
                    if (c == kSlices - 1) mma_commit_warp(&done[0]);
                    mma_commit_warp(qcfull);  // last: nothing is in flight once its reader has it
                } else {
                    const uint32_t qs = take_q(0, qn + kSlices + c), buf = i & 1;
                    if (!ok || (i > 1 && !wait(&kcfree[buf], ((i >> 1) - 1) & 1))) break;
                    tc_fence_after();
                    const SDesc qb = sdesc_plus(vq, qs * kPair);
                    const SDesc gb = sdesc_plus(vq, qs * kPair + kSlot);
                    const uint32_t d = tm + kColC + 64 + 64 * buf;
                    const SDesc p2 = c < 8 ? pt : dst;
#pragma unroll
                    for (int s = 0; s < kRows / 16; s++) {
                        if (s >= ksr) continue;
                        mma_bf16_ss_warp(d, dst.at(128 * s), qb.at(128 * s), idK, s > 0);
                        mma_bf16_ss_warp(d, p2.at(128 * s), gb.at(128 * s), idK, 1u);
                    }
                    mma_commit_warp(&kcfull[buf]);
                    if (i > 0 && !wait(dfree, (i - 1) & 1)) break;
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < kRows / 16; s++)
                        if (s < ksr)
                            mma_bf16_ss_warp(tm + kColD, qb.at(128 * s), ddb.at((s >> 2) * (32 * 8) + (s & 3) * 2), idD, s > 0);
                    mma_commit_warp(&qempty[qs]);
                    if (c == kSlices - 1) mma_commit_warp(&done[1]);
                    mma_commit_warp(dfull);  // last
                }
            }
        }
    } else if (warp < 8) {
        // ------------------------------- softmax, then the products' readers
        const int q4 = warp & 3, hf = warp >> 2, r = q4 * 32 + lane, j = r % kBlock, hl = r / kBlock;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        TileCursor cu(p);
        Tile cur;
        bool ok = true;
        uint32_t i = 0, k = 0;
        for (; ok && cu.next(p, cur); k++) {
            // softmax: this warp's 64 context keys, warps 0 - 3 the draft keys too
            const bool live = hl < cur.nh;
            const float z = live ? p.lse[((size_t)cur.b * p.n_h + cur.h0 + hl) * p.R + (size_t)kBlock * cur.n + j] * kLog2e
                                 : 0.f;
            ok = warp_all(mbar_wait(sfull, k & 1, abort_flag, wlim));
            if (!ok) break;
            tc_fence_after();
            // visible context slots of this warp's 64
            const int lo = max(0, p.W - 1 - cur.a) - 64 * hf, hi = (live ? p.W - 1 : -1) - 64 * hf;
            const uint32_t in[2] = {slot_mask(lo, hi), slot_mask(lo - 32, hi - 32)};
            float P[64], D4[4] = {0.f, 0.f, 0.f, 0.f}, pd[8], gd[8];
#pragma unroll
            for (int x = 0; x < 64; x++) P[x] = 0.f;
            const bool some = 64 * hf < p.ctxpad;  // (ctxpad is a multiple of 32: half a slice may be unused)
            if (some) {
#pragma unroll
                for (int cc = 0; cc < 2; cc++) {
                    if (64 * hf + 32 * cc >= p.ctxpad) continue;
                    float s[32], g[32];
                    tmem_ld32(trow + kColS + 64 * hf + 32 * cc, s);
                    tmem_ld32(trow + kColP + 64 * hf + 32 * cc, g);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 32; x++) s[x] = ex2(fmaf(s[x], p.scale_log2, -z));
                    if (!warp_all(in[cc] == 0xffffffffu)) {
#pragma unroll
                        for (int x = 0; x < 32; x++) {
                            s[x] = (in[cc] >> x) & 1 ? s[x] : 0.f;
                            g[x] = (in[cc] >> x) & 1 ? g[x] : 0.f;
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 32; x++) {
                        P[32 * cc + x] = s[x];
                        D4[x & 3] = fmaf(s[x], g[x], D4[x & 3]);
                    }
                }
            }
            if (hf == 0) {
                tmem_ld8(trow + kColS + p.ctxpad, pd);
                tmem_ld8(trow + kColP + p.ctxpad, gd);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < kBlock; x++) {
                    pd[x] = live ? ex2(fmaf(pd[x], p.scale_log2, -z)) : 0.f;
                    D4[0] = live ? fmaf(pd[x], gd[x], D4[0]) : 0.f;
                }
            }
            float D = (D4[0] + D4[1]) + (D4[2] + D4[3]);
            xd[hf * 128 + r] = D;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&lbar[q4]);
            ok = warp_all(mbar_wait(&lbar[q4], k & 1, abort_flag, wlim));
            if (!ok) break;
            tc_fence_after();
            D += xd[(hf ^ 1) * 128 + r];
            // the products of the tile before have read P and dS
            if (k > 0) {
                ok = warp_all(mbar_wait(&done[0], (k - 1) & 1, abort_flag, wlim)) &&
                     warp_all(mbar_wait(&done[1], (k - 1) & 1, abort_flag, wlim));
                if (!ok) break;
            }
            if (some) {
#pragma unroll
                for (int cc = 0; cc < 2; cc++) {
                    if (64 * hf + 32 * cc >= p.ctxpad) continue;
                    float g[32];
                    tmem_ld32(trow + kColP + 64 * hf + 32 * cc, g);
                    tmem_wait_ld();
                    if (!warp_all(in[cc] == 0xffffffffu)) {
#pragma unroll
                        for (int x = 0; x < 32; x++) g[x] = (in[cc] >> x) & 1 ? g[x] : D;
                    }
                    // dS twice: rows x keys over S in tensor memory (both halves have read it),
                    // for dq, and in shared memory, read transposed, for dk
                    uint32_t b[16];
#pragma unroll
                    for (int x = 0; x < 16; x++)
                        b[x] = pack_bf16x2(P[32 * cc + 2 * x] * (g[2 * x] - D) * p.scale,
                                           P[32 * cc + 2 * x + 1] * (g[2 * x + 1] - D) * p.scale);
                    tmem_st16u(trow + kColS + 32 * hf + 16 * cc, b);
                    if (r < kRows) {
#pragma unroll
                        for (int u = 0; u < 4; u++) {
                            const float *pp = &P[32 * cc + 8 * u];
                            const uint32_t at = hf * kSlot + sw128(r, 4 * cc + u);
                            *reinterpret_cast<uint4 *>(sm + oPr + at) =
                                make_uint4(pack_bf16x2(pp[0], pp[1]), pack_bf16x2(pp[2], pp[3]), pack_bf16x2(pp[4], pp[5]),
                                           pack_bf16x2(pp[6], pp[7]));
                            *reinterpret_cast<uint4 *>(sm + oDS + at) =
                                make_uint4(b[4 * u], b[4 * u + 1], b[4 * u + 2], b[4 * u + 3]);
                        }
                    }
                }
            }
            if (hf == 0) {
                // draft keys: one bf16 to each of their rows
                uint8_t *dd = sm + oDD + (r >> 6) * (32 * 128) + (r & 7) * 2;
                const int u = (r & 63) >> 3;
                float ds[8];
#pragma unroll
                for (int x = 0; x < 8; x++) ds[x] = x < kBlock && live ? pd[x] * (gd[x] - D) * p.scale : 0.f;
                uint32_t b[8];
#pragma unroll
                for (int x = 0; x < 8; x++) b[x] = x < 4 ? pack_bf16x2(ds[2 * (x & 3)], ds[2 * (x & 3) + 1]) : 0u;
                tmem_st8u(trow + kColS + p.ctxpad / 2, b);
#pragma unroll
                for (int x = 0; x < kBlock; x++) {
                    *reinterpret_cast<__nv_bfloat16 *>(dd + sw128(x, u)) = __float2bfloat16_rn(ds[x]);
                    *reinterpret_cast<__nv_bfloat16 *>(dd + sw128(16 + x, u)) = __float2bfloat16_rn(pd[x]);
                }
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(pds);
            if (hf == 0) {
                // dq: the rope slice turned back
                const float4 *tab = reinterpret_cast<const float4 *>(p.tab + (size_t)(cur.a + j) * (kDR / 2));
                float *dd = p.dacc + ((size_t)cur.b * p.L + p.S + kBlock * cur.n) * kDK + (r & 63);
#pragma unroll 1
                for (int c = 0; c < kSlices; c++, i++) {
                    ok = warp_all(mbar_wait(qcfull, i & 1, abort_flag, wlim));
                    if (!ok) break;
                    tc_fence_after();
                    float v[2][32];
                    tmem_ld32(trow + kColC, v[0]);
                    tmem_ld32(trow + kColC + 32, v[1]);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(qcfree);
                    if (c == 8) {
#pragma unroll
                        for (int u = 0; u < 16; u++) {
                            const float4 cs = __ldg(tab + u);
                            float *x = &v[u >> 3][4 * (u & 7)];
                            const float x0 = x[0], x1 = x[1], x2 = x[2], x3 = x[3];
                            x[0] = x0 * cs.x + x1 * cs.y;
                            x[1] = x1 * cs.x - x0 * cs.y;
                            x[2] = x2 * cs.z + x3 * cs.w;
                            x[3] = x3 * cs.z - x2 * cs.w;
                        }
                    }
                    if (i > 0) ok = warp_all(mbar_wait(ofree, (i - 1) & 1, abort_flag, wlim));
                    if (!ok) break;
                    if (r < kRows) {
#pragma unroll
                        for (int u = 0; u < 8; u++) {
                            const float *x = &v[u >> 2][8 * (u & 3)];
                            *reinterpret_cast<uint4 *>(sm + oO + sw128(r, u)) =
                                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                           pack_bf16x2(x[6], x[7]));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ofull);
                    // dd: lanes 0 - 63 Q^T dS_d (columns 0 - 4), lanes 64 - 127 dO^T P_d (columns 16 - 20);
                    // of the rope slice, lanes 64 - 127 its lo's share of dS_d
                    ok = warp_all(mbar_wait(dfull, i & 1, abort_flag, wlim));
                    if (!ok) break;
                    tc_fence_after();
                    float d[8];
                    tmem_ld8(trow + kColD + (q4 >= 2 && c < 8 ? 16 : 0), d);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(dfree);
#pragma unroll
                    for (int e = 0; e < kBlock; e++) red1(dd + (size_t)e * kDK + 64 * c, d[e]);
                }
            } else {
                // dk: the warp's 32 key slots, 32 columns at a time through shared memory, a
                // box that one copy adds to the accumulators. (Added by the lanes from there,
                // whole lines each, 3% slower; rows one to a lane, 16 or 32 bytes of a line
                // each, 15%, although that spares shared memory the trip.) Rows past the
                // block's own keys add zero.
                const int first = cur.a - (p.W - 1);
                float *base = p.dacc + (size_t)cur.b * p.L * kDK;
                uint8_t *stg = sm + oT + q4 * 4096;
#pragma unroll 1
                for (int c = 0; c < kSlices; c++, i++) {
                    const uint32_t buf = i & 1;
                    ok = warp_all(mbar_wait(&kcfull[buf], (i >> 1) & 1, abort_flag, wlim));
                    if (!ok) break;
                    tc_fence_after();
                    float v[2][32];
                    tmem_ld32(trow + kColC + 64 + 64 * buf, v[0]);
                    tmem_ld32(trow + kColC + 64 + 64 * buf + 32, v[1]);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kcfree[buf]);
                    if (32 * q4 >= p.W - 1 || first + 32 * q4 + 31 < 0) continue;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        if (lane == 0) bulk_wait_read_all();
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < 8; u++) {
                            const float *x = &v[h][4 * u];
                            *reinterpret_cast<float4 *>(stg + sw128(lane, u)) =
                                32 * q4 + lane < p.W - 1 ? make_float4(x[0], x[1], x[2], x[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        if (first + 32 * q4 >= 0) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_red_3d(&tm_acc, stg, 64 * c + 32 * h, first + 32 * q4, cur.b);
                                bulk_commit();
                            }
                        } else {  // (a box may not start before the first row)
                            __syncwarp();
#pragma unroll 1
                            for (int u = 0; u < 8; u++) {
                                const int row = 4 * u + (lane >> 3), slot = 32 * q4 + row, pos = first + slot;
                                const float4 x = *reinterpret_cast<const float4 *>(stg + sw128(row, lane & 7));
                                if (slot < p.W - 1 && pos >= 0)
                                    red4(base + (size_t)pos * kDK + 64 * c + 32 * h + 4 * (lane & 7), x.x, x.y, x.z, x.w);
                            }
                        }
                    }
                }
            }
        }
    }

    if (warp >= 4 && warp < 8 && lane == 0) bulk_wait_all();

    // ---------------------------------------------------------- teardown
    __syncthreads();
    if (*abort_flag && warp >= kWarpM && warp < kWarpO) mma_commit_warp(&drain[warp - kWarpM]);
    if (*abort_flag && lane == 0) {
        volatile int never = 0;
        const uint32_t ring = warp == kWarpK ? kKSlots : kPairs2;
        uint64_t *full = warp == kWarpK ? kfull : qfull;
        if (warp == kWarpK || warp == kWarpQ)
            for (uint32_t s = 0; s < ring; s++)
                for (int kind = 0; kind < 2; kind++)
                    if ((n_used[kind] >> s) & 1) mbar_wait(&full[kind * ring + s], ((n_phase[kind] >> s) & 1) ^ 1, &never);
        if (warp >= kWarpM && warp < kWarpO) mbar_wait(&drain[warp - kWarpM], 0, &never);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpM) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicOr(p.err, kErrTimeout);
}

// The accumulators as boxes of 32 rows x 32 columns.
bool make_acc_map(CUtensorMap *m, float *acc, uint64_t L, uint64_t B) {
    auto fn = encode_fn();
    const cuuint64_t d[3] = {kDK, L, B}, s[2] = {kDK * 4, L * kDK * 4};
    const cuuint32_t b[3] = {32, 32, 1}, es[3] = {1, 1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, acc, d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Accumulators to outputs: dc rounded, the rope part turned back to its
// position and rounded. One warp per position.
__global__ void __launch_bounds__(256) k_lat_bwd_out(const float *__restrict__ dacc, const int32_t *__restrict__ anchors,
                                                     const float2 *__restrict__ tab, __nv_bfloat16 *__restrict__ dc,
                                                     __nv_bfloat16 *__restrict__ dkr, int B, int S, int N, int L, int P) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const size_t row = (size_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= (size_t)B * L) return;
    const float4 *src = reinterpret_cast<const float4 *>(dacc + row * kDK);
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = src[lane * 2 + (i & 1) + (i >> 1) * 64];
    const float2 x = reinterpret_cast<const float2 *>(dacc + row * kDK + kDL)[lane];
    const int key = (int)(row % (unsigned)L), b = (int)(row / (unsigned)L);
    int pos = key;
    if (key >= S) pos = anchors[(size_t)b * N + (key - S) / kBlock] + (key - S) % kBlock;
    const float2 cs = tab[(size_t)min(max(pos, 0), P - 1) * (kDR / 2) + lane];
#pragma unroll
    for (int i = 0; i < 2; i++)
        reinterpret_cast<uint4 *>(dc + row * kDL)[lane + 32 * i] =
            make_uint4(pack_bf16x2(v[2 * i].x, v[2 * i].y), pack_bf16x2(v[2 * i].z, v[2 * i].w),
                       pack_bf16x2(v[2 * i + 1].x, v[2 * i + 1].y), pack_bf16x2(v[2 * i + 1].z, v[2 * i + 1].w));
    reinterpret_cast<uint32_t *>(dkr + row * kDR)[lane] = pack_bf16x2(x.x * cs.x + x.y * cs.y, x.y * cs.x - x.x * cs.y);
}

}  // namespace

bool lat_bwd_tc_supported(const Prob &p) { return lat_tc_supported(p); }

cudaError_t launch_lat_bwd_tc(const Prob &p, const void *q, const void *c, const int32_t *anchors, const float *lse,
                              const void *dout, void *dq, void *dc, void *dkr, const LatWs &ws, cudaStream_t st) {
    // (the preparation before this has written padding blocks' rows of dq, turned the
    // queries' rope slices and cleared the accumulators)
    if (p.B == 0) return cudaSuccess;
    int dev = 0, nsm = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if (p.N > 0) {
        Args a{};
        a.n_h = p.n_h; a.S = p.S; a.N = p.N; a.W = p.W; a.R = p.R; a.B = p.B; a.L = p.L;
        a.ctxpad = (p.W - 1 + 31) / 32 * 32;
        a.tiles = (p.n_h + kHeads - 1) / kHeads;
        a.hp = (p.n_h + a.tiles - 1) / a.tiles;
        const long long blocks = (long long)p.B * p.N;
        a.nsplit = (int)std::max<long long>(1, std::min<long long>(a.tiles, nsm / blocks));
        a.per = (a.tiles + a.nsplit - 1) / a.nsplit;
        a.nsplit = (a.tiles + a.per - 1) / a.per;
        if (blocks * a.nsplit >= (1ll << 31) - 4096) return cudaErrorInvalidValue;
        a.n_work = (int)(blocks * a.nsplit);
        a.scale = p.scale;
        a.scale_log2 = p.scale_log2;
        a.cnt = ws.base.cnt;
        a.sorted_n = ws.base.sorted_n;
        a.sorted_a = ws.base.sorted_a;
        a.tab = ws.base.rope;
        a.lse = lse;
        a.dacc = ws.dacc;
        a.err = ws.base.err;
        a.wait_ns = p.wait_ns;
        CUtensorMap mq, mg, mr, mc, mh, ml, mc5, mh5, ml5, mdq, macc;
        const uint64_t L = p.L, B = p.B, R = p.R, H = p.n_h;
        const uint64_t qd[4] = {kDK, R, H, B}, qs[3] = {kDK * 2, R * kDK * 2, H * R * kDK * 2};
        const uint64_t gd[4] = {kDL, R, H, B}, gs[3] = {kDL * 2, R * kDL * 2, H * R * kDL * 2};
        const uint64_t sd[4] = {2 * kDR, R, H, B}, ss[3] = {kDR * 4, R * kDR * 4, H * R * kDR * 4};
        const uint32_t qb[4] = {64, kBlock, (uint32_t)a.hp, 1};
        const uint64_t cd[3] = {kDL, L, B}, cs[2] = {kDL * 2, L * kDL * 2};
        const uint64_t rd[3] = {kDR, L, B}, rs[2] = {kDR * 2, L * kDR * 2};
        const uint32_t wb[3] = {64, (uint32_t)std::max(p.W - 1, 1), 1}, db[3] = {64, kBlock, 1};
        if (!make_map_nd(&mq, q, 4, qd, qs, qb) || !make_map_nd(&mdq, dq, 4, qd, qs, qb) ||
            !make_map_nd(&mg, dout, 4, gd, gs, qb) ||
            !make_map_nd(&mr, ws.q_rot, 4, sd, ss, qb) || !make_map_nd(&mc, c, 3, cd, cs, wb) ||
            !make_map_nd(&mh, ws.kr_hi, 3, rd, rs, wb) || !make_map_nd(&mc5, c, 3, cd, cs, db) ||
            !make_map_nd(&mh5, ws.kr_hi, 3, rd, rs, db) || !make_map_nd(&ml, ws.kr_lo, 3, rd, rs, wb) ||
            !make_map_nd(&ml5, ws.kr_lo, 3, rd, rs, db) || !make_acc_map(&macc, ws.dacc, L, B))
            return cudaErrorInvalidValue;
        e = cudaFuncSetAttribute(k_lat_bwd_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        count_launch();
        e = launch_pdl(k_lat_bwd_tc, dim3(std::min(a.n_work, nsm)), dim3(kThreads), kSmem, st, mq, mg, mr, mc, mh, ml,
                       mc5, mh5, ml5, mdq, macc, a);
        if (e != cudaSuccess) return e;
    }
    count_launch();
    return launch_pdl(k_lat_bwd_out, dim3((unsigned)(((size_t)p.B * p.L + 7) / 8)), dim3(256), 0, st,
                      (const float *)ws.dacc, anchors, (const float2 *)ws.base.rope, (__nv_bfloat16 *)dc,
                      (__nv_bfloat16 *)dkr, p.B, p.S, p.N, p.L, p.P);
}

}  // namespace dspark
