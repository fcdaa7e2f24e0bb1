// Helpers of the latent-space tensor-core kernels beside dspark_tc_common.cuh.
#pragma once

#include "dspark_latent_paged.cuh"
#include "dspark_tc_common.cuh"

namespace dspark {
namespace tc {

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// Products and commits issued by a whole warp, in converged code (its elected
// lane, the same one each time, executes them): operands that are known to be the
// same in all lanes take fewer instructions than one lane's own (34 - 40 cycles a
// product against 47 - 51, more beside busy warps). Where products of 144 keys, 80
// cycles each, hide one lane's instructions, the extra steps cost more than they give.
__device__ __forceinline__ void mma_bf16_ss_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_bf16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_commit_warp(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar))
        : "memory");
}
// The value of lane 0, known to be the same in all lanes.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ SDesc uniform(const SDesc &d) { return SDesc{uniform(d.lo), uniform(d.hi)}; }
__device__ __forceinline__ SDesc sdesc_plus(const SDesc &d, uint32_t bytes) { return SDesc{d.lo + bytes / 16, d.hi}; }
// 4-D tiled TMA load (no multicast) completing on bar's transaction count.
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *m, uint64_t *bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"((uint64_t)m), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
// Bits [lo, hi) of 32 (both may lie outside).
__device__ __forceinline__ uint32_t slot_mask(int lo, int hi) {
    if (hi <= 0 || lo >= 32 || hi <= lo) return 0u;
    return (hi >= 32 ? 0xffffffffu : (1u << hi) - 1u) & ~(lo <= 0 ? 0u : (1u << lo) - 1u);
}
// 4-D tiled TMA store and this thread's bulk group.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *m, const void *src, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"((uint64_t)m),
                 "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// 32 bytes to global memory: one store where the address allows it.
__device__ __forceinline__ void st_global_32B(void *p, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
// x = hi + lo, both bf16, to 2^-17 of x; pairs packed low half first. An
// infinity has no remainder.
__device__ __forceinline__ void split_bf16x2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(x0, x1);
    const float h0 = __uint_as_float(hi << 16), h1 = __uint_as_float(hi & 0xffff0000u);
    lo = pack_bf16x2(fabsf(h0) <= 3.4e38f ? x0 - h0 : 0.f, fabsf(h1) <= 3.4e38f ? x1 - h1 : 0.f);
}

// bf16 tensor map of up to 4 dimensions (strides in bytes, of dimensions 1 ..),
// 128-byte swizzle; box[0] = 64 elements.
inline bool make_map_nd(CUtensorMap *m, const void *base, int nd, const uint64_t *dims, const uint64_t *strides,
                        const uint32_t *box) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[4], s[3];
    cuuint32_t b[4], es[4] = {1, 1, 1, 1};
    for (int i = 0; i < nd; i++) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i) s[i - 1] = strides[i - 1];
    }
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, nd, const_cast<void *>(base), d, s, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries of the paged attention, a tile's rows of 64 columns: columns, heads,
// tokens (the stride of an extent of one is not used).
inline bool make_q_map(CUtensorMap *m, const Paged &p, const PagedPlan &w) {
    const uint64_t dk = (uint64_t)(p.d_l + p.d_r), d[3] = {dk, (uint64_t)p.n_h, (uint64_t)p.T};
    const uint64_t s[2] = {p.n_h > 1 ? 2 * (uint64_t)p.q_hs : 2 * dk, p.T > 1 ? 2 * (uint64_t)p.q_ts : 2 * dk};
    const uint32_t b[3] = {64, (uint32_t)(p.n_h < 128 ? p.n_h : 128), (uint32_t)w.tpt};
    return make_map_nd(m, p.q, 3, d, s, b);
}

}  // namespace tc

// ---- work items of the draft kernels -------------------------------------------
// Item w is a kept block (batch rows in order, blocks by anchor) and one of
// nsplit runs of its tiles of heads.
struct DraftItem {
    int b, n, a, t0, t1;
};
struct DraftCursor {
    const int32_t *cnt, *sorted_n, *sorted_a;
    int B, N, nsplit, tiles, per;  // per: tiles in a run
    int b = 0, base = 0;           // batch row, kept blocks before it
    __device__ __forceinline__ bool at(int w, DraftItem &it) {  // w must not go down
        const int blk = w / nsplit, part = w % nsplit;
        while (b < B) {
            const int c = cnt[b];
            if (blk < base + c) break;
            base += c;
            b++;
        }
        if (b >= B) return false;
        const size_t i = (size_t)b * N + (blk - base);
        it.b = b;
        it.n = sorted_n[i];
        it.a = sorted_a[i];
        it.t0 = part * per;
        it.t1 = min(tiles, it.t0 + per);
        return true;
    }
};

}  // namespace dspark
