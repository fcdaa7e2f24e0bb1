// Rope keys of the latent draft attention turned to their positions, the rows of
// padding blocks, and what else a backward starts from: the launch between the mask
// descriptor and the attention kernels.
#include <algorithm>

#include "dspark_latent_tc.cuh"

namespace dspark {

namespace {

__device__ __forceinline__ float2 pair_f(float2 v) { return v; }
__device__ __forceinline__ float2 pair_f(__nv_bfloat162 v) { return __bfloat1622float2(v); }
template <typename T> struct Pair;
template <> struct Pair<float> { using V = float2; };
template <> struct Pair<__nv_bfloat16> { using V = __nv_bfloat162; };

// The queries' rope slices turned to their positions, hi then lo, and the key
// gradients' accumulators cleared: 313 MB at S = 4096, N = 512, B = 4, 48 us at the
// measured copy rate, beside 76 MB of padding rows (in a launch of its own after the
// padding rows: 14 us more).
__device__ __forceinline__ void bwd_rows(const BwdPrep &w, const int32_t *__restrict__ anchors,
                                         const float2 *__restrict__ tab, int n_h, int N, int P) {
    const size_t t0 = (size_t)blockIdx.x * blockDim.x + threadIdx.x, nt = (size_t)gridDim.x * blockDim.x;
    for (size_t e = t0; e < w.acc4; e += nt) w.acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int R = kBlock * N;
    // eight threads to a row, four pairs each
    for (size_t e = t0; e < w.rows * 8; e += nt) {
        const size_t row = e >> 3;
        const int u = (int)(e & 7), r = (int)(row % (unsigned)R), b = (int)(row / (unsigned)R / (unsigned)n_h);
        const int pos = min(max(anchors[(size_t)b * N + r / kBlock] + r % kBlock, 0), P - 1);
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(w.q + row * (kTcDL + kTcDR) + kTcDL) + u);
        const float4 *cs = reinterpret_cast<const float4 *>(tab + (size_t)pos * (kTcDR / 2)) + 2 * u;
        const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1);
        uint4 hi, lo;
        auto turn = [](uint32_t x, float c, float s, uint32_t &h, uint32_t &l) {
            const float a = __uint_as_float(x << 16), b = __uint_as_float(x & 0xffff0000u);
            tc::split_bf16x2(a * c - b * s, a * s + b * c, h, l);
        };
        turn(v.x, c0.x, c0.y, hi.x, lo.x);
        turn(v.y, c0.z, c0.w, hi.y, lo.y);
        turn(v.z, c1.x, c1.y, hi.z, lo.z);
        turn(v.w, c1.z, c1.w, hi.w, lo.w);
        reinterpret_cast<uint4 *>(w.out + row * 2 * kTcDR)[u] = hi;
        reinterpret_cast<uint4 *>(w.out + row * 2 * kTcDR + kTcDR)[u] = lo;
    }
}

constexpr int kPadHeads = 8;

// Position key of batch row b: context c -> c, draft key S + 5n + i -> A_n + i
// (positions of padding or invalid blocks are clamped into the table; those
// keys are never attended). Warp w takes positions 4 w .. 4 w + 3, lane i pairs
// i, i + 32, ....
//   f32: the turned keys in fp32 (CUDA-core kernels);
//   hi, lo: x = hi + lo to 2^-17, both bf16, for the tensor cores: with one
//   bf16 the scores would be off by up to 2^-8 of their rope part, and the fp32
//   LSE with them; with three products hi hi + lo hi + hi lo it keeps 2^-16.
// The warps also go over the blocks and write the padding ones' rows, and, before a
// backward, turn the queries' rope slices and clear the accumulators.
template <typename T>
__global__ void __launch_bounds__(256) k_lat_prep(const T *__restrict__ kr, const int32_t *__restrict__ anchors,
                                                  const uint8_t *__restrict__ keep, const float2 *__restrict__ tab,
                                                  float *__restrict__ f32, __nv_bfloat16 *__restrict__ hi,
                                                  __nv_bfloat16 *__restrict__ lo, int B, int S, int N, int L, int d_r,
                                                  int P, int n_h, int pad_blocks, PadRows pad, BwdPrep bw) {
    pdl_wait();
    pdl_trigger();
    const int half = d_r / 2, lane = threadIdx.x & 31;
    const size_t rows = half > 0 ? (size_t)B * L : 0;
    using V = typename Pair<T>::V;
    constexpr int kRows = 4;
    const size_t row0 = ((size_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kRows;
    if (row0 < rows) {
        int pos[kRows];
#pragma unroll
        for (int r = 0; r < kRows; r++) {
            const size_t row = min(row0 + r, rows - 1);
            const int key = (int)(row % (unsigned)L), b = (int)(row / (unsigned)L);
            int ps = key;
            if (key >= S) ps = anchors[(size_t)b * N + (key - S) / kBlock] + (key - S) % kBlock;
            pos[r] = min(max(ps, 0), P - 1);
        }
        for (int i = lane; i < half; i += 32) {
            float2 v[kRows], c[kRows];
#pragma unroll
            for (int r = 0; r < kRows; r++) {
                const size_t row = min(row0 + r, rows - 1);
                v[r] = pair_f(reinterpret_cast<const V *>(kr + row * d_r)[i]);
                c[r] = tab[(size_t)pos[r] * half + i];
            }
#pragma unroll
            for (int r = 0; r < kRows; r++) {
                if (row0 + r >= rows) continue;
                const float y0 = v[r].x * c[r].x - v[r].y * c[r].y, y1 = v[r].x * c[r].y + v[r].y * c[r].x;
                const size_t at = (row0 + r) * half + i;
                if (f32) reinterpret_cast<float2 *>(f32)[at] = make_float2(y0, y1);
                if (hi) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
                    const float2 hf = __bfloat1622float2(h);
                    reinterpret_cast<__nv_bfloat162 *>(hi)[at] = h;
                    // (an infinity has no remainder)
                    reinterpret_cast<__nv_bfloat162 *>(lo)[at] = __floats2bfloat162_rn(
                        fabsf(hf.x) <= 3.4e38f ? y0 - hf.x : 0.f, fabsf(hf.y) <= 3.4e38f ? y1 - hf.y : 0.f);
                }
            }
        }
    }
    // padding blocks: one warp to a block's eight heads
    const uint4 z = make_uint4(0, 0, 0, 0);
    const int groups = (n_h + kPadHeads - 1) / kPadHeads;
    const long long units = (long long)pad_blocks * groups, step = (long long)gridDim.x * 8;
    for (long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); id < units; id += step) {
        const int g = (int)(id % groups), n = (int)(id / groups % N), b = (int)(id / groups / N);
        const int a = anchors[(size_t)b * N + n];
        if (keep[(size_t)b * N + n] && a >= 0 && a <= S - 2) continue;
        const int h0 = g * kPadHeads, h1 = min(n_h, h0 + kPadHeads), w8 = pad.width[0] / 8;
        for (int h = h0; h < h1; h++) {
            uint4 *dst = reinterpret_cast<uint4 *>(
                reinterpret_cast<__nv_bfloat16 *>(pad.t[0]) +
                (((size_t)b * n_h + h) * pad.rows[0] + (size_t)kBlock * n) * pad.width[0]);
            for (int e = lane; e < kBlock * w8; e += 32) dst[e] = z;
        }
        if (pad.lse)
            for (int e = kBlock * h0 + lane; e < kBlock * h1; e += 32)
                pad.lse[((size_t)b * n_h + e / kBlock) * kBlock * N + (size_t)kBlock * n + e % kBlock] = -INFINITY;
    }
    if constexpr (sizeof(T) == 2)
        if (bw.acc) bwd_rows(bw, anchors, tab, n_h, N, P);
}

}  // namespace

cudaError_t launch_lat_prep(const Prob &p, const void *kr, const int32_t *anchors, const uint8_t *keep,
                            const PadRows *pad, bool tc, bool bwd, const void *q, const LatWs &ws, cudaStream_t st) {
    const size_t rows = p.d_r > 0 ? (size_t)p.B * p.L : 0;
    const int pad_blocks = pad ? p.N * p.B : 0;
    const size_t units = (size_t)pad_blocks * ((p.n_h + kPadHeads - 1) / kPadHeads);
    BwdPrep bw{};
    if (bwd) {
        bw.q = (const __nv_bfloat16 *)q;
        bw.out = ws.q_rot;
        bw.acc = (float4 *)ws.dacc;
        bw.rows = (size_t)p.B * p.n_h * p.R;
        bw.acc4 = (size_t)p.B * p.L * (kTcDL + kTcDR) / 4;
    }
    const size_t most = std::max({(units + 7) / 8, (bw.acc4 + 255) / 256, (bw.rows * 8 + 255) / 256});
    const unsigned grid = (unsigned)std::max<size_t>((rows + 31) / 32, std::min<size_t>(most, 148 * 8));
    if (grid == 0) return cudaSuccess;
    PadRows pr{};
    if (pad) pr = *pad;
    float *f32 = tc ? nullptr : ws.kr_f32;
    __nv_bfloat16 *hi = tc ? ws.kr_hi : nullptr, *lo = tc ? ws.kr_lo : nullptr;
    count_launch();
    if (p.dtype == DSPARK_BF16)
        return launch_pdl(k_lat_prep<__nv_bfloat16>, dim3(grid), dim3(256), 0, st, (const __nv_bfloat16 *)kr, anchors,
                          keep, (const float2 *)ws.base.rope, f32, hi, lo, p.B, p.S, p.N, p.L, p.d_r, p.P, p.n_h,
                          pad_blocks, pr, bw);
    return launch_pdl(k_lat_prep<float>, dim3(grid), dim3(256), 0, st, (const float *)kr, anchors, keep,
                      (const float2 *)ws.base.rope, f32, hi, lo, p.B, p.S, p.N, p.L, p.d_r, p.P, p.n_h, pad_blocks,
                      pr, bw);
}

}  // namespace dspark
