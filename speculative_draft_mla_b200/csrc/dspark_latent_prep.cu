// Rope keys of the latent draft attention turned to their positions, and the
// rows of padding blocks: the launch between the mask descriptor and the
// attention kernels.
#include <algorithm>

#include "dspark_latent.cuh"

namespace dspark {

namespace {

__device__ __forceinline__ float2 pair_f(float2 v) { return v; }
__device__ __forceinline__ float2 pair_f(__nv_bfloat162 v) { return __bfloat1622float2(v); }
template <typename T> struct Pair;
template <> struct Pair<float> { using V = float2; };
template <> struct Pair<__nv_bfloat16> { using V = __nv_bfloat162; };

// Position key of batch row b: context c -> c, draft key S + 5n + i -> A_n + i
// (positions of padding or invalid blocks are clamped into the table; those
// keys are never attended). Warp w takes positions 4 w .. 4 w + 3, lane i pairs
// i, i + 32, ....
//   f32: the turned keys in fp32 (CUDA-core kernels);
//   hi, lo: x = hi + lo to 2^-17, both bf16, for the tensor cores: with one
//   bf16 the scores would be off by up to 2^-8 of their rope part, and the fp32
//   LSE with them; with three products hi hi + lo hi + hi lo it keeps 2^-16.
// CTA g also takes blocks g, g + G, ... and writes the padding ones' rows.
template <typename T>
__global__ void __launch_bounds__(256) k_lat_prep(const T *__restrict__ kr, const int32_t *__restrict__ anchors,
                                                  const uint8_t *__restrict__ keep, const float2 *__restrict__ tab,
                                                  float *__restrict__ f32, __nv_bfloat16 *__restrict__ hi,
                                                  __nv_bfloat16 *__restrict__ lo, int B, int S, int N, int L, int d_r,
                                                  int P, int n_h, int pad_blocks, PadRows pad) {
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
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int id = blockIdx.x; id < pad_blocks; id += gridDim.x) {
        const int n = id % N, b = id / N;
        const int a = anchors[(size_t)b * N + n];
        if (keep[(size_t)b * N + n] && a >= 0 && a <= S - 2) continue;
#pragma unroll
        for (int k = 0; k < 3; k++) {
            if (!pad.t[k]) continue;
            // t[0] belongs to the heads, t[1] and t[2] are shared by them
            const int w8 = pad.width[k] / 8, heads = k == 0 ? n_h : 1;
            for (int h = 0; h < heads; h++) {
                uint4 *dst = reinterpret_cast<uint4 *>(
                    reinterpret_cast<__nv_bfloat16 *>(pad.t[k]) +
                    (((size_t)b * heads + h) * pad.rows[k] + pad.first[k] + (size_t)kBlock * n) * pad.width[k]);
                for (int e = threadIdx.x; e < kBlock * w8; e += blockDim.x) dst[e] = z;
            }
        }
        if (pad.lse)
            for (int e = threadIdx.x; e < kBlock * n_h; e += blockDim.x)
                pad.lse[((size_t)b * n_h + e / kBlock) * kBlock * N + (size_t)kBlock * n + e % kBlock] = -INFINITY;
    }
}

}  // namespace

cudaError_t launch_lat_prep(const Prob &p, const void *kr, const int32_t *anchors, const uint8_t *keep,
                            const PadRows *pad, bool tc, const LatWs &ws, cudaStream_t st) {
    const size_t rows = p.d_r > 0 ? (size_t)p.B * p.L : 0;
    const int pad_blocks = pad ? p.N * p.B : 0;
    const unsigned grid = (unsigned)std::max<size_t>((rows + 31) / 32, (size_t)std::min(pad_blocks, 148 * 4));
    if (grid == 0) return cudaSuccess;
    PadRows pr{};
    if (pad) pr = *pad;
    float *f32 = tc ? nullptr : ws.kr_f32;
    __nv_bfloat16 *hi = tc ? ws.kr_hi : nullptr, *lo = tc ? ws.kr_lo : nullptr;
    count_launch();
    if (p.dtype == DSPARK_BF16)
        return launch_pdl(k_lat_prep<__nv_bfloat16>, dim3(grid), dim3(256), 0, st, (const __nv_bfloat16 *)kr, anchors,
                          keep, (const float2 *)ws.base.rope, f32, hi, lo, p.B, p.S, p.N, p.L, p.d_r, p.P, p.n_h,
                          pad_blocks, pr);
    return launch_pdl(k_lat_prep<float>, dim3(grid), dim3(256), 0, st, (const float *)kr, anchors, keep,
                      (const float2 *)ws.base.rope, f32, hi, lo, p.B, p.S, p.N, p.L, p.d_r, p.P, p.n_h, pad_blocks,
                      pr);
}

}  // namespace dspark
