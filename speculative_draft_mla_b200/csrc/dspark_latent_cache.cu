// The paged latent cache: rows written (RMS norm, rope turn, rounding) and read
// back as the values that they stand for. One warp per token; both are bound by
// the bytes of the rows at many tokens and by one launch's latency at few.
#include <cmath>

#include "dspark_latent.cuh"

namespace dspark {

// (a thread's last table is kept: it depends on these two values alone)
RopeFreq rope_freq(int d_r, double base) {
    thread_local RopeFreq r{};
    thread_local int have_d = -1;
    thread_local double have_base = 0.0;
    if (d_r == have_d && base == have_base) return r;
    have_d = d_r;
    have_base = base;
    for (int i = 0; i < d_r / 2 && i < 64; i++) r.f[i] = std::pow(base, -2.0 * i / d_r);
    return r;
}

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ uint32_t bf2(float a, float b) {
    __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&t);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf2(v[0], v[1]), bf2(v[2], v[3]), bf2(v[4], v[5]), bf2(v[6], v[7]));
}

// A 64-bit value cut to 32 bits with its lowest bit set when anything was cut
// off: rounding the result once more, to at most 22 bits, then gives the
// nearest value of the original (no double rounding at a border).
__device__ __forceinline__ float to_f_sticky(double x) {
    const float f = __double2float_rz(x);
    return (double)f == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Least e >= -117 with amax <= 448 * 2^e (448 = 0.875 * 2^9); 0 for amax = 0.
__device__ __forceinline__ int fp8_exp(double amax) {
    if (amax == 0.0) return 0;
    int x;
    const double m = frexp(amax, &x);
    return max(m <= 0.875 ? x - 9 : x - 8, -117);
}
__device__ __forceinline__ double pow2d(int e) { return __longlong_as_double((long long)(e + 1023) << 52); }

__device__ __forceinline__ uint32_t e4m3_code(float x) {
    // a value that is not finite is kept as NaN, not saturated
    if (!(fabsf(x) <= 3.4028235e38f)) return 0x7fu;
    return (uint32_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kWarps * 32) k_cache_write(dspark_latent_cache p, const T *__restrict__ c,
                                                             const T *__restrict__ kr, const T *__restrict__ w,
                                                             double eps, RopeFreq freq,
                                                             const int32_t *__restrict__ pos,
                                                             const int64_t *__restrict__ slots,
                                                             uint8_t *__restrict__ cache, size_t row_bytes) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int64_t slot = slots[t];
    if (slot < 0 || slot >= (int64_t)p.n_pages * p.page_size) return;  // the whole warp
    uint8_t *row = cache + (size_t)slot * row_bytes;
    // lane l holds values 8 l .. 8 l + 7 and, above 256 wide, 256 + 8 l ..
    float x[2][8];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int d = 256 * i + 8 * lane;
        if (d < p.d_l) {
            load8(c + (size_t)t * p.d_l + d, x[i]);
#pragma unroll
            for (int k = 0; k < 8; k++) ss += (double)x[i][k] * (double)x[i][k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) x[i][k] = 0.f;
        }
    }
    double rn = 1.0;
    if (w) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rn = 1.0 / sqrt(ss / p.d_l + eps);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int d = 256 * i + 8 * lane;
        double y[8];
        if (w && d < p.d_l) {
            float wv[8];
            load8(w + d, wv);
#pragma unroll
            for (int k = 0; k < 8; k++) y[k] = (double)x[i][k] * rn * (double)wv[k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) y[k] = (double)x[i][k];
        }
        if constexpr (KIND == DSPARK_CACHE_FP8) {
            // a group of 128 values is 16 lanes
            double am = 0.0;
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const double v = fabs(y[k]);
                if (v <= 1.7976931348623157e308) am = fmax(am, v);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) am = fmax(am, __shfl_xor_sync(0xffffffffu, am, o));
            const int e = fp8_exp(am);
            const double inv = pow2d(-e);
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                lo |= e4m3_code(to_f_sticky(y[k] * inv)) << (8 * k);
                hi |= e4m3_code(to_f_sticky(y[4 + k] * inv)) << (8 * k);
            }
            if (d < p.d_l) {
                *reinterpret_cast<uint2 *>(row + d) = make_uint2(lo, hi);
                if ((lane & 15) == 0)
                    *reinterpret_cast<float *>(row + p.d_l + 2 * p.d_r + 4 * (d >> 7)) = (float)pow2d(e);
            }
        } else {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; k++) f[k] = KIND == DSPARK_CACHE_BF16 ? to_f_sticky(y[k]) : (float)y[k];
            if (d < p.d_l) {
                if constexpr (KIND == DSPARK_CACHE_BF16)
                    store8(reinterpret_cast<__nv_bfloat16 *>(row) + d, f);
                else
                    store8(reinterpret_cast<float *>(row) + d, f);
            }
        }
    }
    // the rope key: lane l turns pairs l, l + 32
    const int ps = pos[t];
    for (int i = lane; i < p.d_r / 2; i += 32) {
        const float2 cs = rope_cs(ps, freq.f[i]);
        const float x0 = to_f(kr[(size_t)t * p.d_r + 2 * i]), x1 = to_f(kr[(size_t)t * p.d_r + 2 * i + 1]);
        const float y0 = x0 * cs.x - x1 * cs.y, y1 = x0 * cs.y + x1 * cs.x;
        if constexpr (KIND == DSPARK_CACHE_F32)
            *reinterpret_cast<float2 *>(row + 4 * ((size_t)p.d_l + 2 * i)) = make_float2(y0, y1);
        else
            *reinterpret_cast<uint32_t *>(row + (KIND == DSPARK_CACHE_FP8 ? (size_t)p.d_l + 4 * i
                                                                          : 2 * ((size_t)p.d_l + 2 * i))) = bf2(y0, y1);
    }
    if constexpr (KIND == DSPARK_CACHE_FP8) {
        const size_t used = (size_t)p.d_l + 2 * p.d_r + 4 * (p.d_l >> 7);
        if (used + 4 * lane < row_bytes) *reinterpret_cast<uint32_t *>(row + used + 4 * lane) = 0u;
    }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kWarps * 32) k_cache_read(dspark_latent_cache p, const uint8_t *__restrict__ cache,
                                                            size_t row_bytes, const int64_t *__restrict__ slots,
                                                            T *__restrict__ c_out, T *__restrict__ kr_out) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int64_t slot = slots[t];
    const bool ok = slot >= 0 && slot < (int64_t)p.n_pages * p.page_size;
    const uint8_t *row = cache + (size_t)(ok ? slot : 0) * row_bytes;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int d = 256 * i + 8 * lane;
        if (d >= p.d_l) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] = 0.f;
        if (ok) {
            if constexpr (KIND == DSPARK_CACHE_FP8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(row + d);
                const float s = *reinterpret_cast<const float *>(row + p.d_l + 2 * p.d_r + 4 * (d >> 7));
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    __nv_fp8_e4m3 q;
                    q.__x = (uint8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
                    v[k] = (float)q * s;
                }
            } else if constexpr (KIND == DSPARK_CACHE_BF16) {
                load8(reinterpret_cast<const __nv_bfloat16 *>(row) + d, v);
            } else {
                load8(reinterpret_cast<const float *>(row) + d, v);
            }
        }
        store8(c_out + (size_t)t * p.d_l + d, v);
    }
    if (!kr_out) return;
    for (int d = 8 * lane; d < p.d_r; d += 256) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] = 0.f;
        if (ok) {
            if constexpr (KIND == DSPARK_CACHE_F32)
                load8(reinterpret_cast<const float *>(row) + p.d_l + d, v);
            else
                load8(reinterpret_cast<const __nv_bfloat16 *>(row + (KIND == DSPARK_CACHE_FP8 ? p.d_l : 2 * p.d_l)) + d,
                      v);
        }
        store8(kr_out + (size_t)t * p.d_r + d, v);
    }
}

}  // namespace

cudaError_t launch_cache_write(const dspark_latent_cache &p, const void *c, const void *kr, const void *w, double eps,
                               const RopeFreq &freq, const int32_t *pos, const int64_t *slots, void *cache,
                               cudaStream_t st) {
    if (p.T == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((p.T + kWarps - 1) / kWarps);
    const size_t rb = cache_row_bytes(p.kind, p.d_l, p.d_r);
    count_launch();
#define DSPARK_WRITE(T, K)                                                                                       \
    k_cache_write<T, K><<<grid, kWarps * 32, 0, st>>>(p, (const T *)c, (const T *)kr, (const T *)w, eps, freq, pos, \
                                                      slots, (uint8_t *)cache, rb)
    if (p.dtype == DSPARK_F32) {
        if (p.kind == DSPARK_CACHE_F32) DSPARK_WRITE(float, DSPARK_CACHE_F32);
        else if (p.kind == DSPARK_CACHE_BF16) DSPARK_WRITE(float, DSPARK_CACHE_BF16);
        else DSPARK_WRITE(float, DSPARK_CACHE_FP8);
    } else {
        if (p.kind == DSPARK_CACHE_F32) DSPARK_WRITE(__nv_bfloat16, DSPARK_CACHE_F32);
        else if (p.kind == DSPARK_CACHE_BF16) DSPARK_WRITE(__nv_bfloat16, DSPARK_CACHE_BF16);
        else DSPARK_WRITE(__nv_bfloat16, DSPARK_CACHE_FP8);
    }
#undef DSPARK_WRITE
    return cudaGetLastError();
}

cudaError_t launch_cache_read(const dspark_latent_cache &p, const void *cache, const int64_t *slots, void *c_out,
                              void *kr_out, cudaStream_t st) {
    if (p.T == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((p.T + kWarps - 1) / kWarps);
    const size_t rb = cache_row_bytes(p.kind, p.d_l, p.d_r);
    count_launch();
#define DSPARK_READ(T, K)                                                                                      \
    k_cache_read<T, K><<<grid, kWarps * 32, 0, st>>>(p, (const uint8_t *)cache, rb, slots, (T *)c_out, (T *)kr_out)
    if (p.dtype == DSPARK_F32) {
        if (p.kind == DSPARK_CACHE_F32) DSPARK_READ(float, DSPARK_CACHE_F32);
        else if (p.kind == DSPARK_CACHE_BF16) DSPARK_READ(float, DSPARK_CACHE_BF16);
        else DSPARK_READ(float, DSPARK_CACHE_FP8);
    } else {
        if (p.kind == DSPARK_CACHE_F32) DSPARK_READ(__nv_bfloat16, DSPARK_CACHE_F32);
        else if (p.kind == DSPARK_CACHE_BF16) DSPARK_READ(__nv_bfloat16, DSPARK_CACHE_BF16);
        else DSPARK_READ(__nv_bfloat16, DSPARK_CACHE_FP8);
    }
#undef DSPARK_READ
    return cudaGetLastError();
}

}  // namespace dspark
