// The paged latent cache: rows written (RMS norm, rope turn, rounding) and read
// back as the values that they stand for. One warp per token; both are bound by
// the bytes of the rows at many tokens and by one launch's latency at few.
//
// A written value is the nearest of the exact x * rsqrt(mean x^2 + eps) * w (to
// 2^-40 of it), so a value that ends in 8 bits has no second rounding on its way.
// That takes more than fp32; fp64 throughout was bound by its conversions, so bf16
// inputs use pairs of fp32: squares and x * w are exact in fp32, the sum keeps its
// rounding errors, and the product with the pair of the root is formed with its
// remainder. 16384 tokens of 512 + 64, normed, bf16 rows: 17.5 us (their 37.7 MB: 5.8)
// with two thirds of the issue slots busy. 32768 8-bit rows read: 12.6 us (59 MB: 9).
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

// |x| within 2^-90 .. 2^120
__device__ __forceinline__ bool middle(float x) {
    return (__float_as_uint(x) & 0x7fffffffu) - (37u << 23) <= (247u - 37u) << 23;
}
// The same of p + e, |e| at most half a unit of p (p not 0, in the middle of fp32's range).
__device__ __forceinline__ float to_f_sticky(float p, float e) {
    if (e == 0.f) return p;
    const uint32_t b = __float_as_uint(p);
    // towards zero where the remainder has the other sign
    return __uint_as_float((((b ^ __float_as_uint(e)) >> 31) ? b - 1 : b) | 1u);
}

// Least e >= -117 with amax <= 448 * 2^e (448 = 0.875 * 2^9); 0 for amax = 0.
// (amax: a value or its sticky form; 0.875 * 2^x is exact in either)
__device__ __forceinline__ int fp8_exp(float amax) {
    if (amax == 0.f) return 0;
    int x;
    const float m = frexpf(amax, &x);
    return max(m <= 0.875f ? x - 9 : x - 8, -117);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3_code(float x) {
    // a value that is not finite is kept as NaN, not saturated
    if (!(fabsf(x) <= 3.4028235e38f)) return 0x7fu;
    return (uint32_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kWarps * 32) k_cache_write(dspark_latent_cache p, const T *__restrict__ c,
                                                             const T *__restrict__ kr, const T *__restrict__ w,
                                                             double eps, double inv_dl, RopeFreq freq,
                                                             const int32_t *__restrict__ pos,
                                                             const int64_t *__restrict__ slots,
                                                             uint8_t *__restrict__ cache, size_t row_bytes) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const int64_t slot = slots[t];
    const int ps = pos[t];
    // lane l holds values 8 l .. 8 l + 7 and, above 256 wide, 256 + 8 l ..
    float x[2][8];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int d = 256 * i + 8 * lane;
        if (d < p.d_l) {
            load8(c + (size_t)t * p.d_l + d, x[i]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) x[i][k] = 0.f;
        }
    }
    if (slot < 0 || slot >= (int64_t)p.n_pages * p.page_size) return;  // the whole warp
    uint8_t *row = cache + (size_t)slot * row_bytes;
    // the rope key: lane l turns pairs l, l + 32 (first: its angles need no other
    // load, and take their time while the latent's arrive)
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
    constexpr bool kPairs = sizeof(T) == 2;  // squares and x * w are exact in fp32
    double ss = 0.0;
    float s1 = 0.f, s2 = 0.f;  // sum of squares and its rounding errors
#pragma unroll
    for (int i = 0; i < 2; i++) {
#pragma unroll
        for (int k = 0; k < 8; k++) {
            if constexpr (kPairs) {
                const float q = x[i][k] * x[i][k], n = s1 + q, v = n - s1;
                s2 += (s1 - (n - v)) + (q - v);
                s1 = n;
            } else {
                ss += (double)x[i][k] * (double)x[i][k];
            }
        }
    }
    double rn = 1.0;
    if (w) {
        // (squares that leave fp32's range at either end: formed again in fp64)
        if (kPairs && s1 >= 1e-20f && s1 <= 3.4028235e38f) {
            ss = (double)s1 + (double)s2;
        } else if (kPairs) {
            for (int i = 0; i < 2; i++)
                for (int k = 0; k < 8; k++) ss += (double)x[i][k] * (double)x[i][k];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rn = rsqrt(fma(ss, inv_dl, eps));
    }
    const float rh = (float)rn, rl = fabsf(rh) <= 3.4028235e38f ? (float)(rn - (double)rh) : 0.f;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int d = 256 * i + 8 * lane;
        float z[8];  // sticky values; for fp32 rows, the nearest
        if (w && d < p.d_l) {
            float wv[8];
            load8(w + d, wv);
            // Pairs where u and q lie within 2^-90 .. 2^120 (there they are exact); zeros
            // and what lies outside in fp64.
            bool far = !kPairs;
            if constexpr (kPairs && KIND == DSPARK_CACHE_BF16) {
                // The product in fp32 is off by 2 units at most: only next to the middle of two
                // bf16 values (its low half 0x8000, 1 in 8000) does that matter.
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float u = x[i][k] * wv[k];
                    z[k] = u * rh;
                    far |= !middle(u) || !middle(z[k]) || ((__float_as_uint(z[k]) + 4u) & 0xffffu) - 0x8000u <= 8u;
                }
            } else if constexpr (kPairs) {
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float u = x[i][k] * wv[k], q = u * rh;
                    far |= !middle(u) || !middle(q);
                    const float e = fmaf(u, rl, fmaf(u, rh, -q)), sum = q + e, rest = (q - sum) + e;
                    z[k] = KIND == DSPARK_CACHE_F32 ? sum : to_f_sticky(sum, rest);
                }
            }
            if (far) {
#pragma unroll 1
                for (int k = 0; k < 8; k++) {
                    // (indexed by comparison: the arrays stay in registers)
                    float xv = 0.f, wk = 0.f;
#pragma unroll
                    for (int m = 0; m < 8; m++)
                        if (m == k) {
                            xv = x[i][m];
                            wk = wv[m];
                        }
                    const double y = (double)xv * rn * (double)wk;
                    const float f = KIND == DSPARK_CACHE_F32 ? (float)y : to_f_sticky(y);
#pragma unroll
                    for (int m = 0; m < 8; m++)
                        if (m == k) z[m] = f;
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) z[k] = x[i][k];
        }
        if constexpr (KIND == DSPARK_CACHE_FP8) {
            // a group of 128 values is 16 lanes
            float am = 0.f;
#pragma unroll
            for (int k = 0; k < 8; k++) {
                const float v = fabsf(z[k]);
                if (v <= 3.4028235e38f) am = fmaxf(am, v);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
            const int e = fp8_exp(am);
            const float inv = pow2f(-e);
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                lo |= e4m3_code(z[k] * inv) << (8 * k);
                hi |= e4m3_code(z[4 + k] * inv) << (8 * k);
            }
            if (d < p.d_l) {
                *reinterpret_cast<uint2 *>(row + d) = make_uint2(lo, hi);
                if ((lane & 15) == 0) *reinterpret_cast<float *>(row + p.d_l + 2 * p.d_r + 4 * (d >> 7)) = pow2f(e);
            }
        } else if (d < p.d_l) {
            if constexpr (KIND == DSPARK_CACHE_BF16)
                store8(reinterpret_cast<__nv_bfloat16 *>(row) + d, z);
            else
                store8(reinterpret_cast<float *>(row) + d, z);
        }
    }
    if constexpr (KIND == DSPARK_CACHE_FP8) {
        const size_t used = (size_t)p.d_l + 2 * p.d_r + 4 * (p.d_l >> 7);
        if (used + 4 * lane < row_bytes) *reinterpret_cast<uint32_t *>(row + used + 4 * lane) = 0u;
    }
}

// NT tokens to a warp: their slots together, then all rows' loads, so that many
// tokens wait for two latencies once (32768 8-bit rows: 18 us with one token to a
// warp). Few tokens keep one to a warp, for as many SMs as there are.
template <typename T, int KIND, int NT>
__global__ void __launch_bounds__(kWarps * 32) k_cache_read(dspark_latent_cache p, const uint8_t *__restrict__ cache,
                                                            size_t row_bytes, const int64_t *__restrict__ slots,
                                                            T *__restrict__ c_out, T *__restrict__ kr_out) {
    const int lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * NT;
    if (t0 >= p.T) return;
    int64_t mine = -1;
    if (lane < NT && t0 + lane < p.T) mine = slots[t0 + lane];
    if (mine >= (int64_t)p.n_pages * p.page_size) mine = -1;
    const uint8_t *row[NT];
    bool ok[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
        const int64_t slot = __shfl_sync(0xffffffffu, mine, n);
        ok[n] = slot >= 0;
        row[n] = cache + (size_t)(ok[n] ? slot : 0) * row_bytes;
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int d = 256 * i + 8 * lane;
        if (d >= p.d_l) continue;
        if constexpr (KIND == DSPARK_CACHE_FP8) {
            uint2 w[NT];
            float s[NT];
#pragma unroll
            for (int n = 0; n < NT; n++) {
                w[n] = ok[n] ? *reinterpret_cast<const uint2 *>(row[n] + d) : make_uint2(0, 0);
                s[n] = ok[n] ? *reinterpret_cast<const float *>(row[n] + p.d_l + 2 * p.d_r + 4 * (d >> 7)) : 0.f;
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
                if (t0 + n >= p.T) continue;
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    __nv_fp8_e4m3 q;
                    q.__x = (uint8_t)((k < 4 ? w[n].x : w[n].y) >> (8 * (k & 3)));
                    v[k] = (float)q * s[n];
                }
                store8(c_out + (size_t)(t0 + n) * p.d_l + d, v);
            }
        } else {
            float v[NT][8];
#pragma unroll
            for (int n = 0; n < NT; n++) {
                if (ok[n]) {
                    if constexpr (KIND == DSPARK_CACHE_BF16)
                        load8(reinterpret_cast<const __nv_bfloat16 *>(row[n]) + d, v[n]);
                    else
                        load8(reinterpret_cast<const float *>(row[n]) + d, v[n]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; k++) v[n][k] = 0.f;
                }
            }
#pragma unroll
            for (int n = 0; n < NT; n++)
                if (t0 + n < p.T) store8(c_out + (size_t)(t0 + n) * p.d_l + d, v[n]);
        }
    }
    if (!kr_out) return;
    // the rope keys: 8 values to a lane, token by token
    const int per = p.d_r / 8;
    for (int e = lane; e < NT * per; e += 32) {
        const int n = e / per, d = 8 * (e % per);
        if (t0 + n >= p.T) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] = 0.f;
        bool good = ok[0];
        const uint8_t *r = row[0];
#pragma unroll
        for (int m = 1; m < NT; m++)
            if (n == m) {
                good = ok[m];
                r = row[m];
            }
        if (good) {
            if constexpr (KIND == DSPARK_CACHE_F32)
                load8(reinterpret_cast<const float *>(r) + p.d_l + d, v);
            else
                load8(reinterpret_cast<const __nv_bfloat16 *>(r + (KIND == DSPARK_CACHE_FP8 ? p.d_l : 2 * p.d_l)) + d, v);
        }
        store8(kr_out + (size_t)(t0 + n) * p.d_r + d, v);
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
    k_cache_write<T, K><<<grid, kWarps * 32, 0, st>>>(p, (const T *)c, (const T *)kr, (const T *)w, eps, 1.0 / p.d_l, freq, pos, \
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
    // four tokens to a warp from where the SMs are full with one
    const int nt = p.T >= 148 * 64 ? 4 : 1;
    const unsigned grid = (unsigned)((p.T + kWarps * nt - 1) / (kWarps * nt));
    const size_t rb = cache_row_bytes(p.kind, p.d_l, p.d_r);
    count_launch();
#define DSPARK_READ_N(T, K, NT)                                                                            \
    k_cache_read<T, K, NT><<<grid, kWarps * 32, 0, st>>>(p, (const uint8_t *)cache, rb, slots, (T *)c_out, \
                                                         (T *)kr_out)
#define DSPARK_READ(T, K)                       \
    do {                                        \
        if (nt == 4) DSPARK_READ_N(T, K, 4);    \
        else DSPARK_READ_N(T, K, 1);            \
    } while (0)
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
#undef DSPARK_READ_N
    return cudaGetLastError();
}

}  // namespace dspark
