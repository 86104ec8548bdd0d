// norm_quant.cu — residual addition, RMSNorm with a gain, and the output in 16
// or 32 bits or in E4M3 with a scale per group of columns:
//   s = round(x + res)            (to the inputs' type; stored if asked for)
//   y = s / sqrt(mean(s^2) + eps) * gain
//   scale = max|y| over the group / 448 (1 for a group of zeros), q = E4M3(y * (1 / scale))
// The norm is of the rounded sum, so that the result is the same as that of
// the addition and the norm called one after the other. Everything between
// the loads and the one rounding at the end is in fp32, the row held in
// registers: each input is read once and each output written once. It is bound
// by HBM once the loads of the next row overlap the sums and stores of this one
// (bf16, GB300): 16384 x 8192 to bf16 171 us, 6.3 TB/s, against 192 us with one
// row per CTA; 4096 x 4096 to E4M3 by 128 columns 20.8 us, 5.7 TB/s, against 28.
#include <math.h>

#include <type_traits>

#include "ops.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// What V elements are accessed as: 2 to 16 bytes at a time.
template <int B>
struct Words { using type = uint4; };
template <>
struct Words<8> { using type = uint2; };
template <>
struct Words<4> { using type = uint32_t; };
template <typename T, int V>
constexpr int kAccess = V * (int)sizeof(T) < 16 ? V * (int)sizeof(T) : 16;

// V consecutive elements as they lie in memory (V = 1: by itself, widened).
template <typename T, int V>
struct Packed {
    static constexpr int W = V == 1 ? 1 : V * (int)sizeof(T) / 4;
    uint32_t u[W];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (V == 1) {
            u[0] = __float_as_uint(to_f32<T>(*p));
        } else {
            constexpr int A = kAccess<T, V>;
            using U = typename Words<A>::type;
#pragma unroll
            for (int i = 0; i < 4 * W / A; ++i) {
                const U v = reinterpret_cast<const U *>(p)[i];
                const uint32_t *w = reinterpret_cast<const uint32_t *>(&v);
#pragma unroll
                for (int j = 0; j < A / 4; ++j) u[i * (A / 4) + j] = w[j];
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) u[i] = 0u;
    }
    __device__ __forceinline__ void get(float f[V]) const {
        if constexpr (V == 1) {
            f[0] = __uint_as_float(u[0]);
        } else {
            constexpr int per = 4 / sizeof(T);
#pragma unroll
            for (int i = 0; i < W; ++i) {
#pragma unroll
                for (int j = 0; j < per; ++j) {
                    if constexpr (sizeof(T) == 4) {
                        f[i] = __uint_as_float(u[i]);
                    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                        f[i * per + j] = j ? bf16hi(u[i]) : bf16lo(u[i]);
                    } else {
                        f[i * per + j] = __half2float(__ushort_as_half((uint16_t)(u[i] >> (16 * j))));
                    }
                }
            }
        }
    }
};
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float f[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(f[0]);
    } else {
        constexpr int A = kAccess<T, V>, per = A / (int)sizeof(T);
        using U = typename Words<A>::type;
#pragma unroll
        for (int i = 0; i < V; i += per) {
            U u;
            T *e = reinterpret_cast<T *>(&u);
#pragma unroll
            for (int j = 0; j < per; ++j) e[j] = from_f32<T>(f[i + j]);
            *reinterpret_cast<U *>(p + i) = u;
        }
    }
}

// Maximum that keeps NaN (fmaxf drops it): the amax of a group with a NaN is
// NaN, and so are its scale and codes.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Reciprocal and reciprocal square root by the hardware's approximations, a
// relative error of a few 2^-24: an IEEE division or root costs about ten times
// the instructions (4096 x 4096 bf16 to E4M3, one row per CTA: 33.9 us with them,
// 28.0 without).
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Sum or maximum over the TPR threads of a row; every thread gets it. `part`
// alternates between two buffers, so that one barrier is enough.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float (*part)[32], int &buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(kFull, v, o);
        v = MAX ? max_nan(v, u) : v + u;
    }
    if constexpr (TPR > 32) {
        buf ^= 1;
        if ((threadIdx.x & 31) == 0) part[buf][threadIdx.x >> 5] = v;
        __syncthreads();
        v = part[buf][0];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i) v = MAX ? max_nan(v, part[buf][i]) : v + part[buf][i];
    }
    return v;
}

// amax of a group to its scale; 1 where amax / 448 would not be a normal float
// (a group of zeros, or one that is below E4M3's reach in any case).
__device__ __forceinline__ float group_scale(float amax) { return amax < 0x1.cp-118f ? 1.f : amax * (1.f / 448.f); }

// TPR threads per row, NV vectors of V elements per thread; vector v of thread
// i starts at column (v * TPR + i) * V. A CTA walks its rows; with PF the next
// row is on its way while this one is summed and stored, and the gain stays in
// registers.
template <typename T, bool E4M3, int TPR, int V, int NV, bool PF>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR) add_rmsnorm_kernel(NormArgs a, float inv_d) {
    constexpr int ROWS = TPR == 32 ? 8 : 1;      // rows of a CTA at a time
    __shared__ float part[2][32];
    extern __shared__ uint32_t amax_s[];         // [ROWS][d / group] where a group is not within a warp
    const int tid = ROWS > 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    int64_t t = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x >> 5 : 0);
    const int d = a.d;
    int buf = 0;
    Packed<T, V> px[NV], pr[NV], pg[NV];
    auto fetch = [&](int64_t row) {
        const T *x = (const T *)a.x + row * a.x_ld + tid * V;
        const T *r = (const T *)a.res + row * a.res_ld + tid * V;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if ((v * TPR + tid) * V < d) {
                px[v].load(x + v * TPR * V);
                if (a.res) pr[v].load(r + v * TPR * V);
            } else {
                px[v].zero();
                pr[v].zero();
            }
        }
    };
    auto fetch_gain = [&]() {
        if (a.gain)
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if ((v * TPR + tid) * V < d) pg[v].load((const T *)a.gain + (v * TPR + tid) * V);
                else pg[v].zero();
            }
    };
    if (PF && t < a.T) {
        fetch(t);
        fetch_gain();
    }
    for (; t < a.T; t += step) {                 // ROWS > 1: whole warps, which share no barrier
        if (!PF) fetch(t);
        float s[NV][V];
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            px[v].get(s[v]);
            if (a.res) {
                float r[V];
                pr[v].get(r);
#pragma unroll
                for (int i = 0; i < V; ++i) s[v][i] = to_f32<T>(from_f32<T>(s[v][i] + r[i]));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(s[v][i], s[v][i], ss);
        }
        // (in place: a row is read before it is written, and no other row is touched)
        if (PF && t + step < a.T) fetch(t + step);
        if (a.sum) {
            T *o = (T *)a.sum + t * a.sum_ld + tid * V;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if ((v * TPR + tid) * V < d) store_vec<T, V>(o + v * TPR * V, s[v]);
        }
        ss = row_reduce<TPR, false>(ss, part, buf);
        float m = fmaf(ss, inv_d, a.eps);
        if (!(m > 1e-30f && m < 1e33f)) {
            // squares, or an eps, at the ends of fp32's range: the row is first scaled by the power of two that takes
            // the larger of its largest element and sqrt(eps) near 1 (a row of 2^-149 to 2^-23), and its root is
            // taken of the scaled values: neither the factor nor the reciprocal root leaves the range
            float big = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < V; ++i) big = max_nan(big, fabsf(s[v][i]));
            big = row_reduce<TPR, true>(big, part, buf);
            if (big > 0.f && big < INFINITY) {
                int ex = ilogbf(big);
                if (a.eps > 0.f) ex = max(ex, ilogbf(a.eps) >> 1);
                const float pre = scalbnf(1.f, -min(max(ex, -126), 126));
                float q = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        s[v][i] *= pre;
                        q = fmaf(s[v][i], s[v][i], q);
                    }
                q = row_reduce<TPR, false>(q, part, buf);
                m = q * inv_d + a.eps * pre * pre;
            }
        }
        // a row of zeros with eps = 0 stays zero
        const float r = m == 0.f ? 0.f : rsqrtf(m);
        if (!PF) fetch_gain();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (a.gain) {
                float g[V];
                pg[v].get(g);
#pragma unroll
                for (int i = 0; i < V; ++i) s[v][i] = s[v][i] * r * g[i];
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) s[v][i] *= r;
            }
        }
        if constexpr (!E4M3) {
            T *o = (T *)a.out + t * a.out_ld + tid * V;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if ((v * TPR + tid) * V < d) store_vec<T, V>(o + v * TPR * V, s[v]);
        } else {
            uint8_t *o = (uint8_t *)a.out + t * a.out_ld + tid * V;
            float *sc = a.scales + t * a.scales_ld;
            const int group = a.group, ng = d / group;
            const int lanes = group / V;         // threads of a group
            const bool in_warp = group % V == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0;
            const int shift = 31 - __clz(group); // in_warp: the group is V times a power of two
            uint32_t *am = amax_s + (ROWS > 1 ? (threadIdx.x >> 5) * ng : 0);
            float row_scale = 0.f, row_inv = 0.f;
            if (ng == 1) {
                float big = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int i = 0; i < V; ++i) big = max_nan(big, fabsf(s[v][i]));
                row_scale = group_scale(row_reduce<TPR, true>(big, part, buf));
                row_inv = fast_rcp(row_scale);
                if (tid == 0) sc[0] = row_scale;
            } else if (!in_warp) {
                if constexpr (TPR > 32) __syncthreads();  // the last row's readers
                else __syncwarp();
                for (int g = tid; g < ng; g += TPR) am[g] = 0u;
                if constexpr (TPR > 32) __syncthreads();
                else __syncwarp();
                // non-negative floats order like their bits, NaN above all
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = (v * TPR + tid) * V;
                    if (c < d) {
#pragma unroll
                        for (int i = 0; i < V; ++i) atomicMax(&am[(c + i) / group], __float_as_uint(fabsf(s[v][i])));
                    }
                }
                if constexpr (TPR > 32) __syncthreads();
                else __syncwarp();
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * TPR + tid) * V;
                if (ng == 1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) s[v][i] *= row_inv;
                } else if (in_warp) {
                    float big = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) big = max_nan(big, fabsf(s[v][i]));
#pragma unroll
                    for (int k = 16; k > 0; k >>= 1)
                        if (k < lanes) big = max_nan(big, __shfl_xor_sync(kFull, big, k));
                    const float scale = group_scale(big), inv = fast_rcp(scale);
                    if (c < d && (tid & (lanes - 1)) == 0) sc[c >> shift] = scale;
#pragma unroll
                    for (int i = 0; i < V; ++i) s[v][i] *= inv;
                } else if (c < d) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float scale = group_scale(__uint_as_float(am[(c + i) / group]));
                        if ((c + i) % group == 0) sc[(c + i) / group] = scale;
                        s[v][i] *= fast_rcp(scale);
                    }
                }
                if (c < d) {
                    if constexpr (V == 1) {
                        o[v * TPR] = (uint8_t)__nv_cvt_float_to_fp8(s[v][0], __NV_SATFINITE, __NV_E4M3);
                    } else if constexpr (V == 2) {
                        *reinterpret_cast<uint16_t *>(o + v * TPR * V) =
                            (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(s[v][0], s[v][1]), __NV_SATFINITE, __NV_E4M3);
                    } else {
                        uint32_t pk[V / 4];
#pragma unroll
                        for (int i = 0; i < V; i += 4) {
                            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(s[v][i], s[v][i + 1]), __NV_SATFINITE, __NV_E4M3);
                            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(s[v][i + 2], s[v][i + 3]), __NV_SATFINITE, __NV_E4M3);
                            pk[i / 4] = lo | (hi << 16);
                        }
                        *reinterpret_cast<uint2 *>(o + v * TPR * V) = make_uint2(pk[0], pk[1]);
                    }
                }
            }
        }
    }
}

template <typename T, bool E4M3, int TPR, int V, int NV>
cudaError_t launch_one(const NormArgs &a, cudaStream_t st) {
    constexpr int ROWS = TPR == 32 ? 8 : 1;
    // the next row (x and res) and the gain in registers while they take at most 48
    constexpr bool PF = V > 1 && NV <= 8 && NV * V * (int)sizeof(T) <= 64;
    const auto kern = add_rmsnorm_kernel<T, E4M3, TPR, V, NV, PF>;
    const int ng = a.d / a.group;
    const size_t smem = E4M3 && ng > 1 ? (size_t)ROWS * ng * 4 : 0;
    int64_t grid = ((int64_t)a.T + ROWS - 1) / ROWS;
    if (PF) {
        // as many CTAs as stay on the SMs at once
        int dev = 0, sms = 0, per = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && grid > sms) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, ROWS * TPR, smem);
        if (e != cudaSuccess) return e;
        if (per > 0 && grid > (int64_t)sms * per) grid = (int64_t)sms * per;
    }
    kern<<<(unsigned)grid, ROWS * TPR, smem, st>>>(a, 1.f / (float)a.d);
    return cudaGetLastError();
}

template <typename T, bool E4M3, int V>
cudaError_t launch_shape(const NormArgs &a, cudaStream_t st) {
    // one warp per row up to 4 vectors a lane, then one CTA per row
    const int nv = (a.d + V - 1) / V;
    if constexpr (V <= 2) {
        // rows off the 16-byte boundaries (12361 x 1102 fp32: 36 us by pairs; by single
        // elements with 1024 threads of 16 each it took 250)
        if (nv <= 128) return launch_one<T, E4M3, 32, V, 4>(a, st);
        if (nv <= 512) return launch_one<T, E4M3, 128, V, 4>(a, st);
        if (nv <= 1024) return launch_one<T, E4M3, 256, V, 4>(a, st);
        if (nv <= 2048) return launch_one<T, E4M3, 256, V, 8>(a, st);
        if (nv <= 4096) return launch_one<T, E4M3, 512, V, 8>(a, st);
        if constexpr (V == 1)
            if (nv > 8192) return launch_one<T, E4M3, 1024, V, 16>(a, st);
        return launch_one<T, E4M3, 512, V, 16>(a, st);
    }
    if (nv <= 32) return launch_one<T, E4M3, 32, V, 1>(a, st);
    if (nv <= 64) return launch_one<T, E4M3, 32, V, 2>(a, st);
    if (nv <= 128) return launch_one<T, E4M3, 32, V, 4>(a, st);
    if (nv <= 256) return launch_one<T, E4M3, 256, V, 1>(a, st);
    // (128 threads of 4 vectors took 10 % longer at d = 4096, 512 of 2 3 % longer at 8192)
    if (nv <= 512) return launch_one<T, E4M3, 256, V, 2>(a, st);
    if (nv <= 1024) return launch_one<T, E4M3, 256, V, 4>(a, st);
    return launch_one<T, E4M3, 512, V, 4>(a, st);
}

template <typename T>
cudaError_t launch_type(const NormArgs &a, cudaStream_t st) {
    const int es = sizeof(T);
    // whether every row of every array starts on a boundary of v elements, up to 16 bytes
    auto fits = [&](int v) {
        auto row = [&](const void *p, int64_t ld, int size) {
            const int b = v * size < 16 ? v * size : 16;
            return !p || ((uintptr_t)p % b == 0 && (ld * size) % b == 0);
        };
        return a.d % v == 0 && row(a.x, a.x_ld, es) && row(a.res, a.res_ld, es) && row(a.sum, a.sum_ld, es) &&
               row(a.gain, 0, es) && row(a.out, a.out_ld, a.e4m3 ? 1 : es);
    };
    if (fits(8)) return a.e4m3 ? launch_shape<T, true, 8>(a, st) : launch_shape<T, false, 8>(a, st);
    if (fits(2)) return a.e4m3 ? launch_shape<T, true, 2>(a, st) : launch_shape<T, false, 2>(a, st);
    return a.e4m3 ? launch_shape<T, true, 1>(a, st) : launch_shape<T, false, 1>(a, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs &a, cudaStream_t st) {
    if (a.type == MOE_T_BF16) return launch_type<__nv_bfloat16>(a, st);
    if (a.type == MOE_T_F16) return launch_type<__half>(a, st);
    return launch_type<float>(a, st);
}

}  // namespace moe
