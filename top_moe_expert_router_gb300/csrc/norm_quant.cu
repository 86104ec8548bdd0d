// norm_quant.cu — residual addition, RMSNorm with a gain, and the output in 16
// or 32 bits or in E4M3 with a scale per group of columns:
//   s = round(x + res)            (to the inputs' type; stored if asked for)
//   y = s / sqrt(mean(s^2) + eps) * gain
//   scale = max|y| over the group / 448 (1 for a group of zeros), q = E4M3(y * (1 / scale))
// The norm is of the rounded sum, so that the result is the same as that of
// the addition and the norm called one after the other. Everything between
// the loads and the one rounding at the end is in fp32, the row held in
// registers: each input is read once and each output written once.
#include <math.h>

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

// V consecutive elements by the widest accesses (V * sizeof(T) is 16 or 32 bytes, or V = 1).
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float f[V]) {
    if constexpr (V == 1) {
        f[0] = to_f32<T>(*p);
    } else {
        constexpr int per = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < V; i += per) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + i);
            const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
            for (int j = 0; j < per; ++j) f[i + j] = to_f32<T>(e[j]);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float f[V]) {
    if constexpr (V == 1) {
        *p = from_f32<T>(f[0]);
    } else {
        constexpr int per = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < V; i += per) {
            uint4 u;
            T *e = reinterpret_cast<T *>(&u);
#pragma unroll
            for (int j = 0; j < per; ++j) e[j] = from_f32<T>(f[i + j]);
            *reinterpret_cast<uint4 *>(p + i) = u;
        }
    }
}

// Maximum that keeps NaN (fmaxf drops it): the amax of a group with a NaN is
// NaN, and so are its scale and codes.
__device__ __forceinline__ float max_nan(float a, float b) { return (a != a || a > b) ? a : b; }

// Sum or maximum over the TPR threads of a row; every thread gets it.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(kFull, v, o);
        v = MAX ? max_nan(v, u) : v + u;
    }
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        __syncthreads();  // part may still be read from the previous use
        if ((threadIdx.x & 31) == 0) part[warp] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < TPR / 32; ++i) v = MAX ? max_nan(v, part[i]) : v + part[i];
    }
    return v;
}

// amax of a group to its scale; 1 where amax / 448 would not be a normal float
// (a group of zeros, or one that is below E4M3's reach in any case).
__device__ __forceinline__ float group_scale(float amax) { return amax < 0x1.cp-118f ? 1.f : amax / 448.f; }

// TPR threads per row, NV vectors of V elements per thread; vector v of thread
// i starts at column (v * TPR + i) * V.
template <typename T, bool E4M3, int TPR, int V, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) add_rmsnorm_kernel(NormArgs a) {
    constexpr int ROWS = TPR == 32 ? 8 : 1;      // rows of a CTA
    __shared__ float part[32];
    extern __shared__ uint32_t amax_s[];         // [ROWS][d / group] where a group is not within a warp
    const int tid = ROWS > 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x >> 5 : 0);
    if (t >= a.T) return;                        // ROWS > 1: whole warps, which share no barrier
    const int d = a.d;
    const T *x = (const T *)a.x + t * a.x_ld;
    const T *res = a.res ? (const T *)a.res + t * a.res_ld : nullptr;
    float s[NV][V];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + tid) * V;
        if (c < d) {
            load_vec<T, V>(x + c, s[v]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) s[v][i] = 0.f;
        }
    }
    if (res) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + tid) * V;
            if (c < d) {
                float r[V];
                load_vec<T, V>(res + c, r);
#pragma unroll
                for (int i = 0; i < V; ++i) s[v][i] = to_f32<T>(from_f32<T>(s[v][i] + r[i]));
            }
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(s[v][i], s[v][i], ss);
    ss = row_reduce<TPR, false>(ss, part);
    float m = ss / (float)d + a.eps;
    float pre = 1.f;
    if (!(m > 1e-30f && m < 1e37f)) {
        // squares that leave fp32's range: the row by its largest element first
        float big = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < V; ++i) big = max_nan(big, fabsf(s[v][i]));
        big = row_reduce<TPR, true>(big, part);
        if (big > 0.f && big < INFINITY) {
            const int ex = min(max(ilogbf(big), -100), 126);
            pre = scalbnf(1.f, -ex);             // a power of two: exact
            float q = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float u = s[v][i] * pre;
                    q = fmaf(u, u, q);
                }
            q = row_reduce<TPR, false>(q, part);
            m = q / (float)d + a.eps * pre * pre;
        }
    }
    // a row of zeros with eps = 0 stays zero
    const float r = m == 0.f ? 0.f : 1.f / sqrtf(m);
    if (a.sum) {
        T *o = (T *)a.sum + t * a.sum_ld;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + tid) * V;
            if (c < d) store_vec<T, V>(o + c, s[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + tid) * V;
        float g[V];
        if (a.gain && c < d) {
            load_vec<T, V>((const T *)a.gain + c, g);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] = 1.f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) s[v][i] = s[v][i] * pre * r * g[i];
    }
    if constexpr (!E4M3) {
        T *o = (T *)a.out + t * a.out_ld;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * TPR + tid) * V;
            if (c < d) store_vec<T, V>(o + c, s[v]);
        }
    } else {
        uint8_t *o = (uint8_t *)a.out + t * a.out_ld;
        float *sc = a.scales + t * a.scales_ld;
        const int group = a.group, ng = d / group;
        const int lanes = group / V;             // threads of a group
        const bool in_warp = group % V == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0;
        uint32_t *am = amax_s + (ROWS > 1 ? (threadIdx.x >> 5) * ng : 0);
        float row_amax = 0.f;
        if (ng == 1) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < V; ++i) row_amax = max_nan(row_amax, fabsf(s[v][i]));
            row_amax = row_reduce<TPR, true>(row_amax, part);
        } else if (!in_warp) {
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
            float inv[V];
            if (ng == 1) {
                const float scale = group_scale(row_amax);
                if (tid == 0 && v == 0) sc[0] = scale;
#pragma unroll
                for (int i = 0; i < V; ++i) inv[i] = 1.f / scale;
            } else if (in_warp) {
                float m8 = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) m8 = max_nan(m8, fabsf(s[v][i]));
                for (int k = lanes >> 1; k > 0; k >>= 1) m8 = max_nan(m8, __shfl_xor_sync(kFull, m8, k));
                const float scale = group_scale(m8);
                if (c < d && (tid & (lanes - 1)) == 0) sc[c / group] = scale;
#pragma unroll
                for (int i = 0; i < V; ++i) inv[i] = 1.f / scale;
            } else if (c < d) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float scale = group_scale(__uint_as_float(am[(c + i) / group]));
                    if ((c + i) % group == 0) sc[(c + i) / group] = scale;
                    inv[i] = 1.f / scale;
                }
            }
            if (c < d) {
                if constexpr (V == 1) {
                    o[c] = (uint8_t)__nv_cvt_float_to_fp8(s[v][0] * inv[0], __NV_SATFINITE, __NV_E4M3);
                } else {
                    uint32_t pk[V / 4];
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                            make_float2(s[v][i] * inv[i], s[v][i + 1] * inv[i + 1]), __NV_SATFINITE, __NV_E4M3);
                        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                            make_float2(s[v][i + 2] * inv[i + 2], s[v][i + 3] * inv[i + 3]), __NV_SATFINITE, __NV_E4M3);
                        pk[i / 4] = lo | (hi << 16);
                    }
                    if constexpr (V == 8) *reinterpret_cast<uint2 *>(o + c) = make_uint2(pk[0], pk[1]);
                    else *reinterpret_cast<uint32_t *>(o + c) = pk[0];
                }
            }
        }
    }
}

template <typename T, bool E4M3, int TPR, int V, int NV>
cudaError_t launch_one(const NormArgs &a, cudaStream_t st) {
    constexpr int ROWS = TPR == 32 ? 8 : 1;
    const int ng = a.d / a.group;
    const size_t smem = E4M3 && ng > 1 ? (size_t)ROWS * ng * 4 : 0;
    const int64_t grid = ((int64_t)a.T + ROWS - 1) / ROWS;
    add_rmsnorm_kernel<T, E4M3, TPR, V, NV><<<(unsigned)grid, ROWS * TPR, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, bool E4M3, int V>
cudaError_t launch_shape(const NormArgs &a, cudaStream_t st) {
    // one warp per row up to 4 vectors a lane, then one CTA per row
    const int nv = (a.d + V - 1) / V;
    if constexpr (V == 1) {
        if (nv <= 128) return launch_one<T, E4M3, 32, V, 4>(a, st);
        if (nv <= 1024) return launch_one<T, E4M3, 256, V, 4>(a, st);
        return launch_one<T, E4M3, 1024, V, 16>(a, st);
    }
    if (nv <= 32) return launch_one<T, E4M3, 32, V, 1>(a, st);
    if (nv <= 64) return launch_one<T, E4M3, 32, V, 2>(a, st);
    if (nv <= 128) return launch_one<T, E4M3, 32, V, 4>(a, st);
    if (nv <= 256) return launch_one<T, E4M3, 256, V, 1>(a, st);
    if (nv <= 512) return launch_one<T, E4M3, 256, V, 2>(a, st);
    if (nv <= 1024) return launch_one<T, E4M3, 256, V, 4>(a, st);
    return launch_one<T, E4M3, 512, V, 4>(a, st);
}

template <typename T>
cudaError_t launch_type(const NormArgs &a, cudaStream_t st) {
    constexpr int V = 8;
    const int es = sizeof(T);
    auto row16 = [&](const void *p, int64_t ld, int size) {
        return !p || ((uintptr_t)p % 16 == 0 && (ld * size) % 16 == 0);
    };
    const bool vec = a.d % V == 0 && row16(a.x, a.x_ld, es) && row16(a.res, a.res_ld, es) &&
                     row16(a.sum, a.sum_ld, es) && row16(a.gain, 0, es) &&
                     (a.e4m3 ? (uintptr_t)a.out % 8 == 0 && a.out_ld % 8 == 0 : row16(a.out, a.out_ld, es));
    if (vec) return a.e4m3 ? launch_shape<T, true, V>(a, st) : launch_shape<T, false, V>(a, st);
    return a.e4m3 ? launch_shape<T, true, 1>(a, st) : launch_shape<T, false, 1>(a, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs &a, cudaStream_t st) {
    if (a.type == MOE_T_BF16) return launch_type<__nv_bfloat16>(a, st);
    if (a.type == MOE_T_F16) return launch_type<__half>(a, st);
    return launch_type<float>(a, st);
}

}  // namespace moe
