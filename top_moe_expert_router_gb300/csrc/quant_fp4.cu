// quant_fp4.cu — rows of 16-bit values to microscaled 4-bit floats and back.
//
//   v = x, or silu(x) * up                                    (fp32)
//   NVFP4: g = the smallest power of two >= max|v_row| / 2688 (6 * 448),
//          s = E4M3(max|v_block| / 6 / g), blocks of 16, code = E2M1(v / (s g))
//   MXFP4: s = 2^(floor(log2 max|v_block|) - 2), blocks of 32, code = E2M1(v / s)
// Bound by memory: 2 bytes in and 0.56 (0.53) out an element.
//
// A thread holds units of 16 elements (half a block of MXFP4), a warp or a CTA a
// row, so that a row is read once, from memory to registers, and its maximum is
// known before its codes are formed. A row asked for many times is quantised once
// and its codes copied, where the caller has room for them.
//
// Rounding. Codes and scales are those of exact quotients. g and MXFP4's scales
// are powers of two; max / 6 (fp4_scale.h) is a product with fp32's 1/6 where
// values have 16 bits, and corrected to the nearest float where they are
// silu(x) * up, of 24 bits. v / s, s an E4M3 value, is v h + v l
// with h + l = 1/s to 40 bits or more: rounded once it meets the middles between
// codes exactly (v h alone misses them for s of 13/8, 14/8, 15/8), and for v of 24
// bits no others: a unit of v's last place, divided by s < 2, is 8/15 of one of
// the quotient's or more.
#include <cuda_fp4.h>

#include "fp4_scale.h"
#include "ops.cuh"

namespace moe {
namespace {

constexpr int kQThreads = 256;        // of a CTA that dequantises
constexpr int kManyRows = 4 * 152;    // rows enough for a warp each to fill the GPU
// of values: most of them have left L2 when the last are written, and go first, so that other lines stay (32768 x 4096 to
// NVFP4 and back to bf16: 80.6 -> 78.4 us)
constexpr int64_t kLongBytes = 96 << 20;
constexpr int64_t kGatherElements = 1 << 25;  // of gathered rows, from which on two launches are faster than one

__device__ __forceinline__ void load32(const void *p, bool vec, uint32_t v[8]) {
    if (vec) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "l"(p));
    } else {
        const uint16_t *h = (const uint16_t *)p;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (uint32_t)h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
}

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t u) {
    if (BF16) return make_float2(bf16lo(u), bf16hi(u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// Eight values to eight codes, the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float2 f[4]) {
    uint32_t o;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(o)
        : "f"(f[0].x), "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x), "f"(f[3].y));
    return o;
}

// The larger magnitude, NaN where one is, under any sign.
template <bool BF16>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
    uint32_t o;
    if (BF16)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}
__device__ __forceinline__ float larger(float a, float b) {
    float o;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(o) : "f"(a), "f"(b));
    return o;
}

// The largest magnitude of a thread's 16 elements as the bits of a float (an
// infinity or NaN stays above every finite one).
template <bool BF16, bool UP>
__device__ __forceinline__ uint32_t top_bits(const uint32_t x[8], const float v[16]) {
    if constexpr (UP) {
        float m[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m[i] = larger(larger(v[i], v[i + 4]), larger(v[i + 8], v[i + 12]));
        return __float_as_uint(larger(larger(m[0], m[1]), larger(m[2], m[3]))) & 0x7FFFFFFFu;
    } else {
        const uint32_t m2 = larger2<BF16>(larger2<BF16>(larger2<BF16>(x[0], x[1]), larger2<BF16>(x[2], x[3])),
                                          larger2<BF16>(larger2<BF16>(x[4], x[5]), larger2<BF16>(x[6], x[7]))) & 0x7FFF7FFFu;
        const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
        if (BF16) return m << 16;
        return m >= 0x7C00u ? 0x7F800000u : __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    }
}

// PER: units of 16 elements of a thread. ROW: threads of a row; THREADS of a CTA.
template <bool BF16, bool NVFP4, bool UP, int ROW, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS) quantize_fp4_kernel(const QuantFp4Args a) {
    static_assert(ROW == 32 || ROW == THREADS, "a row is a warp's or a CTA's");
    __shared__ uint32_t part[THREADS / 32];
    // the product that reads the codes may set itself up meanwhile; it waits for the end of this kernel before it reads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    pdl_wait();
    const int tid = threadIdx.x % ROW, units = a.K / 16;
    const int r = blockIdx.x * (THREADS / ROW) + threadIdx.x / ROW;
    if (r >= a.R) return;
    int t = r;
    if (a.rows) {
        t = a.rows[r];
        if ((unsigned)t >= (unsigned)a.T) return;           // the row stays as it is
    }
    const uint16_t *x = (const uint16_t *)a.x + (int64_t)t * a.x_ld;
    const uint16_t *up = UP ? (const uint16_t *)a.up + (int64_t)t * a.up_ld : nullptr;
    uint32_t xv[PER][8], uv[UP ? PER : 1][8], top[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int u = tid + p * ROW;
#pragma unroll
        for (int i = 0; i < 8; ++i) xv[p][i] = 0u;
        if (u < units) load32(x + u * 16, a.vec, xv[p]);
        if constexpr (UP) {
#pragma unroll
            for (int i = 0; i < 8; ++i) uv[p][i] = 0u;
            if (u < units) load32(up + u * 16, a.vec, uv[p]);
        }
    }
    float v[UP ? PER : 1][16];
    uint32_t big = 0u;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        if constexpr (UP) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = widen<BF16>(xv[p][i]), w = widen<BF16>(uv[p][i]);
                v[p][2 * i] = __fdividef(f.x, 1.f + __expf(-f.x)) * w.x;
                v[p][2 * i + 1] = __fdividef(f.y, 1.f + __expf(-f.y)) * w.y;
            }
        }
        top[p] = top_bits<BF16, UP>(xv[p], v[UP ? p : 0]);
        big = max(big, top[p]);
    }
    float g = 1.f, inv_g = 1.f;
    bool finite = true;
    if constexpr (NVFP4) {
        big = __reduce_max_sync(0xFFFFFFFFu, big);
        if constexpr (ROW > 32) {
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = big;
            __syncthreads();
            big = part[0];
#pragma unroll
            for (int i = 1; i < ROW / 32; ++i) big = max(big, part[i]);
        }
        finite = big < 0x7F800000u;
        if (big && finite) {
            const uint32_t q = __float_as_uint(__fdiv_rn(__uint_as_float(big), 2688.f));
            const uint32_t e = max((q >> 23) + ((q & 0x7FFFFFu) != 0u), 27u);   // at least 2^-100
            g = __uint_as_float(e << 23);
            inv_g = __uint_as_float((254u - e) << 23);
            if (e > 127u + 80u) {
                // The parts of 1 / (s g) would leave the range of normal numbers: 2^-64 goes to the elements first. (bf16
                // alone, or a product, is as large. What becomes subnormal has code 0 either way.)
                inv_g *= 18446744073709551616.f;
#pragma unroll
                for (int p = 0; p < PER; ++p) {
                    top[p] = __float_as_uint(__uint_as_float(top[p]) * 5.421010862427522e-20f);
                    if constexpr (UP) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[p][i] *= 5.421010862427522e-20f;
                    } else if constexpr (BF16) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            xv[p][i] = (uint32_t)f32_to_bf16_rn(bf16lo(xv[p][i]) * 5.421010862427522e-20f) |
                                       (uint32_t)f32_to_bf16_rn(bf16hi(xv[p][i]) * 5.421010862427522e-20f) << 16;
                    }
                }
            }
        }
        if (tid == 0) a.g[r] = finite ? g : __int_as_float(0x7FFFFFFF);
        if (!finite) {                                      // zeros, and NaN as the row's scale
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int u = tid + p * ROW;
                if (u >= units) continue;
                *reinterpret_cast<uint2 *>(a.q + (int64_t)r * (a.K / 2) + u * 8) = make_uint2(0u, 0u);
                a.s[(int64_t)r * units + u] = 0u;
            }
            return;
        }
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int u = tid + p * ROW;
        float2 hi, lo;
        uint32_t s;
        bool none;                                          // codes 0 whatever the elements
        if constexpr (NVFP4) {
            const float scaled = __uint_as_float(top[p]) * inv_g;
            s = __nv_cvt_float_to_fp8(UP ? fp4_sixth(scaled) : fp4_sixth_of_short(scaled), __NV_SATFINITE, __NV_E4M3);
            const __half_raw hr = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s, __NV_E4M3);
            const float sf = __half2float(*reinterpret_cast<const __half *>(&hr));
            none = s == 0u;
            // h within 2^-22 of 1 / s, l what it lacks; times 1 / g, a power of two
            float h;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(sf));
            hi.x = hi.y = h * inv_g;
            lo.x = lo.y = fmaf(-h, sf, 1.f) * hi.x;
        } else {
            const uint32_t m = max(top[p], __shfl_xor_sync(0xFFFFFFFFu, top[p], 1));
            none = m >= 0x7F800000u;
            // floor(log2 m) - 2 as a biased exponent, at least 0 (subnormal m among them)
            const int e = max((int)(m >> 23) - 2, 0);
            s = none ? 255u : (uint32_t)e;
            hi.x = hi.y = __uint_as_float((uint32_t)(254 - e) << 23);
            lo = hi;
        }
        uint32_t c[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float2 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (UP)
                    f[i] = make_float2(v[p][8 * h + 2 * i], v[p][8 * h + 2 * i + 1]);
                else
                    f[i] = widen<BF16>(xv[p][4 * h + i]);
                f[i] = NVFP4 ? fma2(f[i], hi, mul2(f[i], lo)) : mul2(f[i], hi);
            }
            c[h] = e2m1x8(f);
            if (none) c[h] = 0u;
        }
        if (u < units) {
            *reinterpret_cast<uint2 *>(a.q + (int64_t)r * (a.K / 2) + u * 8) = make_uint2(c[0], c[1]);
            if (NVFP4)
                a.s[(int64_t)r * units + u] = (uint8_t)s;
            else if ((u & 1) == 0)
                a.s[(int64_t)r * (units / 2) + u / 2] = (uint8_t)s;
        }
    }
}

// Rows of codes and scales by their index, a warp a row. V: bytes that the scales of a row are moved by.
template <typename V>
__global__ void __launch_bounds__(kQThreads) gather_fp4_kernel(const GatherFp4Args a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    pdl_wait();
    const int r = blockIdx.x * (kQThreads / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (r >= a.R) return;
    const int t = a.rows[r];
    if ((unsigned)t >= (unsigned)a.T) return;               // the row stays as it is
    const uint4 *q = reinterpret_cast<const uint4 *>(a.q_from + (int64_t)t * a.q_bytes);
    const V *s = reinterpret_cast<const V *>(a.s_from + (int64_t)t * a.s_bytes);
    uint4 *q_to = reinterpret_cast<uint4 *>(a.q + (int64_t)r * a.q_bytes);
    V *s_to = reinterpret_cast<V *>(a.s + (int64_t)r * a.s_bytes);
#pragma unroll 4
    for (int i = lane; i < a.q_bytes / 16; i += 32) q_to[i] = q[i];
    for (int i = lane; i < a.s_bytes / (int)sizeof(V); i += 32) s_to[i] = s[i];
    if (a.g && lane == 0) a.g[r] = a.g_from[t];
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// FIRST: among the first lines that leave L2.
template <bool FIRST>
__device__ __forceinline__ void store32(void *p, const uint32_t v[8]) {
    if constexpr (FIRST)
        asm volatile("st.global.L2::evict_first.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                     "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
}

// A thread turns units of 16 codes of its row into values. (LONG: more of them than L2 holds.)
template <typename T, bool NVFP4, int ROW, bool LONG>
__global__ void __launch_bounds__(kQThreads) dequantize_fp4_kernel(const DequantFp4Args a) {
    pdl_wait();
    const int tid = threadIdx.x % ROW, units = a.K / 16;
    const int r = blockIdx.x * (kQThreads / ROW) + threadIdx.x / ROW;
    if (r >= a.R) return;
    const float g = NVFP4 && a.g ? a.g[a.g_rows ? r : 0] : 1.f;
    T *out = (T *)a.out + (int64_t)r * a.out_ld;
#pragma unroll 4
    for (int u = tid; u < units; u += ROW) {
        const uint2 c = *reinterpret_cast<const uint2 *>(a.q + (int64_t)r * (a.K / 2) + u * 8);
        float unit;
        if constexpr (NVFP4) {
            const __half_raw hr = __nv_cvt_fp8_to_halfraw(a.s[(int64_t)r * units + u], __NV_E4M3);
            unit = __half2float(*reinterpret_cast<const __half *>(&hr)) * g;
        } else {
            const uint32_t s = a.s[(int64_t)r * (units / 2) + u / 2];
            unit = __uint_as_float(s == 0 ? 0x00400000u : s == 255u ? 0x7FFFFFFFu : s << 23);
        }
        uint32_t h[8];
        e2m1x8_to_f16x2(c.x, h);
        e2m1x8_to_f16x2(c.y, h + 4);
        float f[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 w = widen<false>(h[i]);
            f[2 * i] = w.x * unit;
            f[2 * i + 1] = w.y * unit;
        }
        if constexpr (sizeof(T) == 4) {
            if (a.vec) {
                uint32_t o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(f[i]);
                store32<LONG>(out + u * 16, o);
                store32<LONG>(out + u * 16 + 8, o + 8);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) out[u * 16 + i] = f[i];
            }
        } else {
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = pack2<T>(f[2 * i], f[2 * i + 1]);
            if (a.vec) {
                store32<LONG>(out + u * 16, o);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) ((uint16_t *)out)[u * 16 + i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
            }
        }
    }
}

template <typename A>
cudaError_t launch(void (*kern)(const A), const A &a, int rows, int row_threads, int threads, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    const int per = threads / row_threads;
    cfg.gridDim = dim3((unsigned)((rows + (int64_t)per - 1) / per));
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

// Many rows: a warp each, up to 4096 columns (2048 with up), so that loads, maxima
// and codes of different rows overlap without a barrier. Few rows: as many threads
// for one as it has units.
template <bool BF16, bool NVFP4, bool UP>
cudaError_t launch_quant(const QuantFp4Args &a, cudaStream_t st) {
    const int units = a.K / 16;
#define MOE_Q(ROW, PER, THREADS) \
    return launch(quantize_fp4_kernel<BF16, NVFP4, UP, ROW, PER, THREADS>, a, a.R, ROW, THREADS, st)
    if (a.R > kManyRows) {
        if (units <= 32) MOE_Q(32, 1, 128);
        if (units <= 64) MOE_Q(32, 2, 128);
        if (units <= 96) MOE_Q(32, 3, 128);
        if (units <= 128) MOE_Q(32, 4, 128);
        if (!UP && units <= 192) MOE_Q(32, 6, 128);
        if (!UP && units <= 256) MOE_Q(32, 8, 128);
        if (units <= 256) MOE_Q(128, 2, 128);
        if (units <= 384) MOE_Q(128, 3, 128);
        if (units <= 512) MOE_Q(128, 4, 128);
    } else {
        if (units <= 32) MOE_Q(32, 1, 128);
        if (units <= 128) MOE_Q(128, 1, 128);
        if (units <= 256) MOE_Q(256, 1, 256);
        if (units <= 512) MOE_Q(256, 2, 256);
    }
    if (units <= 768) MOE_Q(256, 3, 256);
    if (units <= 1024) MOE_Q(256, 4, 256);
    if (units <= 1536) MOE_Q(512, 3, 512);
    MOE_Q(512, 4, 512);
#undef MOE_Q
}

bool aligned32(const void *p, int64_t ld_bytes, int rows) {
    return ((uintptr_t)p | (rows > 1 ? (uintptr_t)ld_bytes : 0)) % 32 == 0;
}

}  // namespace

// Rows that are many times the tokens: every token once, into the scratch, and a copy of its codes for each row, which
// moves 0.56 bytes an element instead of 2. Each row by itself and so, us, NVFP4 of bf16: 32768 rows of 4096 tokens x 4096
// 38.5 / 26.7; 16384 rows 22.1 / 19.3; 8192 of 2048 x 4096 12.2 / 11.9; 12288 of 4096 x 4096 17.8 / 18.7; 4096 of 512 x 4096
// 6.0 / 6.6. With up: 16384 of 4096 x 4096 42.3 / 21.5, 4096 of 1024 x 4096 11.6 / 9.6.
size_t quantize_fp4_scratch(const QuantFp4Args &a) {
    if (!a.rows || a.R < (a.up ? 3 : 4) * (int64_t)a.T || (int64_t)a.R * a.K * (a.up ? 2 : 1) < kGatherElements) return 0;
    return (size_t)a.T * (a.K / 2) + ((size_t)a.T * (a.K / (a.nvfp4 ? 16 : 32)) + 15) / 16 * 16 + (size_t)a.T * 4;
}

static cudaError_t launch_quantize_once(QuantFp4Args a, uint8_t *scratch, cudaStream_t st) {
    GatherFp4Args c{};
    c.q_bytes = a.K / 2;
    c.s_bytes = a.K / (a.nvfp4 ? 16 : 32);
    c.rows = a.rows;
    c.T = a.T;
    c.R = a.R;
    c.q = a.q;
    c.s = a.s;
    c.g = a.nvfp4 ? a.g : nullptr;
    c.q_from = a.q = scratch;
    c.s_from = a.s = scratch + (size_t)a.T * c.q_bytes;
    c.g_from = a.g = (float *)(a.s + ((size_t)a.T * c.s_bytes + 15) / 16 * 16);
    a.rows = nullptr;
    a.R = a.T;
    const cudaError_t e = launch_quantize_fp4(a, nullptr, st);
    if (e != cudaSuccess) return e;
    const uintptr_t at = (uintptr_t)c.s | (uintptr_t)c.s_bytes;
    if (at % 16 == 0) return launch(gather_fp4_kernel<uint4>, c, c.R, 32, kQThreads, st);
    if (at % 4 == 0) return launch(gather_fp4_kernel<uint32_t>, c, c.R, 32, kQThreads, st);
    return launch(gather_fp4_kernel<uint16_t>, c, c.R, 32, kQThreads, st);
}

cudaError_t launch_quantize_fp4(QuantFp4Args a, uint8_t *scratch, cudaStream_t st) {
    if (scratch && quantize_fp4_scratch(a)) return launch_quantize_once(a, scratch, st);
    a.vec = aligned32(a.x, 2 * a.x_ld, a.T) && (!a.up || aligned32(a.up, 2 * a.up_ld, a.T));
    const bool bf = a.type == MOE_T_BF16;
    if (a.nvfp4) {
        if (a.up) return bf ? launch_quant<true, true, true>(a, st) : launch_quant<false, true, true>(a, st);
        return bf ? launch_quant<true, true, false>(a, st) : launch_quant<false, true, false>(a, st);
    }
    if (a.up) return bf ? launch_quant<true, false, true>(a, st) : launch_quant<false, false, true>(a, st);
    return bf ? launch_quant<true, false, false>(a, st) : launch_quant<false, false, false>(a, st);
}

// Few rows: a unit a thread, as far as a CTA reaches; more rows: two or four, whose loads overlap. NVFP4 to bf16 with one,
// two, four, us: 608 x 1536 1.6 / 1.9 / 2.1; 2432 x 2560 3.6 / 3.4 / 3.3; 4864 x 4096 10.4 / 9.8 / 10.7; 32768 x 1536
// 25.7 / 22.7 / 21.5; 32768 x 4096 58.9 / 54.0 / 52.9.
template <typename T, bool LONG>
static cudaError_t launch_dequant(const DequantFp4Args &a, cudaStream_t st) {
#define MOE_DQ(ROW)                                                                                        \
    return a.nvfp4 ? launch(dequantize_fp4_kernel<T, true, ROW, LONG>, a, a.R, ROW, kQThreads, st)         \
                   : launch(dequantize_fp4_kernel<T, false, ROW, LONG>, a, a.R, ROW, kQThreads, st)
    const int each = a.R < 8 * 152 ? 1 : a.R < 32 * 152 ? 2 : 4, units = a.K / 16;
    if (units <= 32 * each) MOE_DQ(32);
    if (units <= 64 * each) MOE_DQ(64);
    if (units <= 128 * each) MOE_DQ(128);
    MOE_DQ(256);
#undef MOE_DQ
}

template <typename T>
static cudaError_t launch_dequant(const DequantFp4Args &a, cudaStream_t st) {
    return (int64_t)a.R * a.K * (int64_t)sizeof(T) > kLongBytes ? launch_dequant<T, true>(a, st)
                                                                : launch_dequant<T, false>(a, st);
}

cudaError_t launch_dequantize_fp4(DequantFp4Args a, cudaStream_t st) {
    a.vec = aligned32(a.out, a.out_ld * (a.type == MOE_T_F32 ? 4 : 2), a.R);
    if (a.type == MOE_T_BF16) return launch_dequant<__nv_bfloat16>(a, st);
    if (a.type == MOE_T_F16) return launch_dequant<__half>(a, st);
    return launch_dequant<float>(a, st);
}

}  // namespace moe
