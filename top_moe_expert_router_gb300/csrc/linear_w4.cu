// linear_w4.cu — y = x W^T (+ bias) for a few tokens and 4-bit weights with a
// scale per group of the contraction index:
//   NVFP4: w = e2m1 * e4m3 (one per 16) * g (one fp32 per tensor)
//   INT4:  w = (q - z) * s, q in 0..15, z and s one per 32, 64 or 128
// The weights are read once, 4 to 4.5 bits each: the floor is their stream.
//
// The products run as mma.sync m16n8k16 with 16 weight rows as the M operand,
// widened to f16 in registers, and 8 tokens as the N operand. tcgen05.mma is
// not the faster path here: it costs the same 189 cycles for 16 tokens as for
// 256, and wants the widened weights written to shared or tensor memory
// first, whereas these go from the load through a few register operations
// straight into the product.
//
// Exactness. Both formats widen to f16 without rounding: e2m1 * e4m3 has 6
// significant bits and magnitudes in [2^-10, 2688]; q - z is an integer. x in
// f16 and E4M3 is exact in f16; x in bf16 is scaled by a power of two per
// token and 128 columns so that the block's largest element lies in [2^14,
// 2^15): elements down to 2^-29 of the largest keep all their bits, smaller
// ones lose at most 2^-40 of it. Products and sums are fp32; an INT4 group's
// sum is multiplied by its scale, a 128-column block's by x's, in fp32.
//
// The k order inside a 128-column block is free as long as both operands use
// the same: each lane takes L consecutive codes of its row (one 16-, 8- or
// 4-byte load), the four lanes of a row together one group of 4 L codes, and x
// is staged in shared memory in that order, so that a lane's B fragments for
// two products are one conflict-free 16-byte read.
#include <math.h>

#include "ops.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kXSmem = 96 * 1024;      // staged x of one pass over K

__device__ __forceinline__ void mma16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t o;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t o;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}

// Four f16 pairs of a word's eight codes. NVFP4: codes (0,1), (2,3), (4,5),
// (6,7) times the block scale `m`. INT4: codes (0,4), (1,5), (2,6), (3,7)
// minus the zero point: 0x6400 | q is 1024 + q, and `m` is 1024 + z, twice.
template <bool NVFP4>
__device__ __forceinline__ void widen(uint32_t w, uint32_t m, uint32_t o[4]) {
    if constexpr (NVFP4) {
        e2m1x8_to_f16x2(w, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = hmul2(o[i], m);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = hsub2(((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u, m);
    }
}

__device__ __forceinline__ float scale_f32(const void *s, size_t i, moe_dtype t) {
    const uint16_t h = __ldg((const uint16_t *)s + i);
    return t == MOE_T_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

// Eight elements of x as fp32.
__device__ __forceinline__ void load_x8(const W4Args &a, int64_t i, bool vec, float f[8]) {
    if (a.x_type == MOE_T_E4M3) {
        const uint8_t *p = (const uint8_t *)a.x + i;
        uint32_t u[2];
        if (vec) {
            const uint2 v = __ldg((const uint2 *)p);
            u[0] = v.x, u[1] = v.y;
        } else {
            u[0] = u[1] = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j >> 2] |= (uint32_t)__ldg(p + j) << (8 * (j & 3));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t h = e4m3x2_to_f16x2((uint16_t)(u[j >> 1] >> (16 * (j & 1))));
            f[2 * j] = __half2float(__ushort_as_half((uint16_t)h));
            f[2 * j + 1] = __half2float(__ushort_as_half((uint16_t)(h >> 16)));
        }
        return;
    }
    const uint16_t *p = (const uint16_t *)a.x + i;
    uint32_t u[4];
    if (vec) {
        const uint4 v = __ldg((const uint4 *)p);
        u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = (uint32_t)__ldg(p + 2 * j) | ((uint32_t)__ldg(p + 2 * j + 1) << 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (a.x_type == MOE_T_BF16) {
            f[2 * j] = bf16lo(u[j]);
            f[2 * j + 1] = bf16hi(u[j]);
        } else {
            f[2 * j] = __half2float(__ushort_as_half((uint16_t)u[j]));
            f[2 * j + 1] = __half2float(__ushort_as_half((uint16_t)(u[j] >> 16)));
        }
    }
}

// Stages 128-column blocks kb0 .. kb0 + nkb - 1 of tokens m0 .. m0 + mt - 1:
// xh[((kb * 4 + sp) * mt + m) * 4 + t] holds the eight elements that lane t of
// a row multiplies in product pair sp, xsc[kb * mt + m] the block's scale.
template <bool NVFP4, int L>
__device__ __forceinline__ void stage_x(const W4Args &a, uint4 *xh, float *xsc, int m0, int mt, int kb0, int nkb,
                                        bool vec) {
    const int units = mt * nkb * 16;             // 16 threads (half a warp) per token and block
    for (int u = threadIdx.x; u < ((units + 31) & ~31); u += kThreads) {
        const bool in = u < units;
        const int j = u & 15, mb = in ? u >> 4 : 0;
        const int kb = mb % nkb, m = mb / nkb;
        const int k = (kb0 + kb) * 128 + 8 * j;
        float f[8];
        if (in && k < a.K) {
            load_x8(a, (int64_t)(m0 + m) * a.x_ld + k, vec, f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
        }
        float inv = 1.f;
        if (a.x_type == MOE_T_BF16) {
            float big = 0.f;                     // largest finite magnitude of the block
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(f[i]) < INFINITY ? fabsf(f[i]) : 0.f);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
            const uint32_t e = max(__float_as_uint(big) >> 23, 15u);
            const float mul = big > 0.f ? __uint_as_float((268u - e) << 23) : 1.f;  // 2^(14 - exponent)
            inv = big > 0.f ? __uint_as_float((e - 14u) << 23) : 1.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= mul;
        } else if (a.x_type == MOE_T_E4M3) {
            if (in && k < a.K) inv = __ldg(a.xs + (int64_t)(m0 + m) * a.xs_ld + k / a.xgroup);
        }
        if (!in) continue;
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // NVFP4: in order; INT4: the pairs (i, i + 4)
            const __half2 v = NVFP4 ? __floats2half2_rn(f[2 * i], f[2 * i + 1]) : __floats2half2_rn(f[i], f[i + 4]);
            h[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        const int gi = j / (L / 2), t = (j % (L / 2)) / (L / 8), sp = gi * (L / 8) + j % (L / 8);
        xh[((size_t)(kb * 4 + sp) * mt + m) * 4 + t] = make_uint4(h[0], h[1], h[2], h[3]);
        if (j == 0) xsc[kb * mt + m] = inv;
    }
}

// CTA: wr warps along the rows (16 each) by kWarps / wr along K; up to 8 NT tokens.
template <int NT, bool NVFP4, int L>
__global__ void __launch_bounds__(kThreads) linear_w4_kernel(W4Args a, int wr, int kb_pass, int vec) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wk = kWarps / wr, rw = warp % wr, kw = warp / wr;
    const int m0 = blockIdx.y * 8 * NT, mt = min(8 * NT, a.M - m0);
    const int row0 = blockIdx.x * 16 * wr;
    const int r_lo = min(row0 + rw * 16 + g, a.N - 1), r_hi = min(row0 + rw * 16 + g + 8, a.N - 1);
    const int nkb = (a.K + 127) / 128;
    uint4 *xh = reinterpret_cast<uint4 *>(smem);
    float *xsc = reinterpret_cast<float *>(smem + (size_t)kb_pass * mt * 256);
    const uint8_t *q_lo = a.q + (size_t)r_lo * (a.K / 2), *q_hi = a.q + (size_t)r_hi * (a.K / 2);
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;

    for (int p0 = 0; p0 < nkb; p0 += kb_pass) {
        const int np = min(kb_pass, nkb - p0);
        if (p0 > 0) __syncthreads();
        stage_x<NVFP4, L>(a, xh, xsc, m0, mt, p0, np, vec != 0);
        __syncthreads();
        for (int kb = kw; kb < np; kb += wk) {
            const int k0 = (p0 + kb) * 128;
            uint32_t w[2][4];
            uint32_t mul[2][4];                  // per product pair: NVFP4 block scale, INT4 1024 + zero point
            float sc[2][4];                      // INT4: the group's scale
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t *q = h ? q_hi : q_lo;
                const int r = h ? r_hi : r_lo;
                if constexpr (L == 32) {
                    const int k = k0 + 32 * t;
                    const uint4 v = k < a.K ? __ldg((const uint4 *)(q + k / 2)) : make_uint4(0, 0, 0, 0);
                    w[h][0] = v.x, w[h][1] = v.y, w[h][2] = v.z, w[h][3] = v.w;
                } else if constexpr (L == 16) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = k0 + 64 * i + 16 * t;
                        const uint2 v = k < a.K ? __ldg((const uint2 *)(q + k / 2)) : make_uint2(0, 0);
                        w[h][2 * i] = v.x, w[h][2 * i + 1] = v.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = k0 + 32 * i + 8 * t;
                        w[h][i] = k < a.K ? __ldg((const uint32_t *)(q + k / 2)) : 0u;
                    }
                }
                if constexpr (NVFP4) {
                    const int k = k0 + 32 * t;
                    const uint32_t s2 =
                        k < a.K ? e4m3x2_to_f16x2(__ldg((const uint16_t *)((const uint8_t *)a.s + (size_t)r * (a.K / 16) + k / 16)))
                                : 0u;
                    mul[h][0] = mul[h][1] = (s2 & 0xFFFFu) * 0x10001u;
                    mul[h][2] = mul[h][3] = (s2 >> 16) * 0x10001u;
                } else {
                    constexpr int per = L / 8;   // product pairs per group
#pragma unroll
                    for (int i = 0; i < 4; i += per) {
                        const int k = k0 + i * 32;
                        const size_t at = (size_t)r * (a.K / (4 * L)) + k / (4 * L);
                        const float s = k < a.K ? scale_f32(a.s, at, a.s_type) : 0.f;
                        const uint32_t z = a.z && k < a.K ? __ldg(a.z + at) : 8u;
                        // 1024 + z, exact in f16 for any byte
#pragma unroll
                        for (int jj = 0; jj < per; ++jj) {
                            sc[h][i + jj] = s;
                            mul[h][i + jj] = (0x6400u + z) * 0x10001u;
                        }
                    }
                }
            }
            float blk[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) blk[n][i] = 0.f;
            float grp[NT][4];
#pragma unroll
            for (int sp = 0; sp < 4; ++sp) {
                uint32_t lo[4], hi[4];
                widen<NVFP4>(w[0][sp], mul[0][sp], lo);
                widen<NVFP4>(w[1][sp], mul[1][sp], hi);
                constexpr int per = L / 8;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint4 b = make_uint4(0, 0, 0, 0);
                    const int m = n * 8 + g;
                    if (m < mt) b = xh[((size_t)(kb * 4 + sp) * mt + m) * 4 + t];
                    if constexpr (NVFP4) {
                        mma16816(blk[n], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                        mma16816(blk[n], lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                    } else {
                        if (sp % per == 0) grp[n][0] = grp[n][1] = grp[n][2] = grp[n][3] = 0.f;
                        mma16816(grp[n], lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                        mma16816(grp[n], lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                        if (sp % per == per - 1) {
                            blk[n][0] = fmaf(grp[n][0], sc[0][sp], blk[n][0]);
                            blk[n][1] = fmaf(grp[n][1], sc[0][sp], blk[n][1]);
                            blk[n][2] = fmaf(grp[n][2], sc[1][sp], blk[n][2]);
                            blk[n][3] = fmaf(grp[n][3], sc[1][sp], blk[n][3]);
                        }
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int m = n * 8 + 2 * t;
                const float x0 = m < mt ? xsc[kb * mt + m] : 0.f, x1 = m + 1 < mt ? xsc[kb * mt + m + 1] : 0.f;
                acc[n][0] = fmaf(blk[n][0], x0, acc[n][0]);
                acc[n][1] = fmaf(blk[n][1], x1, acc[n][1]);
                acc[n][2] = fmaf(blk[n][2], x0, acc[n][2]);
                acc[n][3] = fmaf(blk[n][3], x1, acc[n][3]);
            }
        }
    }
    // the K-warps' sums, added in their order; then the tensor scale and the bias
    __syncthreads();
    const int rows = 16 * wr;
    constexpr int MP = 8 * NT + 1;               // odd: rows fall on different banks
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float *r = red + ((size_t)kw * rows + rw * 16 + g) * MP + n * 8 + 2 * t;
        r[0] = acc[n][0];
        r[1] = acc[n][1];
        r[8 * MP] = acc[n][2];
        r[8 * MP + 1] = acc[n][3];
    }
    __syncthreads();
    const float gs = NVFP4 ? __ldg(a.g) : 1.f;
    for (int i = tid; i < rows * mt; i += kThreads) {
        const int r = i % rows, m = i / rows, n = row0 + r;
        if (n >= a.N) continue;
        float v = 0.f;
        for (int k = 0; k < wk; ++k) v += red[((size_t)k * rows + r) * MP + m];
        v *= gs;
        if (a.bias) v += __ldg(a.bias + n);
        const int64_t o = (int64_t)(m0 + m) * a.y_ld + n;
        if (a.y_type == MOE_T_F32) ((float *)a.y)[o] = v;
        else if (a.y_type == MOE_T_BF16) ((__nv_bfloat16 *)a.y)[o] = __float2bfloat16_rn(v);
        else ((__half *)a.y)[o] = __float2half_rn(v);
    }
}

template <int NT, bool NVFP4, int L>
cudaError_t launch_one(const W4Args &a, cudaStream_t st) {
    static std::atomic<uint64_t> attr_set{0};
    const cudaError_t e = set_smem_limit_once((const void *)linear_w4_kernel<NT, NVFP4, L>, 200 * 1024, attr_set);
    if (e != cudaSuccess) return e;
    const int mt = a.M < 8 * NT ? a.M : 8 * NT;
    const int nkb = (a.K + 127) / 128;
    int kb_pass = kXSmem / (mt * 256);
    if (kb_pass > nkb) kb_pass = nkb;
    int wr = 8;
    while (wr > 1 && (a.N + 16 * wr - 1) / (16 * wr) < 304) wr /= 2;
    const size_t xb = (size_t)kb_pass * mt * 260;
    const size_t rb = (size_t)kWarps * 16 * (8 * NT + 1) * 4;
    const int es = a.x_type == MOE_T_E4M3 ? 1 : 2;
    const int vec = (uintptr_t)a.x % (8 * es) == 0 && (a.x_ld * es) % (8 * es) == 0;
    const dim3 grid((a.N + 16 * wr - 1) / (16 * wr), (a.M + 8 * NT - 1) / (8 * NT));
    linear_w4_kernel<NT, NVFP4, L><<<grid, kThreads, xb > rb ? xb : rb, st>>>(a, wr, kb_pass, vec);
    return cudaGetLastError();
}

template <int NT>
cudaError_t launch_fmt(const W4Args &a, cudaStream_t st) {
    if (a.nvfp4) return launch_one<NT, true, 32>(a, st);
    if (a.group == 128) return launch_one<NT, false, 32>(a, st);
    if (a.group == 64) return launch_one<NT, false, 16>(a, st);
    return launch_one<NT, false, 8>(a, st);
}

}  // namespace

cudaError_t launch_linear_w4(const W4Args &a, cudaStream_t st) {
    if (a.M <= 8) return launch_fmt<1>(a, st);
    if (a.M <= 16) return launch_fmt<2>(a, st);
    return launch_fmt<4>(a, st);
}

}  // namespace moe
