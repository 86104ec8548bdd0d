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
// ones lose at most 2^-39 of it. Products and sums are fp32; an INT4 group's
// sum is multiplied by its scale, a 128-column block's by x's, in fp32.
//
// Structure. A CTA takes tiles of 64 or 128 rows: a producer warp streams their
// codes by TMA through a ring of 256-column stages; four warps along the rows by
// two along a stage's columns widen and multiply them, 16 or 32 rows a warp (at 32
// x is read once for two products). K is split over a cluster of up to 8 CTAs
// where there are few tiles; their sums meet in distributed shared memory, added
// in rank order. What bounds it: the large sizes, about 18 instructions per 256
// weights that issue in 51 % of the slots while the ring, three stages beside x,
// keeps DRAM 60 % busy; the small ones, staging x and joining the parts.
// Measured on the way (131072 x 4096 NVFP4, 4 tokens, 45 us of stream): loads
// into registers one block ahead 92 us (waiting for one block's load waited
// for later ones too), two batches of four blocks in turn 70 us, a ring of
// 16-byte asynchronous copies 88 us (the L1's tag and data cycles: 82 % busy);
// now 61 us. 256-row tiles on one CTA of 16 warps took 63 us, pairs of CTAs that
// share a run of tiles, to end together, 64 us.
//
// The k order inside a 128-column block is free as long as both operands use
// the same. NVFP4: lane t of a row takes the row's 32 codes from 32 t on (one
// 16-byte read, two block scales). INT4: of each 32 codes the eight from 8 t on
// (ldmatrix), so that a product pair lies within one group. x is staged in
// shared memory in that order: a lane's B fragments for two products are one
// conflict-free 16-byte read.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "gemm.cuh"
#include "ops.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kCons = 8;               // warps: 4 along a tile's rows by the 2 blocks of a stage
constexpr int kConsThreads = 32 * kCons;
constexpr int kThreads = kConsThreads + 32;

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
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t o;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o) : "r"(a), "r"(b), "r"(c));
    return o;
}

// Four f16 pairs of a word's eight codes. NVFP4: codes (0,1), (2,3), (4,5),
// (6,7) times the block scale, `m` twice that scale in f16.
__device__ __forceinline__ void widen_fp4(uint32_t w, uint32_t m, uint32_t o[4]) {
    e2m1x8_to_f16x2(w, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = hmul2(o[i], m);
}

// INT4: codes (0,4), (1,5), (2,6), (3,7) minus the zero point. 0x6400 | q is
// 1024 + q in f16 and 0x6400 | 16 q is 1024 + 16 q: m0 = 1024 + z is subtracted
// from the first, m1 = -(64 + z) added to a sixteenth of the second: integers
// below 2048, all exact.
__device__ __forceinline__ void widen_int4(uint32_t w, uint32_t m0, uint32_t m1, uint32_t o[4]) {
    const uint32_t w8 = w >> 8;
    o[0] = hsub2((w & 0x000F000Fu) | 0x64006400u, m0);
    o[1] = hfma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, m1);
    o[2] = hsub2((w8 & 0x000F000Fu) | 0x64006400u, m0);
    o[3] = hfma2((w8 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, m1);
}

// Every global load here is an ordinary one: the kernel may be on the SMs before
// the one that writes its x (or scales, or bias) has ended, and the path for data
// that is constant while a kernel runs is not ordered by the wait for that end.

// Eight elements of x as they are loaded (E4M3: two words).
template <typename T>
__device__ __forceinline__ uint4 load_x8(const T *p, bool vec) {
    uint32_t u[4] = {0u, 0u, 0u, 0u};
    if constexpr (sizeof(T) == 1) {
        if (vec) {
            const uint2 v = *(const uint2 *)p;
            return make_uint4(v.x, v.y, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
    } else {
        if (vec) return *(const uint4 *)p;
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Units of 16 bytes from one product pair's staged x to the next: 2 modulo 8,
// so that the stores of half a warp (four product pairs, two lanes' columns a
// quarter) fall on different banks.
__device__ __host__ __forceinline__ int pair_stride(int mt) { return 4 * mt + ((mt & 1) ? 6 : 2); }

// Stages 128-column blocks kb0 .. kb0 + nkb - 1 of tokens m0 .. m0 + mt - 1:
// xh[(kb * 4 + sp) * pair_stride + m * 4 + t] holds the eight elements that lane
// t of a row multiplies in product pair sp, xsc[kb * mt + m] the block's scale.
// Half a warp per token and block; the loads of U come first.
template <bool NVFP4, moe_dtype XT>
__device__ __forceinline__ void stage_x_type(const W4Args &a, uint4 *xh, float *xsc, int m0, int mt, int kb0, int nkb,
                                             bool vec) {
    constexpr int U = XT == MOE_T_BF16 ? 4 : 8, slots = kConsThreads / 16, L = NVFP4 ? 32 : 8;
    using T = typename std::conditional<XT == MOE_T_E4M3, uint8_t, uint16_t>::type;
    const int j = threadIdx.x & 15, n = mt * nkb, ps = pair_stride(mt);
    const uint32_t half = 0xFFFFu << (threadIdx.x & 16);
    const int gi = j / (L / 2), t = (j % (L / 2)) / (L / 8), sp = gi * (L / 8) + j % (L / 8);
    const int dm = slots / nkb, dk = slots % nkb;
    int m = (threadIdx.x >> 4) / nkb, kb = (threadIdx.x >> 4) % nkb;
    const T *p = (const T *)a.x + (int64_t)(m0 + m) * a.x_ld + (kb0 + kb) * 128 + 8 * j;
    const int64_t dp = (int64_t)dm * a.x_ld + dk * 128, wrap = a.x_ld - (int64_t)nkb * 128;
    const int kmax = (a.K - 8 * j + 127) / 128 - kb0;  // this thread's columns of block kb exist below kmax
    for (int i0 = threadIdx.x >> 4; i0 < n; i0 += U * slots) {
        uint4 raw[U];
        float sc[U];
        int to[U];                               // the block's first unit, and its scale's place
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to[u] = kb << 8 | m;
            const bool in = i0 + u * slots < n && kb < kmax;
            raw[u] = in ? load_x8(p, vec) : make_uint4(0u, 0u, 0u, 0u);
            sc[u] = 1.f;
            if (XT == MOE_T_E4M3 && j == 0 && in) {
                const int gb = kb0 + kb;
                sc[u] = a.xs[(int64_t)(m0 + m) * a.xs_ld + (a.xgroup == 128 ? gb : gb * 128 / a.xgroup)];
            }
            m += dm;
            kb += dk;
            p += dp;
            if (kb >= nkb) {
                kb -= nkb;
                ++m;
                p += wrap;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u * slots >= n) break;
            uint32_t h[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
            if constexpr (XT == MOE_T_E4M3) {
                const uint32_t lo = h[0], hi = h[1];
                h[0] = e4m3x2_to_f16x2((uint16_t)lo);
                h[1] = e4m3x2_to_f16x2((uint16_t)(lo >> 16));
                h[2] = e4m3x2_to_f16x2((uint16_t)hi);
                h[3] = e4m3x2_to_f16x2((uint16_t)(hi >> 16));
            }
            if constexpr (XT == MOE_T_BF16) {
                // the block's largest magnitude, as bf16 bits
                uint32_t b2 = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) b2 = __vmaxu2(b2, h[i] & 0x7FFF7FFFu);
                uint32_t big = max(b2 & 0xFFFFu, b2 >> 16);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(half, big, o));
                if (big >= 0x7F80u) {            // infinities or NaN in the block: the largest finite one
                    big = 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t e = (h[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
                        big = max(big, e < 0x7F80u ? e : 0u);
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(half, big, o));
                }
                const uint32_t e = max(big >> 7, 15u);
                const float mul = big ? __uint_as_float((268u - e) << 23) : 1.f;  // 2^(14 - exponent)
                sc[u] = big ? __uint_as_float((e - 14u) << 23) : 1.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __half2 v = __floats2half2_rn(bf16lo(h[i]) * mul, bf16hi(h[i]) * mul);
                    h[i] = *reinterpret_cast<const uint32_t *>(&v);
                }
            }
            // NVFP4: in order; INT4: the pairs (i, i + 4)
            uint4 o = make_uint4(h[0], h[1], h[2], h[3]);
            if constexpr (!NVFP4)
                o = make_uint4(__byte_perm(h[0], h[2], 0x5410), __byte_perm(h[0], h[2], 0x7632),
                               __byte_perm(h[1], h[3], 0x5410), __byte_perm(h[1], h[3], 0x7632));
            const int ku = to[u] >> 8, mu = to[u] & 255;
            xh[(ku * 4 + sp) * ps + mu * 4 + t] = o;
            if (j == 0) xsc[ku * mt + mu] = sc[u];
        }
    }
}

template <bool NVFP4>
__device__ __forceinline__ void stage_x(const W4Args &a, uint4 *xh, float *xsc, int m0, int mt, int kb0, int nkb,
                                        bool vec) {
    if (a.x_type == MOE_T_BF16) stage_x_type<NVFP4, MOE_T_BF16>(a, xh, xsc, m0, mt, kb0, nkb, vec);
    else if (a.x_type == MOE_T_F16) stage_x_type<NVFP4, MOE_T_F16>(a, xh, xsc, m0, mt, kb0, nkb, vec);
    else stage_x_type<NVFP4, MOE_T_E4M3>(a, xh, xsc, m0, mt, kb0, nkb, vec);
}

__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 ldmatrix4(uint32_t a) {
    uint4 v;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// A tile has 64 MT rows, 16 MT per warp. A ring stage: two 128-column blocks
// of the tile's codes, [block][row][64 B] (INT4: with TMA's 64-byte swizzle),
// and with TS NVFP4's scales, [row][16 B].
template <int MT>
constexpr int kRows = 64 * MT;
template <int MT>
constexpr int kCodes = 2 * kRows<MT> * 64;
template <int MT, bool TS>
constexpr int kStage = kCodes<MT> + (TS ? kRows<MT> * 16 : 0);

// A lane's scales of its warp's block where they do not come with the stage:
// rows 8 j + g of the warp's 16 MT. NVFP4: v[j], the two block scales. INT4:
// scale | zero point << 16 of the block's 128 / G groups, spread over the four
// lanes of a row: item 4 j' + t of the warp's 2 MT rows by 128 / G groups.
template <int MT, bool NVFP4, int G>
struct Scales {
    static constexpr int per_row = NVFP4 ? 4 : 128 / G;
    static constexpr int NV = (2 * MT * per_row + 3) / 4;
    uint32_t v[NV];
};

template <int MT, bool NVFP4, int G>
__device__ __forceinline__ void load_scales(const W4Args &a, int row, int kb, int lane, Scales<MT, NVFP4, G> &s) {
    using S = Scales<MT, NVFP4, G>;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int j = 0; j < S::NV; ++j) {
        // rows past N and columns past K: others of the array, for products that are zero or not stored
        const int item = 4 * j + t, jj = NVFP4 ? j : item / S::per_row;
        const size_t r = min(row + 8 * jj + g, a.N - 1);
        if constexpr (NVFP4) {
            const int k = min(128 * kb + 32 * t, a.K - 32);
            s.v[j] = *(const uint16_t *)((const uint8_t *)a.s + r * (a.K / 16) + (k >> 4));
        } else {
            const int ng = a.K / G, gi = min(kb * S::per_row + item % S::per_row, ng - 1);
            s.v[j] = ((const uint16_t *)a.s)[r * ng + gi] | (a.z ? (uint32_t)a.z[r * ng + gi] : 8u) << 16;
        }
    }
}

__device__ __forceinline__ float s_value(uint32_t h, moe_dtype t) {
    return t == MOE_T_BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((uint16_t)h));
}

// acc += a warp's 16 MT rows by one block. Shared-memory addresses: `codes` and
// `scales` of this lane's first row, `x` of the block's staged x (product pair sp
// of token n at x + sp * ps + tok[n]), `xs` of its scales (column n at xs + col[n]).
template <int NT, int MT, bool NVFP4, int G, bool TS>
__device__ __forceinline__ void mul_block(const W4Args &a, uint32_t codes, uint32_t scales, int lane,
                                          const Scales<MT, NVFP4, G> &sc, uint32_t x, uint32_t xs, int ps,
                                          const uint32_t (&tok)[NT], const uint32_t (&col)[NT][2],
                                          float (&acc)[MT][NT][4]) {
    using S = Scales<MT, NVFP4, G>;
    float x0[NT], x1[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        x0[n] = lds_f32(xs + col[n][0]);
        x1[n] = lds_f32(xs + col[n][1]);
    }
    uint32_t w[2 * MT][4];
    uint32_t s2[2 * MT];                         // NVFP4: the lane's two block scales of each row, in f16
#pragma unroll
    for (int j = 0; j < 2 * MT; ++j) {
        uint4 v;
        if constexpr (NVFP4) {
            v = lds128(codes + j * 512);
            s2[j] = e4m3x2_to_f16x2((uint16_t)(TS ? lds16(scales + j * 128) : sc.v[j]));
        } else {
            v = ldmatrix4(codes + j * 512);
        }
        w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
    }
    constexpr int per = NVFP4 ? 4 : G / 32;      // product pairs of one partial sum
#pragma unroll
    for (int gi = 0; gi < 4 / per; ++gi) {
        float sf[2 * MT];
        uint32_t z0[2 * MT], z1[2 * MT];
        if constexpr (!NVFP4) {
#pragma unroll
            for (int j = 0; j < 2 * MT; ++j) {
                const int item = j * S::per_row + gi;
                const uint32_t u = __shfl_sync(kFull, sc.v[item / 4], (lane & ~3) | (item & 3));
                sf[j] = s_value(u & 0xFFFFu, a.s_type);
                z0[j] = (0x6400u + (u >> 16)) * 0x10001u;
                z1[j] = hsub2(0x63806380u, z0[j]);  // 960 - (1024 + z), exact
            }
        }
        float part[MT][NT][4];
#pragma unroll
        for (int h = 0; h < MT; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) part[h][n][e] = 0.f;
#pragma unroll
        for (int sp = gi * per; sp < (gi + 1) * per; ++sp) {
            uint32_t f[2 * MT][4];
#pragma unroll
            for (int j = 0; j < 2 * MT; ++j) {
                // NVFP4: codes 0..15 of the lane are its first block of 16, 16..31 the second
                if constexpr (NVFP4) widen_fp4(w[j][sp], __byte_perm(s2[j], 0, sp < 2 ? 0x1010 : 0x3232), f[j]);
                else widen_int4(w[j][sp], z0[j], z1[j], f[j]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 xv = lds128(x + sp * ps + tok[n]);
#pragma unroll
                for (int h = 0; h < MT; ++h) {
                    mma16816(part[h][n], f[2 * h][0], f[2 * h + 1][0], f[2 * h][1], f[2 * h + 1][1], xv.x, xv.y);
                    mma16816(part[h][n], f[2 * h][2], f[2 * h + 1][2], f[2 * h][3], f[2 * h + 1][3], xv.z, xv.w);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < MT; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // (the weights' scale first: its product with x's may leave the range where the sum does not)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[h][n][e] = fmaf(NVFP4 ? part[h][n][e] : part[h][n][e] * sf[2 * h + (e >> 1)], (e & 1) ? x1[n] : x0[n],
                                        acc[h][n][e]);
            }
    }
}

// y of a tile's rows that this part owns, from the sums of all parts.
__device__ __forceinline__ void store_tile(const W4Args &a, const float *sums, int parts, int own, int part, int mp, int m0,
                                        int mt, int row0, int rows, float gs) {
    const int first = part * own, n_own = min(own, rows - first);
    for (int e = threadIdx.x; e < own * mt; e += kConsThreads) {
        const int m = e / own, r = e - m * own, n = row0 + first + r;
        if (r >= n_own || n >= a.N) continue;
        const float *at = sums + r * mp + m;
        float v = 0.f;
        for (int p = 0; p < parts; ++p) v += at[2 * p * own * mp] + at[(2 * p + 1) * own * mp];
        v *= gs;
        if (a.bias) v += a.bias[n];
        const int64_t o = (int64_t)(m0 + m) * a.y_ld + n;
        if (a.y_type == MOE_T_F32) ((float *)a.y)[o] = v;
        else if (a.y_type == MOE_T_BF16) ((__nv_bfloat16 *)a.y)[o] = __float2bfloat16_rn(v);
        else ((__half *)a.y)[o] = __float2half_rn(v);
    }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Error bits of the products on a device (moe_linear_w4_status).
__device__ uint32_t w4_err;

// mbarrier wait that gives up after kWaitLimitNs, or soon after another warp of
// the CTA has: *bad says so. The tile's outputs are then NaN.
__device__ __forceinline__ void wait_full(uint64_t *bar, uint32_t parity, volatile int *bad) {
    if (mbar_try_wait(bar, parity)) return;
    const unsigned long long t0 = global_ns();
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
        if ((it & 7u) == 0 && *bad) return;
        if ((it & 255u) == 0 && global_ns() - t0 > kWaitLimitNs) {
            atomicOr(&w4_err, ERRBIT_TIMEOUT);
            *bad = 1;
            return;
        }
    }
}

struct Shape {
    int tokens;     // of a token block
    int parts;      // CTAs of a cluster, along K
    int st_pass;    // stages whose x is staged at a time
    int ring;       // stages in flight
    int bars;       // offset of the barriers in shared memory
    int vec;
    int hold;       // test hook: the producers copy nothing
};

// blockIdx.x: the part of K; .y: the first row tile (then every gridDim.y-th);
// .z: the token block. x is staged once where the CTA's part of it fits.
template <int NT, int MT, int CPS, bool NVFP4, int G, bool TS>
__global__ void __launch_bounds__(kThreads, CPS) linear_w4_kernel(const __grid_constant__ CUtensorMap tq,
                                                                const __grid_constant__ CUtensorMap ts, const W4Args a,
                                                                const Shape sh) {
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int MP = 8 * NT + 2;               // even for stores of two columns, and rows on different banks
    constexpr int kR = kRows<MT>, kSt = kStage<MT, TS>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int m0 = blockIdx.z * sh.tokens, mt = min(sh.tokens, a.M - m0);
    const int tiles = (a.N + kR - 1) / kR, parts = sh.parts, part = blockIdx.x;
    const int nst = (a.K + 255) / 256;
    const int s0 = (int)((int64_t)part * nst / parts), s1 = (int)((int64_t)(part + 1) * nst / parts);
    const int R = sh.ring, ps = pair_stride(mt), own = (kR + parts - 1) / parts;
    // ring | two buffers of the tile's sums | x | x's scales | barriers
    float *red = reinterpret_cast<float *>(smem + (size_t)R * kSt);
    uint4 *xh = reinterpret_cast<uint4 *>(red + (parts * 4 * own * MP + 3) / 4 * 4);
    float *xsc = reinterpret_cast<float *>(xh + (size_t)sh.st_pass * 8 * ps);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + sh.bars);
    uint64_t *empty = full + 8;
    volatile int *bad = reinterpret_cast<volatile int *>(empty + 8);
    if (tid == 0) {
        for (int i = 0; i < R; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kCons);
        }
        *bad = 0;
        fence_barrier_init();
    }
    __syncthreads();
    // launched ahead of the end of the kernel before it; lets the next one do the same
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (parts > 1) cluster_arrive();             // this CTA runs: its shared memory may be written to
    pdl_wait();

    if (warp == kCons) {
        // producer: every tile's stages in order; the cluster barrier of a
        // tile is passed before the next one is arrived at
        int i = 0;
        const int s_end = sh.hold ? s0 : s1;
        for (int tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
            if (lane == 0)
                for (int st = s0; st < s_end; ++st, ++i) {
                    const int slot = i % R;
                    if (i >= R) wait_full(&empty[slot], ((i / R) - 1) & 1, bad);
                    if (*bad) break;
                    unsigned char *dst = smem + (size_t)slot * kSt;
                    mbar_arrive_expect_tx(&full[slot], TS ? kSt : kCodes<MT>);
                    tma_load_2d(dst, &tq, st * 128, tile * kR, &full[slot]);
                    tma_load_2d(dst + kR * 64, &tq, st * 128 + 64, tile * kR, &full[slot]);
                    if (TS) tma_load_2d(dst + kCodes<MT>, &ts, st * 16, tile * kR, &full[slot]);
                }
            __syncwarp();
            if (parts > 1) {
                cluster_wait();                  // the start's, or the tile's before
                cluster_arrive();
            }
        }
        // every copy issued must land before the CTA exits (where a wait gave up, nobody else has seen to it)
        if (lane == 0)
            for (int j = i > R ? i - R : 0; j < i; ++j) mbar_wait(&full[j % R], (j / R) & 1, &w4_err);
        __syncwarp();
        if (parts > 1) {
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }

    const int g = lane >> 2, t = lane & 3, wrow = (warp & 3) * 16 * MT, b = warp >> 2;
    // tokens past mt repeat the last one: an output column depends on its own token only
    uint32_t tok[NT], col[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        tok[n] = (min(n * 8 + g, mt - 1) * 4 + t) * 16;
        col[n][0] = min(n * 8 + 2 * t, mt - 1) * 4;
        col[n][1] = min(n * 8 + 2 * t + 1, mt - 1) * 4;
    }
    // NVFP4: the row's codes from 32 t on. INT4, ldmatrix: lane l names row l & 7
    // of matrix l >> 3, which is 16-byte chunk l >> 3 of eight rows.
    const uint32_t code_at = b * (kR * 64) + (NVFP4 ? (wrow + g) * 64 + 16 * t
                                                    : (wrow + (lane & 7)) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4));
    const uint32_t scale_at = kCodes<MT> + (wrow + g) * 16 + 8 * b + 2 * t;
    const uint32_t ring = smem_u32(smem), x_at = smem_u32(xh) + b * 4 * ps * 16, xs_at = smem_u32(xsc) + b * mt * 4;
    const float gs = NVFP4 ? *a.g : 1.f;
    Scales<MT, NVFP4, G> sc;                     // loaded by the lanes one stage ahead unless they come with it
    if (!TS) load_scales<MT, NVFP4, G>(a, blockIdx.y * kR + wrow, 2 * s0 + b, lane, sc);
    bool staged = false;
    int buf = 0, slot = 0;
    uint32_t phase = 0;
    for (int tile = blockIdx.y; tile < tiles; tile += gridDim.y, buf ^= 1) {
        float acc[MT][NT][4];
#pragma unroll
        for (int h = 0; h < MT; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[h][n][e] = 0.f;
        for (int p0 = s0; p0 < s1; p0 += sh.st_pass) {
            const int pe = min(p0 + sh.st_pass, s1);
            if (!staged) {
                named_bar(1, kConsThreads);
                stage_x<NVFP4>(a, xh, xsc, m0, mt, 2 * p0, 2 * (pe - p0), sh.vec != 0);
                named_bar(1, kConsThreads);
                staged = s1 - s0 <= sh.st_pass;
            }
            uint32_t x = x_at, xs = xs_at;
            for (int st = p0; st < pe; ++st) {
                Scales<MT, NVFP4, G> cur;
                if (!TS) {
                    cur = sc;
                    const bool more = st + 1 < s1;
                    const int nt = more ? tile : tile + (int)gridDim.y;
                    if (nt < tiles) load_scales<MT, NVFP4, G>(a, nt * kR + wrow, 2 * (more ? st + 1 : s0) + b, lane, sc);
                }
                wait_full(&full[slot], phase, bad);
                const uint32_t stage = ring + slot * kSt;
                mul_block<NT, MT, NVFP4, G, TS>(a, stage + code_at, stage + scale_at, lane, cur, x, xs, ps * 16, tok, col, acc);
                x += 8 * ps * 16;
                xs += 2 * mt * 4;
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);
                if (++slot == R) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        // The sums meet at the part that owns the row, 1 / parts of the tile's:
        // [source part][K-warp][own row], added there in that order; then the
        // tensor scale and the bias. The barrier also tells that every CTA is
        // done reading the other buffer's last tile.
        const uint32_t sums = smem_u32(red) + buf * (parts * 2 * own * MP * 4);
        if (parts > 1 && tile == (int)blockIdx.y) cluster_wait();  // every CTA of the cluster runs
        if (*bad) {                              // a wait that gave up: the rows' owners store NaN
#pragma unroll
            for (int h = 0; h < MT; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[h][n][e] = NAN;
        }
#pragma unroll
        for (int h = 0; h < MT; ++h)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int r = wrow + 16 * h + g + 4 * e, p = r / own;
                const uint32_t at = sums + (((part * 2 + b) * own + r - p * own) * MP + 2 * t) * 4;
                uint32_t ra = at;
                if (parts > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(at), "r"(p));
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n * 8 + 2 * t >= mt) continue;
                    if (parts > 1)
                        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(ra + n * 32), "f"(acc[h][n][e]), "f"(acc[h][n][e + 1]) : "memory");
                    else
                        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(ra + n * 32), "f"(acc[h][n][e]), "f"(acc[h][n][e + 1]) : "memory");
                }
            }
        if (parts > 1) {
            cluster_arrive();
            cluster_wait();
        } else {
            named_bar(1, kConsThreads);
        }
        store_tile(a, red + buf * (parts * 2 * own * MP), parts, own, part, MP, m0, mt, tile * kR, kR, gs);
    }
    if (parts > 1) {                             // no CTA leaves while another may still write to it
        cluster_arrive();
        cluster_wait();
    }
}

std::atomic<int> w4_hold{0};

bool code_map(CUtensorMap *tm, const void *base, uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t box_rows,
              bool swizzle) {
    auto enc = get_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of 1 to 8 CTAs with `smem` bytes each that the device holds at once, as
// n[1 .. 8]; asked for once per kernel and device. (Fewer than the SMs suggest: a
// cluster's CTAs lie in one group of SMs.)
constexpr int kMaxDevices = 64;
struct Clusters {
    std::atomic<int> n[kMaxDevices][9];
};
cudaError_t resident_clusters(const void *kern, size_t smem, int dev, Clusters &known, int (&n)[9]) {
    for (int p = 1; p <= 8; ++p) {
        n[p] = dev < kMaxDevices ? known.n[dev][p].load(std::memory_order_relaxed) : 0;
        if (n[p] > 0) continue;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(p, 1024);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = p;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n[p], kern, &cfg);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) known.n[dev][p].store(n[p], std::memory_order_relaxed);
    }
    return n[1] > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int NT, int MT, int CPS, bool NVFP4, int G, bool TS>
cudaError_t launch_one(const W4Args &a, cudaStream_t st) {
    static std::atomic<uint64_t> attr_set{0};
    const auto kern = linear_w4_kernel<NT, MT, CPS, NVFP4, G, TS>;
    cudaError_t e = set_smem_limit_once((const void *)kern, 226 * 1024, attr_set);
    if (e != cudaSuccess) return e;
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    CUtensorMap tq, ts;
    constexpr int R = kRows<MT>;
    if (!code_map(&tq, a.q, a.N, a.K / 2, 64, R, !NVFP4)) return cudaErrorInvalidValue;
    Shape sh{};
    ts = tq;
    if (TS && !code_map(&ts, a.s, a.N, a.K / 16, 16, R, false)) return cudaErrorInvalidValue;
    const int mb = (a.M + 8 * NT - 1) / (8 * NT), mt = (a.M + mb - 1) / mb;
    sh.tokens = mt;
    const int nst = (a.K + 255) / 256, tiles = (a.N + R - 1) / R;
    // the shared memory of a CTA where CPS of them share an SM's (131072 x 4096, 1
    // token: a ring of 4 stages in 113 KB 54.6 us, of 3 in 112 KB 56.3)
    constexpr int kSt = kStage<MT, TS>, kRoom = CPS == 2 ? 113 * 1024 : 225 * 1024, kBars = 16 * 8 + 16;
    const int xst = 8 * pair_stride(mt) * 16 + 8 * mt;  // bytes of x and its scales for one stage
    auto sums_bytes = [&](int p) { return (p * 4 * ((R + p - 1) / p) * (8 * NT + 2) * 4 + 15) / 16 * 16; };
    static Clusters known;
    int resident[9];
    if ((e = resident_clusters((const void *)kern, kRoom, dev, known, resident)) != cudaSuccess) return e;
    // K in 1 to 8 parts: the fewest stages that one of the resident CTAs takes, a
    // tile's start and sum counted as four, and half as many again where x does not
    // fit beside two stages and is staged anew for every tile
    sh.parts = 1;
    int64_t best = INT64_MAX;
    for (int p = 1; p <= 8 && 2 * p <= nst + 1; ++p) {
        const int st = (nst + p - 1) / p;
        if (resident[p] < 1) continue;
        int64_t per = ((int64_t)tiles * mb + resident[p] - 1) / resident[p] * (st + 4);
        if (st * xst + sums_bytes(p) + 2 * kSt + kBars > kRoom) per += per / 2;
        if (per < best) {
            best = per;
            sh.parts = p;
        }
    }
    // each CTA stages its part of x once and walks the row tiles
    int gy = resident[sh.parts] / mb;
    gy = gy < 1 ? 1 : gy > tiles ? tiles : gy;
    const int part_st = (nst + sh.parts - 1) / sh.parts;
    const int sums = sums_bytes(sh.parts);
    sh.st_pass = (kRoom - sums - 2 * kSt - kBars) / xst;
    if (sh.st_pass > part_st) sh.st_pass = part_st;
    sh.ring = (kRoom - sums - kBars - sh.st_pass * xst) / kSt;
    if (sh.ring > 8) sh.ring = 8;
    const int es = a.x_type == MOE_T_E4M3 ? 1 : 2;
    sh.vec = (uintptr_t)a.x % (8 * es) == 0 && (a.x_ld * es) % (8 * es) == 0;
    sh.hold = w4_hold.load(std::memory_order_relaxed);
    sh.bars = (sh.ring * kSt + sums + sh.st_pass * xst + 7) / 8 * 8;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sh.parts, gy, mb);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sh.bars + 16 * 8 + 8;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = sh.parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    // The start overlaps the end of the kernel before where a CTA takes one
    // tile (0.5 us of 6 to 14); CTAs that stay would share their SM with it
    // (131072 x 4096, 4 tokens: 62 -> 70 us).
    cfg.numAttrs = gy == tiles ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, tq, ts, a, sh);
}

template <int NT, int MT, int CPS>
cudaError_t launch_fmt(const W4Args &a, cudaStream_t st) {
    if (a.nvfp4) {
        // TMA takes the scales where their rows are multiples of 16 bytes
        if (a.K % 256 == 0 && (uintptr_t)a.s % 16 == 0) return launch_one<NT, MT, CPS, true, 16, true>(a, st);
        return launch_one<NT, MT, CPS, true, 16, false>(a, st);
    }
    if (a.group == 128) return launch_one<NT, MT, CPS, false, 128, false>(a, st);
    if (a.group == 64) return launch_one<NT, MT, CPS, false, 64, false>(a, st);
    return launch_one<NT, MT, CPS, false, 32, false>(a, st);
}

}  // namespace

void hold_linear_w4(bool hold) { w4_hold.store(hold, std::memory_order_relaxed); }

// Reads and clears the current device's error bits, after `st`'s work.
cudaError_t linear_w4_errors(cudaStream_t st, uint32_t *bits) {
    void *at = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&at, w4_err);
    return e == cudaSuccess ? take_error_bits((uint32_t *)at, st, bits) : e;
}

cudaError_t launch_linear_w4(const W4Args &a, cudaStream_t st) {
    // 32 rows a warp (each x fragment serves two products), where their sums fit in
    // the registers of two CTAs on an SM (up to 8 tokens) or of one (over 16); one
    // CTA also holds twice the x, which is then rarely staged anew for every tile
    // (41 tokens, 7684 x 6816: 81 us with 16 rows and two CTAs, 40 us so).
    // Few rows: tiles of 64 where 8 parts of 128-row tiles would leave half of the
    // CTAs' places empty (1 token, 2081 x 8960 NVFP4: 7.5 -> 6.2 us, 7 tokens, 415 x
    // 9856 INT4: 8.6 -> 7.4; but 4096 x 4096 INT4 6.7 -> 7.3, 131072 x 4096 61 -> 73).
    if (a.M <= 8) return a.N <= 128 * 152 / 8 ? launch_fmt<1, 1, 2>(a, st) : launch_fmt<1, 2, 2>(a, st);
    // In between it is the length of a CTA's work that decides, since a lone CTA
    // waits at every tile's start and sum. 16 tokens, two CTAs / one, us: 8192 x 4096
    // INT4 17.4 / 15.5, 8192 x 4096 8-bit x 13.1 / 11.4, 32768 x 4096 f16 x 35.1 /
    // 32.9; but 43485 x 2048 INT4 34.1 / 37.8, 2048 x 12288 11.6 / 12.7, 512 x 4096
    // 5.3 / 5.8.
    if (a.M <= 16) return a.K >= 4096 && a.N >= 4096 ? launch_fmt<2, 2, 1>(a, st) : launch_fmt<2, 1, 2>(a, st);
    if (a.M <= 24 || (a.M > 32 && a.M <= 48)) return launch_fmt<3, 2, 1>(a, st);
    return launch_fmt<4, 2, 1>(a, st);
}

}  // namespace moe
