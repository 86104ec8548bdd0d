// ops.cuh — arguments and launchers of the operators around the expert layer:
// routing from logits (route_logits.cu), residual + RMSNorm with an 8-bit
// output (norm_quant.cu), products with 4-bit weights (linear_w4.cu), 4-bit
// floats (quant_fp4.cu) and products of two such matrices (linear_fp4.cu), and
// products grouped by expert (grouped_linear.cu, linear_fp4.cu). Their C entries
// are in ops_api.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

constexpr int kRouteMaxE = 512;
constexpr int kRouteMaxK = 16;
constexpr int kRouteMaxGroups = 32;
constexpr int kRouteMaxT = 1 << 18;
constexpr int kRouteMaxChunks = 304;   // two CTAs on each of 152 SMs
constexpr int kRouteFusedChunks = 8;   // batches of up to 8 times 32 tokens run as one launch

struct RouteArgs {
    const void *logits;      // [T, E], rows `stride` elements apart; nsplit slices to be summed in order
    int64_t stride, split_stride;
    int nsplit;
    moe_dtype type;
    int T, E, k;
    bool sigmoid;
    const float *bias;       // [E] or null: added to the score for the choice only
    int groups, keep;        // keep == groups: no group stage
    bool top2;               // group score: sum of the two best choices, else the best
    bool renorm;
    float scale;
    int32_t *ids;            // [T, k]
    float *w;
    int32_t *counts, *offsets, *perm, *pos;  // any may be null
    uint16_t *chunk_cnt;     // scratch of route_scratch_bytes, 16-byte aligned
    int chunk;               // tokens per CTA (set by the launcher)
    int32_t perm_fill;       // written to the rows of perm past the last pair
    // of a layer's workspace (null otherwise): used experts, 128-row tile offsets and their counts
    int32_t *uniq, *tile_off, *n_uniq, *n_tiles;
    uint32_t group_inv;      // ceil(2^22 / (E / groups)) (this and the next four set by the launcher)
    int lanes_per_group;     // a power of two, at most 32 / groups
    bool direct;             // the groups are whole lanes: lanes_per_group of them each
    bool vec_bias;           // the bias may be read as 16-byte vectors
    bool vec;                // a lane's logits may be read as 16-byte (or smaller) vectors
};

// Tokens of a chunk: 32, or a multiple of 16 that makes kRouteMaxChunks of them.
inline int route_chunk_tokens(int T) {
    const int c = (T + kRouteMaxChunks - 1) / kRouteMaxChunks;
    return c <= 32 ? 32 : (c + 15) / 16 * 16;
}
// The counts of every chunk, 16 bits each, in rows of E rounded up to 8.
inline size_t route_scratch_bytes(int T, int E) {
    const int c = route_chunk_tokens(T), rows = (T + c - 1) / c;
    return rows <= kRouteFusedChunks ? 0 : sizeof(uint16_t) * (size_t)rows * ((E + 7) & ~7);
}

// route_logits.cu; T >= 1. *launches (may be null) is advanced by the launches made.
cudaError_t launch_route_logits(RouteArgs a, cudaStream_t st, int *launches);

struct NormArgs {
    const void *x, *res, *gain;  // [T, d], [T, d] or null, [d] or null, all of `type`
    void *sum, *out;             // sum may be null
    float *scales;               // [T, d / group] (E4M3 output)
    int64_t x_ld, res_ld, sum_ld, out_ld, scales_ld;  // elements from one row to the next
    int T, d, group;             // group divides d
    float eps;
    moe_dtype type;
    bool e4m3;                   // out is E4M3 with scales, else of `type`
};
constexpr int kNormMaxD = 16384;
cudaError_t launch_add_rmsnorm(const NormArgs &a, cudaStream_t st);

struct W4Args {
    const uint8_t *q;        // [N, K/2]
    const void *s;           // NVFP4: [N, K/16] E4M3; INT4: [N, K/group] f16 or bf16
    const float *g;          // NVFP4: one fp32 scale
    const uint8_t *z;        // INT4: [N, K/group] zero points, or null (8)
    const void *x;           // [M, K]
    const float *xs;         // E4M3 x: [M, K/xgroup]
    const float *bias;       // [N] or null
    void *y;                 // [M, N]
    int64_t x_ld, xs_ld, y_ld;
    int M, N, K, group, xgroup;
    bool nvfp4;
    moe_dtype s_type, x_type, y_type;
};
constexpr int kW4MaxM = 64;
constexpr int kW4MaxK = 32768;
constexpr int kW4MaxN = 1 << 30;
cudaError_t launch_linear_w4(const W4Args &a, cudaStream_t st);
cudaError_t linear_w4_errors(cudaStream_t st, uint32_t *bits);
// Reads a device's error bits and clears those it has read, after `st`'s work: a bit that a kernel on another stream sets
// meanwhile stays for the next to read.
cudaError_t take_error_bits(uint32_t *word, cudaStream_t st, uint32_t *bits);
void hold_linear_w4(bool hold);

// Microscaled 4-bit floats (quant_fp4.cu): two e2m1 codes to a byte, the low
// nibble first; NVFP4: an E4M3 scale per 16 and a second, fp32 scale; MXFP4: a
// power of two per 32, as its biased exponent.
struct QuantFp4Args {
    const void *x, *up;      // [T, K] of `type`; up may be null
    int64_t x_ld, up_ld;
    const int32_t *rows;     // [R] or null (R == T)
    int T, R, K;
    uint8_t *q, *s;          // [R, K/2], [R, K/16 or K/32]
    float *g;                // [R] (NVFP4)
    moe_dtype type;
    bool nvfp4;
    bool vec;                // rows of x (and up) may be read as 32-byte vectors (set by the launcher)
};
struct DequantFp4Args {
    const uint8_t *q, *s;
    const float *g;          // NVFP4: [R] or [1]; null: 1
    bool g_rows;
    int R, K;
    void *out;               // [R, K]
    int64_t out_ld;
    moe_dtype type;
    bool nvfp4;
    bool vec;                // rows of out may be written as 32-byte vectors (set by the launcher)
};
constexpr int kFp4MaxK = 32768;
struct GatherFp4Args {
    const uint8_t *q_from, *s_from;
    const float *g_from;
    const int32_t *rows;     // [R]
    int T, R, q_bytes, s_bytes;
    uint8_t *q, *s;
    float *g;                // or null
};
// scratch: 16-byte aligned, of at least quantize_fp4_scratch's bytes, or null
size_t quantize_fp4_scratch(const QuantFp4Args &a);
cudaError_t launch_quantize_fp4(QuantFp4Args a, uint8_t *scratch, cudaStream_t st);
cudaError_t launch_dequantize_fp4(DequantFp4Args a, cudaStream_t st);

// Products of rows grouped by expert (products.cuh).
constexpr int kProdMaxGroups = 512;
constexpr int kProdMaxRows = 1 << 24;
struct ProdArgs {
    int groups;
    const int32_t *offsets;  // [groups + 1], or null: one group of all M rows
    int M, N, K;
    bool bf16;               // 16-bit operands: bf16, else f16
    const uint8_t *xs, *ws;  // 4-bit operands: block scales of x [M] and of the weights [groups, N]
    const float *xg;         // [M] or null
    const float *wg;         // [groups], or [groups, N] with wg_cols, or null
    bool wg_cols;
    const float *bias;       // [groups, N] or null
    void *y;                 // [M, N]
    int64_t y_ld;
    moe_dtype y_type;
    int ks;                  // parts of K, each a CTA of a cluster (set by the launcher)
    bool wide;               // y takes 16-byte stores (set by the launcher)
    int s_copy;              // alignment of the scales' rows: 16, 4 or 2 (set by the launcher)
    int hold;                // test hook (set by the launcher)
};
cudaError_t launch_grouped_linear(const ProdArgs &a, const void *x, int64_t x_ld, const void *w, cudaStream_t st);
cudaError_t launch_linear_fp4(ProdArgs a, bool nvfp4, const uint8_t *xq, const uint8_t *wq, cudaStream_t st);
cudaError_t products_errors(cudaStream_t st, uint32_t *bits);
void hold_products(int hold);

#ifdef __CUDACC__

// Programmatic dependent launch: `wait` returns once the grids before this one
// in the stream have completed and their writes are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Two floats by one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 o;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(o.x), "=f"(o.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return o;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 o;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(o.x), "=f"(o.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return o;
}

#endif

}  // namespace moe
