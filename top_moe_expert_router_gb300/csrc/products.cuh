// products.cuh — y[r] = W[e(r)] x[r] + b[e(r)]: products of rows that are grouped
// by expert (or belong to one matrix) on the 5th-generation tensor cores, with
// operands in 16 bits (grouped_linear.cu) or in microscaled 4-bit floats
// (linear_fp4.cu).
//
// The weights are the M = 128 operand of tcgen05.mma and the rows of a group the
// N operand, in steps of 16 up to TN: a group of 5 rows costs 16, not 128, which
// is what ragged groups and decode batches need, and a tile of weights is read
// once for up to TN rows. Both operands are K-major tiles of 128-byte rows (64
// columns of 16 bits, 256 of 4) brought by TMA through a ring; accumulators in
// tensor memory, two of them, so that one tile is stored while the next is
// summed. Tiles are dealt to persistent CTAs in an order that the offsets on the
// device determine: group by group, in bands of 12 weight tiles, so that the
// CTAs running at a time share weight and row tiles in L2.
//
// With few rows and few tiles K is split over a cluster of CTAs, whose sums meet
// in distributed shared memory; with many rows a pair of CTAs shares a tile of
// 256 weight rows (cta_group::2), each with half of the rows of x in its shared
// memory.
//
// Warps: 0 TMA, 1 MMA (owns the tensor memory), 2..9 epilogue, and for 4-bit
// operands 18 and 19, which bring the block scales to shared memory, and 10..17,
// which bring them from there to tensor memory: the layout there is lane r % 32,
// column r / 32 for row r, the scale bytes of one MMA (K = 64) in a column, the
// same in all four lane quarters.
//
// What bounds it: with few rows, or ragged groups, the stream of the weights
// (32768 rows by 256 experts of 1536 x 4096: bf16 530 us, NVFP4 165 us, 1.00 and
// 0.96 of the copy rate); with many, 16 bits: the MMAs (4096 x 8192 x 4096 bf16
// 143 us, 1.92 PFLOP/s); 4 bits: issue slots, with short K those of the epilogue (8192
// x 4096 x 512 NVFP4 28 us, 15 without results). The warp that issues the MMAs has 200
// ns for a stage, and shares its scheduler with two that bring scales and two of
// the epilogue (4096 x 8192 x 8192 NVFP4 98 us, 5.6 PFLOP/s; without the scales 82
// us, without the stores 88, without both 73, without loads and both 70; without
// loads alone 96; MXFP4, which fills as many columns of tensor memory with half of the
// scales, 105). The MMAs are those of K = 64; sm_103a also has dense ones of K = 96, half as
// much work again for an instruction, which are not used here. Tried there: the warps with the scales waiting for the operands
// too, so that the MMAs take one wait and one commit a stage (110 us), waits that
// spin (103 to 121 us).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "gemm.cuh"
#include "ops.cuh"

namespace moe {

enum { PROD_16 = 0, PROD_NVFP4 = 1, PROD_MXFP4 = 2 };

constexpr int kProdRows = 128;           // weight rows of a tile
constexpr int kProdBand = 12;            // weight tiles of a band
constexpr uint32_t kProdABytes = kProdRows * 128;

int products_held();                     // test hook: 1 copy no operands, 2 every second CTA copies none

#ifdef __CUDACC__

// Error bits of this device's products (of one translation unit).
static __device__ uint32_t prod_err;

// Reads and clears the bits of the current device, after `st`'s work.
static inline cudaError_t prod_take_errors(cudaStream_t st, uint32_t *bits) {
    void *at = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&at, prod_err);
    return e == cudaSuccess ? take_error_bits((uint32_t *)at, st, bits) : e;
}

// Floats from one column of partial sums to the next: 32 rows, and 4 against bank conflicts.
constexpr int kPartRow = 36;
constexpr int kNoTile = 0x7FFFFFFF;
constexpr int kMostParts = 4;            // of K, CTAs of a cluster
// columns of partial sums that a CTA receives for a tile, at most: of ks parts (ks - 1) 4 ceil(32 / ks)
constexpr int kPartCols = 96;
static_assert((kMostParts - 1) * 4 * ((32 + kMostParts - 1) / kMostParts) <= kPartCols, "partial sums");

// CG: CTAs of a tile, 1 or 2 (a pair, 256 weight rows)
template <int KIND, int TN, int CG>
struct ProdShape {
    static constexpr bool kFp4 = KIND != PROD_16;
    static constexpr int kShare = TN / CG;                   // rows of x in a CTA's shared memory
    static constexpr int kBox = kShare % 64 ? 32 : 64;       // rows of one TMA copy of x
    static constexpr int kStep = 16 * CG;                    // the N of an MMA is a multiple
    static constexpr uint32_t kStage = kProdABytes + kShare * 128;
    // scales come kBatch stages at a time: 32 bytes of a row (of MXFP4 16), a whole sector. (Four stages at a time in two
    // slots, with one tile stage less: the same time.)
    static constexpr int kBatch = 2;
    static constexpr int kBatchBytes = (KIND == PROD_NVFP4 ? 16 : 8) * kBatch;
    static constexpr int kScaleRows = kProdRows + TN;
    static constexpr int kBatches = kFp4 ? 3 : 0;            // such batches in the ring
    // (rows that begin on odd words of 16 bits lie 24 bytes apart)
    static constexpr int kSlotBytes = kScaleRows * (KIND == PROD_NVFP4 ? kBatchBytes : 24);
    static constexpr uint32_t kScales = kFp4 ? kBatches * kSlotBytes : 0;
    static constexpr int kScaleBox = TN % 64 ? 32 : 64;      // rows of one TMA copy of x's scales
    // results on their way to 16-byte stores: 32 rows x 128 columns of 16 bits for each half of the epilogue's warps
    static constexpr bool kWide = TN > 32;
    static constexpr int kOutBufs = kFp4 ? 2 : 1;            // (with 16 bits a stage more is worth more)
    static constexpr uint32_t kOut = kWide ? kOutBufs * 2 * 32 * 256 : 0;
    // K may be split over a cluster of CTAs: the sums that the others bring for this CTA's share of the columns, of two tiles
    static constexpr bool kSplit = CG == 1 && TN == 32;
    static constexpr uint32_t kParts = kSplit ? 2 * kPartCols * kPartRow * 4 : 0;
    static constexpr uint32_t kMeta = kProdMaxGroups * 16 + 16 + 512 + 256;  // group tables, barriers, scratch of 64 words
    static constexpr int kRoom = (int)((227 * 1024 - 1024 - kMeta - kScales - kOut - kParts) / kStage);
    static constexpr int kStages = kRoom < 10 ? kRoom : 10;
    static constexpr uint32_t kSmem = 1024 + kStages * kStage + kScales + kOut + kParts + kMeta;
    static constexpr int kThreads = kFp4 ? 640 : 320;
    // tensor memory: two accumulators, then up to four buffers of scales (16 columns for the weights, kBCols for each of
    // the four MMAs of a stage for x)
    static constexpr int kBCols = TN > 128 ? TN / 32 : 4;
    static constexpr uint32_t kScaleCols = 16 + 4 * kBCols;
    static constexpr uint32_t kScaleAt = 2 * TN;
    static constexpr int kScaleRoom = (int)((kTmemCols - kScaleAt) / kScaleCols);
    static constexpr int kScaleBufs = !kFp4 ? 1 : kScaleRoom < 4 ? kScaleRoom : 4;
    static_assert(!kFp4 || kScaleAt + kScaleBufs * kScaleCols <= kTmemCols, "tensor memory");
    static_assert(2 * TN <= (int)kTmemCols, "tensor memory");
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap *tm) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}

// One lane of a warp whose 32 lanes are here. The roles that issue TMA copies and
// MMAs run as whole warps, with the instructions predicated on that lane: their
// operands then stay in uniform registers, where the instructions want them. One
// lane alone in a branch moves each operand there first: an MMA of 64 columns or
// fewer took 116 cycles so and takes 55, a stage of four with its wait 465 and 250.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

#define MOE_MMA_16(CGS)                                                        \
    asm volatile(                                                              \
        "{\n\t.reg .pred p, q;\n\t"                                        \
        "setp.ne.b32 p, %4, 0;\n\t"                                          \
        "setp.ne.b32 q, %5, 0;\n\t"                                          \
        "@q tcgen05.mma.cta_group::" CGS ".kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), \
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)                          \
        : "memory")
#define MOE_MMA_FP4(CGS, KINDS)                                                \
    asm volatile(                                                              \
        "{\n\t.reg .pred p, q;\n\t"                                        \
        "setp.ne.b32 p, %6, 0;\n\t"                                          \
        "setp.ne.b32 q, %7, 0;\n\t"                                          \
        "@q tcgen05.mma.cta_group::" CGS "." KINDS " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), \
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc), "r"(on)        \
        : "memory")

template <int CG>
__device__ __forceinline__ void mma_16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t on) {
    if constexpr (CG == 1)
        MOE_MMA_16("1");
    else
        MOE_MMA_16("2");
}

template <int KIND, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                        uint32_t acc, uint32_t on) {
    if constexpr (KIND == PROD_NVFP4 && CG == 1)
        MOE_MMA_FP4("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (KIND == PROD_NVFP4)
        MOE_MMA_FP4("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (CG == 1)
        MOE_MMA_FP4("1", "kind::mxf4.block_scale.scale_vec::2X");
    else
        MOE_MMA_FP4("2", "kind::mxf4.block_scale.scale_vec::2X");
}
#undef MOE_MMA_16
#undef MOE_MMA_FP4

// Arrives at `bar`, with CG = 2 at that of both CTAs, once the MMAs so far are done.
template <int CG>
__device__ __forceinline__ void commit_on(uint64_t *bar, uint32_t on) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
            "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(
                smem_u32(bar)),
            "r"(on), "h"((uint16_t)3)
            : "memory");
}

// The address of this CTA's shared word in the CTA of rank 0.
__device__ __forceinline__ uint32_t in_leader(const void *p) {
    uint32_t o;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(o) : "r"(smem_u32(p)));
    return o;
}

// One arrival of the warp, whose lanes' work so far it covers, at the leader's barrier.
template <int CG>
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) != 0) return;
    if constexpr (CG == 1)
        mbar_arrive(bar);
    else
        // what this orders between the CTAs lies in tensor memory, by the fences beside it; an arrival and a wait that
        // ordered memory across the cluster would empty the L1 each time (8192 x 16384 x 8192 NVFP4: 1158 us)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(in_leader(bar)) : "memory");
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync_all() {
    cluster_arrive();
    cluster_wait();
}

__device__ __forceinline__ void expect_on(uint64_t *bar, uint32_t bytes, uint32_t on) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "r"(bytes), "r"(on)
        : "memory");
}

// `bar`: an address in the cluster's shared memory (with CG = 2 the leader's).
template <int CG>
__device__ __forceinline__ void tma_on(uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar, uint32_t on) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "r"(on)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void prod_tmem_alloc(uint32_t *slot) {
    if constexpr (CG == 1) {
        tmem_alloc(slot, kTmemCols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void prod_tmem_free(uint32_t at) {
    if constexpr (CG == 1)
        tmem_dealloc(at, kTmemCols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(kTmemCols) : "memory");
}

__device__ __forceinline__ bool warp_wait_loop(uint64_t *bar, uint32_t parity, uint32_t *err, volatile int *abort) {
    const unsigned long long t0 = global_ns();
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
        if ((it & 255u) == 0) {
            const bool late = global_ns() - t0 > kWaitLimitNs;
            if (late) {
                atomicOr(err, ERRBIT_TIMEOUT);
                *abort = 1;
            }
            if (__any_sync(0xFFFFFFFFu, late || *abort)) return false;
        }
    }
}

static __device__ __noinline__ bool warp_wait_called(uint64_t *bar, uint32_t parity, uint32_t *err, volatile int *abort) {
    return warp_wait_loop(bar, parity, err, abort);
}

// A bounded wait of a whole warp, with one answer for its lanes: false once the limit has passed or another warp of the
// CTA gave up. (CALL: what a wait that is not over at once runs is a function. With two waits a stage, as with 4-bit
// operands, that is faster: 4096 x 8192 x 8192 NVFP4 105 -> 100 us; with one it is slower: a stage of 16 bits and 32
// rows 111 -> 142 ns.)
template <bool CALL>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t *err, volatile int *abort) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    return CALL ? warp_wait_called(bar, parity, err, abort) : warp_wait_loop(bar, parity, err, abort);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t v[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t v[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Asynchronous copy of N bytes to shared memory, of which the first `size` are read and the others zeros.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, int size) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(size) : "memory");
}
// Arrives at `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The groups that have rows, as the tiles need them, in shared memory.
struct ProdGroups {
    int32_t *start;          // [n + 1] first tile of each
    int32_t *row0;           // [n]
    int32_t *rows, *group;   // [n]
    int n;
};

struct ProdTile {
    int g, w, row0, rows;    // group, weight tile, first row and rows (up to TN)
};

// The tile of the given number; i: its place among the groups, which only grows.
template <int TN>
__device__ __forceinline__ ProdTile prod_tile(const ProdGroups &gr, int nw, int tile, int &i) {
    if (gr.start[i + 1] <= tile) {               // the last group that starts at or before the tile
        int lo = i + 1, hi = gr.n;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (gr.start[mid] <= tile)
                lo = mid;
            else
                hi = mid;
        }
        i = lo;
    }
    const int local = tile - gr.start[i], rows = gr.rows[i], nt = (rows + TN - 1) / TN;
    const int band = local / (kProdBand * nt), r = local - band * (kProdBand * nt);
    const int bw = min(kProdBand, nw - band * kProdBand), t = r / bw;
    ProdTile p;
    p.g = gr.group[i];
    p.w = band * kProdBand + r - t * bw;
    p.row0 = gr.row0[i] + t * TN;
    p.rows = min(TN, rows - t * TN);
    return p;
}

// Walks a CTA's tiles in order.
template <int TN>
struct ProdWalk {
    int tile, i;             // i: of the groups with rows
    __device__ __forceinline__ explicit ProdWalk(int first) : tile(first), i(0) {}
    __device__ __forceinline__ ProdTile at(const ProdGroups &gr, int nw) { return prod_tile<TN>(gr, nw, tile, i); }
};

// Fills the tables; every thread of the CTA, one or two groups each. -> the number of tiles, 0 where offsets that run
// backwards make them more than M rows can have: a ragged tile a group and M / TN full ones
template <int TN>
__device__ __forceinline__ int prod_groups(const ProdArgs &a, ProdGroups &gr, int nw, int32_t *scratch) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    int lo[2], rows[2], tiles[2], used = 0;
    long long sum = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int g = 2 * t + j;
        lo[j] = rows[j] = 0;
        if (g < a.groups) {
            // whatever the offsets hold, no row outside [0, M) is touched
            int hi = a.M;
            if (a.offsets) {
                lo[j] = min(max(a.offsets[g], 0), a.M);
                hi = min(max(a.offsets[g + 1], lo[j]), a.M);
            }
            rows[j] = hi - lo[j];
        }
        tiles[j] = (rows[j] + TN - 1) / TN * nw;
        sum += tiles[j];
        used += rows[j] > 0;
    }
    long long end = sum;
    int last = used;                             // inclusive sums over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, end, o);
        const int u = __shfl_up_sync(0xFFFFFFFFu, last, o);
        if (lane >= o) end += v, last += u;
    }
    if (lane == 31) {
        reinterpret_cast<long long *>(scratch)[warp] = end;
        scratch[40 + warp] = last;
    }
    __syncthreads();
    long long all = 0;
    int n = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        if (w == warp) end += all, last += n;
        all += reinterpret_cast<const long long *>(scratch)[w];
        n += scratch[40 + w];
    }
    if (all > ((long long)a.M / TN + min(a.groups, a.M)) * nw) all = n = 0;
    int at = (int)(end - sum), i = last - used;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (rows[j] > 0 && n) {
            gr.start[i] = at;
            gr.row0[i] = lo[j];
            gr.rows[i] = rows[j];
            gr.group[i] = 2 * t + j;
            at += tiles[j];
            ++i;
        }
    if (t == 0) gr.start[n] = (int)all;
    gr.n = n;
    __syncthreads();
    return (int)all;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t v[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 rounded(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half rounded(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float rounded(float v) { return v; }

__device__ __forceinline__ void store_one(void *y, int64_t at, moe_dtype t, float v) {
    if (t == MOE_T_BF16)
        ((__nv_bfloat16 *)y)[at] = rounded<__nv_bfloat16>(v);
    else if (t == MOE_T_F16)
        ((__half *)y)[at] = rounded<__half>(v);
    else
        ((float *)y)[at] = v;
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t v[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(taddr));
}

// What a tile's results are multiplied by and added to, read before they are waited for: this thread's column (scale
// and bias), and the scales of rows lane, lane + 32, ...
template <bool FP4, int TN>
struct ProdScales {
    float col, bias, row[FP4 ? TN / 32 : 1];
    __device__ __forceinline__ ProdScales(const ProdArgs &a, const ProdTile &t, int n) : col(1.f), bias(0.f) {
        const bool mine = n < a.N;
        if (a.bias && mine) bias = a.bias[(int64_t)t.g * a.N + n];
        if constexpr (FP4) {
            if (a.wg && mine) col = a.wg[a.wg_cols ? (int64_t)t.g * a.N + n : t.g];
#pragma unroll
            for (int j = 0; j < TN / 32; ++j) {
                const int r = 32 * j + (threadIdx.x & 31);
                row[j] = a.xg && r < t.rows ? a.xg[t.row0 + r] : 1.f;
            }
        }
    }
};

// A tile's rows: this thread owns column n of y and walks the rows, 32 accumulator columns at a time, every other 32
// (from `half` on).
template <bool FP4, int TN, typename T>
__device__ __forceinline__ void prod_store(const ProdArgs &a, const ProdTile &t, const ProdScales<FP4, TN> &sc, uint32_t tbase,
                                           int n, int half, bool failed) {
    const bool mine = n < a.N;
    T *y = (T *)a.y + (int64_t)t.row0 * a.y_ld + n;
#pragma unroll
    for (int j = 0; j < TN / 32; ++j) {
        if (32 * j >= t.rows) break;
        if ((j & 1) != half) {
            if (j + 1 < TN / 32) y += 32 * a.y_ld;
            continue;
        }
        uint32_t v[32];
        tmem_ld32(tbase + 32 * j, v);
        tmem_ld_wait();
        if constexpr (FP4) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = __float_as_uint(__uint_as_float(v[i]) * (sc.col * __shfl_sync(0xFFFFFFFFu, sc.row[j], i)));
        }
        const int rows = t.rows - 32 * j;
        if (mine && !failed && rows >= 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                *y = rounded<T>(__uint_as_float(v[i]) + sc.bias);
                y += a.y_ld;
            }
        } else if (mine) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (i < rows) *y = rounded<T>(failed ? __int_as_float(0x7FFFFFFF) : __uint_as_float(v[i]) + sc.bias);
                y += a.y_ld;
            }
        }
    }
}

// A tile of up to 32 rows, four at a time in a loop that stays one: with a tile or two for a CTA, what the stores take is
// the time to fetch their code.
template <bool FP4>
__device__ __forceinline__ void prod_store_few(const ProdArgs &a, const ProdTile &t, const ProdScales<FP4, 32> &sc, uint32_t tbase,
                                               int n, bool ok) {
    int64_t at = (int64_t)t.row0 * a.y_ld + n;
#pragma unroll 1
    for (int i = 0; i < t.rows; i += 4) {
        uint32_t v[4];
        tmem_ld4(tbase + i, v);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y = ok ? __uint_as_float(v[k]) : __int_as_float(0x7FFFFFFF);
            if constexpr (FP4) y *= sc.col * __shfl_sync(0xFFFFFFFFu, sc.row[0], i + k);
            if (n < a.N && i + k < t.rows) store_one(a.y, at, a.y_type, y + sc.bias);
            at += a.y_ld;
        }
    }
}

// 16 lanes x 32 columns of tensor memory: with t the lane of the warp, v[4c], v[4c + 1] are columns 8c + 2 (t % 4) and the
// next of lane t / 4, v[4c + 2], v[4c + 3] those of lane t / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t v[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

template <typename T>
__device__ __forceinline__ uint32_t rounded2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t rounded2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t rounded2<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// The same for 16-bit results in rows that take 16-byte stores, all 128 columns of the tile inside the matrix: 32 rows at
// a time are transposed through shared memory, so that a row leaves as 256 adjacent bytes instead of 64 from each warp
// (4096 x 8192 x 2048 NVFP4: 51 -> 43 us; two values an instruction 38; two buffers by turns, and so one barrier, 36.6).
// `stage`: 8 KB of this half of the warps, or with 4-bit operands twice that. Rows that begin between 16 bytes gain
// nothing this way: 23383 rows by 129 experts of 3362 x 272 by shifted pieces 112 us, by elements 76.
template <bool FP4, int TN, typename T>
__device__ __forceinline__ void prod_store_wide(const ProdArgs &a, const ProdTile &t, const ProdScales<FP4, TN> &sc,
                                                uint32_t tbase, int n0, int half, bool ok, unsigned char *stage, int &turn) {
    const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
    // this thread's four columns of a fragment: 16 l + 8 h + lane / 4 of the warp's 32
    float col[4], bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        col[i] = FP4 ? __shfl_sync(0xFFFFFFFFu, sc.col, 8 * i + (lane >> 2)) : 1.f;
        bias[i] = __shfl_sync(0xFFFFFFFFu, sc.bias, 8 * i + (lane >> 2));
        if (!ok) bias[i] = __int_as_float(0x7FFFFFFF);
    }
    const int row0 = 8 * q + (lane >> 4), piece0 = lane & 15;  // what it stores: rows row0, row0 + 2, ..
    T *y = (T *)a.y + (int64_t)(t.row0 + row0) * a.y_ld + n0 + 8 * piece0;
    // 16-byte pieces of a row are swapped by the row's low bits, against bank conflicts
    const int mj = lane >> 3, mi = lane & 7;                 // the matrix and row that this lane addresses for stmatrix
#pragma unroll
    for (int j = 0; j < TN / 32; ++j) {
        if (32 * j >= t.rows) break;
        if ((j & 1) != half) continue;
        unsigned char *const buf = FP4 ? stage + turn * 8192 : stage;
        const uint32_t to = smem_u32(buf);
        turn ^= 1;
        uint32_t v[2][16];
        tmem_ld_16x32(tbase + 32 * j, v[0]);
        tmem_ld_16x32(tbase + (16u << 16) + 32 * j, v[1]);
        tmem_ld_wait();
        if (!FP4) named_bar(2 + half, 128);                  // the rows before have left the buffer
        float2 rs[4];                                        // of columns 8 c + 2 (lane % 4) and the next
        if constexpr (FP4) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                rs[c].x = __shfl_sync(0xFFFFFFFFu, sc.row[j], 8 * c + 2 * (lane & 3));
                rs[c].y = __shfl_sync(0xFFFFFFFFu, sc.row[j], 8 * c + 2 * (lane & 3) + 1);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                uint32_t m[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {                // matrix (c + i / 2, h = i % 2)
                    const int cc = c + (i >> 1), at = 4 * cc + 2 * (i & 1), k = 2 * l + (i & 1);
                    float2 o = make_float2(__uint_as_float(v[l][at]), __uint_as_float(v[l][at + 1]));
                    const float2 b2 = make_float2(bias[k], bias[k]);
                    if constexpr (FP4)
                        o = fma2(o, mul2(rs[cc], make_float2(col[k], col[k])), b2);
                    else
                        o = fma2(o, make_float2(1.f, 1.f), b2);
                    m[i] = rounded2<T>(o.x, o.y);
                }
                const int row = 8 * (c + (mj >> 1)) + mi, piece = 4 * q + 2 * l + (mj & 1);
                asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                                 to + row * 256 + ((piece ^ (row & 7)) << 4)),
                             "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3])
                             : "memory");
            }
        }
        named_bar(2 + half, 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + 2 * i;
            const uint4 o = *reinterpret_cast<const uint4 *>(buf + row * 256 + ((piece0 ^ (row & 7)) << 4));
            if (32 * j + row < t.rows) *reinterpret_cast<uint4 *>(y + (32 * j + 2 * i) * a.y_ld) = o;
        }
    }
}

// The address of this CTA's shared word in the CTA of the given rank.
__device__ __forceinline__ uint32_t in_rank(const void *p, int rank) {
    uint32_t o;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(o) : "r"(smem_u32(p)), "r"(rank));
    return o;
}

// A word into the shared memory of another CTA of the cluster.
__device__ __forceinline__ void store_there(uint32_t to, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
}

// Takes bytes that nobody will copy off what a barrier of this CTA waits for.
__device__ __forceinline__ void complete_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

// Four words into the shared memory of another CTA, counted at a barrier there.
__device__ __forceinline__ void send4(uint32_t to, const uint32_t v[4], uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
                 : "memory");
}

// The CTA that adds the sums of the four columns from 4 u on.
__device__ __forceinline__ int part_owner(int u, int ks) { return ((u + 1) * ks - 1) / 32; }

// K split over the ks CTAs of a cluster: each owns a share of the tile's 128 columns, four or a multiple. The sums go to
// the owners as asynchronous stores that a barrier there counts (parts[sender][column of the share][row]); the owners add
// them in the order of their ranks and store. Two such buffers by turns: whoever sends a tile's sums has read, as all
// warps of the CTA have, those of the tile before, so nobody writes where another still reads.
// `lost`: the CTA's tile (lt) whose sums this warp waited for in vain, its limit having passed, or kNoTile. It has sent its own
// for the tiles up to that one, and from then on stays away from the barriers, whose phases no longer fit: arriving at one
// twice in a phase is undefined. (Ordinary stores, which the cluster's last barrier would order, take 0.25 to 0.4 us more a
// tile: 1 x 4096 x 4096 NVFP4 7.9 -> 8.1 us, bf16 8.4 -> 8.7.)
template <bool FP4, int TN>
__device__ __forceinline__ void prod_store_split(const ProdArgs &a, const ProdTile &t, const ProdScales<FP4, TN> &sc,
                                                 uint32_t tbase, int n, bool ok, float *parts, int part, uint64_t *pfull,
                                                 int lt, int &lost, uint32_t *err, volatile int *abort_flag) {
    static_assert(TN == 32, "one chunk of rows");
    bool together = lost == kNoTile;
    const int ks = a.ks, lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3;
    const int local = q * 32 + lane, share = (32 + ks - 1) / ks * 4;
    const int owner = part_owner(local / 4, ks), col = local - 32 * owner / ks * 4;
    const int quads = (t.rows + 3) / 4;
    float *buf = parts + (lt & 1) * (kPartCols * kPartRow);
    uint64_t *bar = pfull + (lt & 1);
    named_bar(2, 128);                           // the tile before the last has been read from this buffer
    if (together && q == 0 && lane == 0) {
        const int own = (32 * (part + 1) / ks - 32 * part / ks) * 4;
        mbar_arrive_expect_tx(bar, (uint32_t)((ks - 1) * own * quads * 16));
    }
    // four rows at a time in loops that stay loops: this code runs once or twice in a kernel, and what it takes is the
    // time to fetch it
    const uint32_t there = in_rank(buf, owner) + (uint32_t)(((part < owner ? part : part - 1) * share + col) * kPartRow * 4);
    const uint32_t bar_there = in_rank(bar, owner);
#pragma unroll 1
    for (int i = 0; i < quads; ++i) {
        uint32_t v[4];
        tmem_ld4(tbase + 4 * i, v);
        tmem_ld_wait();
        if (!ok) v[0] = v[1] = v[2] = v[3] = 0x7FFFFFFFu;
        if (together && owner != part) send4(there + 16 * i, v, bar_there);
    }
    if (together && !warp_wait<true>(bar, (lt >> 1) & 1, err, abort_flag)) {
        together = false;
        lost = lt;
    }
    ok &= together;
    asm volatile(                                // (the same once more, in the scope of the cluster)
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "r"((lt >> 1) & 1)
        : "memory");
    const bool mine = owner == part && n < a.N;
    int64_t at = (int64_t)t.row0 * a.y_ld + n;
#pragma unroll 1
    for (int i = 0; i < quads; ++i) {
        uint32_t v[4];
        tmem_ld4(tbase + 4 * i, v);
        tmem_ld_wait();
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        const float *from = buf + col * kPartRow + 4 * i;
#pragma unroll 1
        for (int r = 0; r < ks; ++r) {
            float4 f = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
            if (r != part) {
                if (mine) f = *reinterpret_cast<const float4 *>(from);
                from += share * kPartRow;
            }
            sum.x += f.x;
            sum.y += f.y;
            sum.z += f.z;
            sum.w += f.w;
        }
        const float o[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y = ok ? o[k] : __int_as_float(0x7FFFFFFF);
            if constexpr (FP4) y *= sc.col * __shfl_sync(0xFFFFFFFFu, sc.row[0], 4 * i + k);
            if (mine && 4 * i + k < t.rows) store_one(a.y, at, a.y_type, y + sc.bias);
            at += a.y_ld;
        }
    }
}

// A pair some of whose waits ran out: waits, one thread of the leader, until the copies of both CTAs have landed. The
// leader has issued those of `mine` stages and counted them and the other's on full[], the other of `theirs`. Where one is
// ahead, the other's share of a stage is taken off what its barrier waits for, or that of the one ahead is added to
// it. (Neither is ahead by more than the ring: a slot is free once an MMA has read it, which takes both.)
template <typename S, int TN>
__device__ __noinline__ void settle_pair(const ProdGroups gr, int nw, int first, int step, int nst, int mine, int theirs,
                                         uint64_t *full, uint32_t *err) {
    const int last = max(mine, theirs);
    for (int j = min(mine, theirs); j < last; ++j) {
        int i = 0;
        const ProdTile t = prod_tile<TN>(gr, nw, first + j / nst * step, i);
        const int share = (t.rows + S::kStep - 1) / S::kStep * 16;
        const uint32_t bytes = kProdABytes + (share + S::kBox - 1) / S::kBox * S::kBox * 128;
        uint64_t *bar = &full[j % S::kStages];
        if (mine > theirs)
            complete_tx(bar, bytes);
        else
            mbar_arrive_expect_tx(bar, bytes);
    }
    for (int j = last > S::kStages ? last - S::kStages : 0; j < last; ++j)
        if (!mbar_wait(&full[j % S::kStages], (j / S::kStages) & 1, err)) break;
}

// The same for K in parts, where the wait for the sums of tile `lost` ran out, one thread of the warp that expects them: until
// what the other CTAs have sent has landed here. Of `lost` all was expected, and what nobody sends is taken off. Of the next
// two tiles what was sent is expected now: others may have had all sums of `lost`, or of the tile after it, but nobody
// those of a third one, which takes sums that follow a wait for the second, and that wait takes this warp. The tiles
// before were waited for.
template <int TN>
__device__ __noinline__ void settle_parts(const ProdGroups gr, int nw, int first, int step, int ntiles, int ks, int part,
                                          int lost, volatile const int *sent, uint64_t *pfull, uint32_t *err) {
    for (int lt = lost; lt < lost + 3 && first + (int64_t)lt * step < ntiles; ++lt) {
        int i = 0;
        const int quads = (prod_tile<TN>(gr, nw, first + lt * step, i).rows + 3) / 4;
        uint32_t all = 0, there = 0;
        for (int r = 0; r < ks; ++r)
            for (int u = 0; u < 32 && r != part; ++u)        // four columns, eight of them a warp's
                if (part_owner(u, ks) == part) {
                    all += quads * 64;
                    there += sent[4 * r + u / 8] > lt ? quads * 64 : 0;
                }
        if (lt > lost && !there) break;
        uint64_t *bar = pfull + (lt & 1);
        if (lt > lost)
            mbar_arrive_expect_tx(bar, there);
        else if (all > there)
            complete_tx(bar, all - there);
        mbar_wait(bar, (lt >> 1) & 1, err);
    }
}

template <int KIND, int TN, int CG>
__global__ void __launch_bounds__(ProdShape<KIND, TN, CG>::kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const __grid_constant__ CUtensorMap tmWS, const __grid_constant__ CUtensorMap tmXS, const ProdArgs a) {
    using S = ProdShape<KIND, TN, CG>;
    constexpr int NS = S::kStages;
    constexpr int kStageK = KIND == PROD_16 ? 64 : 256, kMmaK = kStageK / 4;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t base_u32 = smem_u32(smem_raw);
    unsigned char *smem = smem_raw + (((base_u32 + 1023u) & ~1023u) - base_u32);
    unsigned char *scales = smem + NS * S::kStage;
    unsigned char *staged = scales + S::kScales;
    float *parts = reinterpret_cast<float *>(staged + S::kOut);
    unsigned char *meta = staged + S::kOut + S::kParts;
    uint64_t *full = reinterpret_cast<uint64_t *>(meta), *empty = full + NS;
    uint64_t *tfull = empty + NS, *tempty = tfull + 2, *sfull = tempty + 2, *sempty = sfull + 4;
    uint64_t *lfull = sempty + 4, *lempty = lfull + 4, *pfull = lempty + 4, *done = pfull + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    [[maybe_unused]] volatile int *issued = abort_flag + 1;  // in a pair's leader: stages whose copies the other has issued
    // with K in parts: how many tiles' sums each warp of each other CTA has sent, where one of its waits ran out
    [[maybe_unused]] volatile int *sent = issued + 1;
    [[maybe_unused]] int issued_here = 0, lost = kNoTile;
    const bool held = a.hold == 1 || (a.hold == 2 && (blockIdx.x & 1));
    ProdGroups gr;
    int32_t *scratch = reinterpret_cast<int32_t *>(meta + 512);
    gr.start = scratch + 64;
    gr.row0 = gr.start + kProdMaxGroups + 1;
    gr.rows = gr.row0 + kProdMaxGroups;
    gr.group = gr.rows + kProdMaxGroups;
    static_assert(kProdMaxGroups <= 2 * S::kThreads, "two groups a thread");
    static_assert((2 * NS + 23) * 8 + (3 + 4 * kMostParts) * 4 <= 512, "barriers and words");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t *err = &prod_err;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 8 * CG);
        }
        for (int b = 0; b < S::kScaleBufs; ++b) {
            mbar_init(&sfull[b], 4 * CG);
            mbar_init(&sempty[b], 1);
        }
        for (int b = 0; b < S::kBatches; ++b) {
            mbar_init(&lfull[b], a.s_copy >= 16 ? 1 : 64);
            mbar_init(&lempty[b], 8);
        }
        if (S::kSplit) {
            mbar_init(&pfull[0], 1);
            mbar_init(&pfull[1], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) prod_tmem_alloc<CG>(tmem_slot);
    if (S::kSplit && warp == 3 && lane < 4 * kMostParts) sent[lane] = kNoTile;
    if (threadIdx.x == 32 * 2) {
        prefetch_map(&tmW);
        prefetch_map(&tmX);
        if (S::kFp4 && a.s_copy >= 16) {
            prefetch_map(&tmWS);
            prefetch_map(&tmXS);
        }
    }
    pdl_wait();                                  // what earlier kernels write is read from here on
    // the CTAs of a cluster walk the tiles together: a pair as one, or each with its part of K
    const int ks = S::kSplit ? a.ks : 1, part = S::kSplit ? (int)blockIdx.x % ks : 0;
    const int rank = CG == 1 ? 0 : (int)(blockIdx.x & 1), first = (int)blockIdx.x / (CG * ks), step = (int)gridDim.x / (CG * ks);
    const int nw = (a.N + CG * kProdRows - 1) / (CG * kProdRows);
    tc_fence_before();
    const int ntiles = prod_groups<TN>(a, gr, nw, scratch);
    // the barriers of all are ready (to partial sums from other CTAs, before those send them)
    if (CG == 2)
        cluster_sync_all();
    else if (ks > 1)
        cluster_arrive();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int nst = (a.K + kStageK - 1) / kStageK;
    constexpr int NB = S::kScaleBufs;
    // this CTA's stages, whole batches of scales
    const int nbt = (nst + S::kBatch - 1) / S::kBatch;
    const int kb0 = ks == 1 ? 0 : nbt * part / ks * S::kBatch, kb1 = ks == 1 ? nst : min(nst, nbt * (part + 1) / ks * S::kBatch);
    const uint32_t tiles = smem_u32(smem);

    if (warp == 0) {
        // ------------------------------- TMA producer -------------------------------
        int it = 0;
        if (!held) {
            const uint32_t on = elect_lane();
            bool ok = true;
            ProdWalk<TN> walk(first);
            for (; walk.tile < ntiles && ok; walk.tile += step) {
                const ProdTile t = walk.at(gr, nw);
                const int wrow = t.g * a.N + (t.w * CG + rank) * kProdRows;
                const int share = CG == 1 ? t.rows : (t.rows + S::kStep - 1) / S::kStep * 16, row0 = t.row0 + rank * share;
                const int loads = (share + S::kBox - 1) / S::kBox;
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int slot = it % NS;
                    if (!warp_wait<S::kFp4>(&empty[slot], ((it / NS) & 1) ^ 1, err, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t st = tiles + slot * S::kStage;
                    // (of both CTAs, where the leader counts them)
                    if (rank == 0) expect_on(&full[slot], CG * (kProdABytes + loads * S::kBox * 128), on);
                    const uint32_t bar = CG == 1 ? smem_u32(&full[slot]) : in_leader(&full[slot]);
                    const int k = kb * (KIND == PROD_16 ? 64 : 128);  // elements of the maps
                    tma_on<CG>(st, &tmW, k, wrow, bar, on);
                    for (int j = 0; j < loads; ++j)
                        tma_on<CG>(st + kProdABytes + j * (S::kBox * 128), &tmX, k, row0 + j * S::kBox, bar, on);
                }
            }
            // every load issued must land before the CTA exits -- one limit for all of them. (A pair's have where its MMAs
            // were all issued; where a wait ran out, settle_pair sees to it.)
            if (CG == 1)
                for (int j = it > NS ? it - NS : 0; j < it; ++j)
                    if (!mbar_wait(&full[j % NS], (j / NS) & 1, err)) break;
        }
        if (CG == 2) {
            if (rank && lane == 0) store_there(in_leader((const void *)issued), (uint32_t)it);
            issued_here = it;
        }
    } else if (warp == 1) {
        // -------------------------------- MMA issuer --------------------------------
        if (rank == 0) {
            const uint32_t on = elect_lane();
            int lt = 0, slot = 0, sb = 0;
            uint32_t phase = 0, sphase = 0;                  // of the ring's and the scales' barriers
            bool ok = true;
            ProdWalk<TN> walk(first);
            for (; walk.tile < ntiles && ok; walk.tile += step, ++lt) {
                // N in units of 8 (from bit 17), M in units of 16 (from bit 24; of 128 from bit 27)
                const uint32_t n8 = __shfl_sync(0xFFFFFFFFu, (uint32_t)((walk.at(gr, nw).rows + S::kStep - 1) / S::kStep * (S::kStep / 8)), 0);
                uint32_t idesc = (n8 << 17) | ((uint32_t)(CG * kProdRows >> 4) << 24);
                if constexpr (S::kFp4)
                    idesc |= (1u << 7) | (1u << 10) | (KIND == PROD_MXFP4 ? 1u << 23 : 0u);
                else
                    idesc |= (1u << 4) | (a.bf16 ? (1u << 7) | (1u << 10) : 0u);
                const int b = lt & 1;
                if (!warp_wait<S::kFp4>(&tempty[b], ((lt >> 1) & 1) ^ 1, err, abort_flag)) break;
                tc_fence_after();
                const uint32_t d = (uint32_t)(b * TN);       // (all columns are this CTA's: they begin at 0)
                uint32_t acc = 0u;
                auto stage = [&](int n) {                    // the n MMAs of a stage; n is a constant where it is 4
                    const uint32_t sa = tiles + slot * S::kStage;
                    const uint64_t ad = smem_desc_sw128(sa), bd = smem_desc_sw128(sa + kProdABytes);
                    const uint32_t sc = S::kScaleAt + (uint32_t)sb * S::kScaleCols;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= n) break;
                        const uint64_t o = (uint64_t)(2 * kk);
                        if constexpr (S::kFp4)
                            mma_fp4<KIND, CG>(d, ad + o, bd + o, idesc, sc + 4 * kk, sc + 16 + S::kBCols * kk, acc, on);
                        else
                            mma_16<CG>(d, ad + o, bd + o, idesc, acc, on);
                        acc = 1u;
                    }
                    commit_on<CG>(&empty[slot], on);         // free once these MMAs have read it
                    if (S::kFp4) commit_on<CG>(&sempty[sb], on);
                    if (++slot == NS) slot = 0, phase ^= 1u;
                    if (++sb == NB) sb = 0, sphase ^= 1u;
                };
                auto wait = [&]() {
                    ok = warp_wait<S::kFp4>(&full[slot], phase, err, abort_flag);
                    if (S::kFp4 && ok) ok = warp_wait<S::kFp4>(&sfull[sb], sphase, err, abort_flag);
                    tc_fence_after();
                    return ok;
                };
                // (the last stage may be shorter)
                const int whole = min(kb1, a.K / kStageK);
                for (int kb = kb0; kb < whole; ++kb) {
                    if (!wait()) break;
                    stage(4);
                }
                if (ok && whole < kb1 && wait()) stage((a.K - whole * kStageK + kMmaK - 1) / kMmaK);
                if (!ok) break;
                commit_on<CG>(&tfull[b], on);
            }
            commit_on<CG>(done, on);
            mbar_wait(done, 0, err);
        }
    } else if (warp < 10) {
        // --------------------------------- epilogue ---------------------------------
        const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter of this warp, its share of the columns
        int lt = 0;
        [[maybe_unused]] int turn = 0;           // of two buffers for results
        bool ok = true;                          // once a wait ran out, phases tell nothing: all later tiles are NaN
        ProdWalk<TN> walk(first);
        for (; walk.tile < ntiles; walk.tile += step, ++lt) {
            const ProdTile t = walk.at(gr, nw);
            const int b = lt & 1;
            const int n0 = (t.w * CG + rank) * kProdRows, n = n0 + q * 32 + lane;
            const ProdScales<S::kFp4, TN> sc(a, t, n);
            ok = ok && warp_wait<S::kFp4>(&tfull[b], (lt >> 1) & 1, err, abort_flag);
            tc_fence_after();
            const uint32_t at = ((uint32_t)(q * 32) << 16) + (uint32_t)(b * TN);
            unsigned char *stage = staged + half * (S::kOutBufs * 8192);
            const bool wide = S::kWide && a.wide && n0 + kProdRows <= a.N;
            bool stored = false;
            if constexpr (S::kSplit) {
                if (ks > 1) {
                    if (lt == 0) cluster_wait();
                    // (32 rows are the first four warps')
                    if (!half)
                        prod_store_split<S::kFp4, TN>(a, t, sc, at, n, ok, parts, part, pfull, lt, lost, err, abort_flag);
                    stored = true;
                }
            }
            if constexpr (TN == 32) {
                if (!stored && !half) prod_store_few<S::kFp4>(a, t, sc, at, n, ok);
                stored = true;
            }
            if (stored)
                ;
            else if (wide && a.y_type == MOE_T_BF16)
                prod_store_wide<S::kFp4, TN, __nv_bfloat16>(a, t, sc, at, n0, half, ok, stage, turn);
            else if (wide)
                prod_store_wide<S::kFp4, TN, __half>(a, t, sc, at, n0, half, ok, stage, turn);
            else if (a.y_type == MOE_T_BF16)
                prod_store<S::kFp4, TN, __nv_bfloat16>(a, t, sc, at, n, half, !ok);
            else if (a.y_type == MOE_T_F16)
                prod_store<S::kFp4, TN, __half>(a, t, sc, at, n, half, !ok);
            else
                prod_store<S::kFp4, TN, float>(a, t, sc, at, n, half, !ok);
            tc_fence_before();
            warp_arrive<CG>(&tempty[b]);
        }
        if (S::kSplit && lost != kNoTile && lane < ks && lane != part)
            store_there(in_rank((const void *)(sent + 4 * part + q), lane), (uint32_t)(lost + 1));
    } else if constexpr (S::kFp4) {
        constexpr int QB = S::kBatchBytes, G = S::kBatch, SB = QB / G, NQ = S::kBatches, kSlot = S::kSlotBytes;
        const int b0 = kb0 / G, b1 = (kb1 + G - 1) / G;
        // the 16-byte halves of 32-byte rows lie in the order of TMA's 32-byte swizzle: rows read together are then on
        // different banks
        auto swizzled = [](int row, int off) { return QB == 32 ? off ^ ((row >> 2) & 1) << 4 : off; };
        if (warp < 18) {
            // ------------------------- scales to tensor memory --------------------------
            // (two groups of four warps, for alternate stages)
            const int q = warp & 3, group = (warp - 10) >> 2;
            int it = 0, qr = 0;
            bool ok = true;
            ProdWalk<TN> walk(first);
            for (; walk.tile < ntiles && ok; walk.tile += step) {
                int wrow = 0, xrow = 0;          // whether the tile's first rows of W and x are odd
                if (KIND == PROD_MXFP4 && a.s_copy <= 2) {
                    const ProdTile p = walk.at(gr, nw);
                    wrow = (p.g & a.N & 1);      // (of g N + a multiple of 128)
                    xrow = p.row0 & 1;           // (behind 128 rows of W)
                }
                for (int kb = kb0; kb < kb1 && ok; kb += G, ++qr) {
                    if (!warp_wait<S::kFp4>(&lfull[qr % NQ], (qr / NQ) & 1, err, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const unsigned char *ring = scales + (qr % NQ) * kSlot;
                    const int n = min(G, kb1 - kb);
                    for (int i = 0; i < n; ++i, ++it) {
                        if ((it & 1) != group) continue;
                        uint32_t va[16], vb[4 * S::kBCols];
                        static_assert(S::kBCols == 4 || S::kBCols == 6, "columns that the stores below cover");
                        auto words = [&](int row, int first_row, uint32_t w[4]) {
                            if constexpr (KIND == PROD_NVFP4) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(ring + row * QB + swizzled(row, i * SB));
                                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                            } else {                 // two scales a column
                                uint2 v;
                                if (a.s_copy > 2) {
                                    v = *reinterpret_cast<const uint2 *>(ring + row * QB + i * SB);
                                } else {             // an odd row begins in the middle of a word
                                    const uint32_t *at = reinterpret_cast<const uint32_t *>(ring + row * 24 + i * SB);
                                    const int shift = ((first_row + row) & 1) * 16;
                                    v.x = __funnelshift_r(at[0], at[1], shift);
                                    v.y = __funnelshift_r(at[1], at[2], shift);
                                }
                                w[0] = v.x & 0xFFFFu, w[1] = v.x >> 16, w[2] = v.y & 0xFFFFu, w[3] = v.y >> 16;
                            }
                        };
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            uint32_t w[4];
                            words(32 * m + lane, wrow, w);
#pragma unroll
                            for (int j = 0; j < 4; ++j) va[4 * j + m] = w[j];
                        }
#pragma unroll
                        for (int m = 0; m < S::kBCols; ++m) {
                            uint32_t w[4] = {0u, 0u, 0u, 0u};
                            if (32 * m < TN) words(kProdRows + 32 * m + lane, xrow, w);
#pragma unroll
                            for (int j = 0; j < 4; ++j) vb[S::kBCols * j + m] = w[j];
                        }
                        if (!warp_wait<S::kFp4>(&sempty[it % NB], ((it / NB) & 1) ^ 1, err, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t to = ((uint32_t)(q * 32) << 16) + S::kScaleAt + (uint32_t)(it % NB) * S::kScaleCols;
                        tmem_st16(to, va);
                        tmem_st16(to + 16, vb);
                        if constexpr (S::kBCols == 6) tmem_st8(to + 32, vb + 16);
                        tmem_st_wait();
                        tc_fence_before();
                        warp_arrive<CG>(&sfull[it % NB]);
                    }
                    warp_arrive<1>(&lempty[qr % NQ]);
                }
            }
        } else if (a.s_copy >= 16) {
            // ----------------------- scales to shared memory, by TMA --------------------
            if (warp == 18 && !held) {
                const uint32_t on = elect_lane(), ring = smem_u32(scales);
                int qr = 0;
                bool ok = true;
                ProdWalk<TN> walk(first);
                for (; walk.tile < ntiles && ok; walk.tile += step) {
                    const ProdTile p = walk.at(gr, nw);
                    const int wrow = p.g * a.N + (p.w * CG + rank) * kProdRows;
                    const int loads = (p.rows + S::kScaleBox - 1) / S::kScaleBox;
                    for (int i = b0; i < b1; ++i, ++qr) {
                        uint64_t *bar = &lfull[qr % NQ];
                        if (!warp_wait<S::kFp4>(&lempty[qr % NQ], ((qr / NQ) & 1) ^ 1, err, abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t to = ring + (qr % NQ) * kSlot;
                        expect_on(bar, (kProdRows + loads * S::kScaleBox) * QB, on);
                        tma_on<CG>(to, &tmWS, i * QB, wrow, smem_u32(bar), on);
                        for (int j = 0; j < loads; ++j)
                            tma_on<CG>(to + (kProdRows + j * S::kScaleBox) * QB, &tmXS, i * QB, p.row0 + j * S::kScaleBox,
                                       smem_u32(bar), on);
                    }
                }
                for (int j = qr > NQ ? qr - NQ : 0; j < qr; ++j)
                    if (!mbar_wait(&lfull[j % NQ], (j / NQ) & 1, err)) break;
            }
        } else {
            // ------------- scales to shared memory, where their rows are not aligned -----
            // by words, the ones of a row by neighbouring threads (whole sectors). What lies behind a row's end is
            // read too, but never what lies behind the array's; no MMA uses it.
            const bool odd = a.s_copy <= 2;      // rows of an odd number of 16-bit words
            const int per = KIND == PROD_NVFP4 || odd ? 8 : 4, words = KIND == PROD_NVFP4 ? 8 : odd ? 5 : 4;
            const int t = threadIdx.x - 18 * 32, piece = t % per, r0 = t / per, rstep = 64 / per;
            const int pitch = a.K / (KIND == PROD_NVFP4 ? 16 : 32);  // bytes of a row's scales
            const int to_pitch = odd ? 24 : QB;
            const uint32_t ring = smem_u32(scales) + r0 * to_pitch + (KIND == PROD_NVFP4 ? swizzled(r0, 4 * piece) : 4 * piece);
            const int64_t wbytes = (int64_t)a.groups * a.N * pitch, xbytes = (int64_t)a.M * pitch;
            int qr = 0;
            bool ok = true;
            // rows `row` to row + n of an array of scales, from column byte k on; n a multiple of rstep
            auto copy = [&](const uint8_t *base, int64_t total, int64_t row, int n, int k, uint32_t to) {
                int64_t off = ((row + r0) * pitch & ~3ll) + k + 4 * piece;
                const int64_t last = (row + n) * pitch + k + 4 * words;
                if (piece >= words) return;
                if (last <= total) {
#pragma unroll 8
                    for (int r = 0; r < n; r += rstep) {
                        cp_async<4>(to, base + off, 4);
                        off += (int64_t)rstep * pitch;
                        to += rstep * to_pitch;
                    }
                } else {
                    for (int r = 0; r < n; r += rstep) {
                        const int64_t left = total - off;
                        const int size = left >= 4 ? 4 : left > 0 ? (int)left : 0;
                        cp_async<4>(to, base + (size ? off : 0), size);
                        off += (int64_t)rstep * pitch;
                        to += rstep * to_pitch;
                    }
                }
            };
            ProdWalk<TN> walk(first);
            for (; walk.tile < ntiles && ok; walk.tile += step) {
                const ProdTile p = walk.at(gr, nw);
                const int64_t wrow = (int64_t)p.g * a.N + (int64_t)(p.w * CG + rank) * kProdRows;
                for (int i = b0; i < b1; ++i, ++qr) {
                    if (!warp_wait<S::kFp4>(&lempty[qr % NQ], ((qr / NQ) & 1) ^ 1, err, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = ring + (qr % NQ) * kSlot;
                    copy(a.ws, wbytes, wrow, kProdRows, i * QB, to);
                    copy(a.xs, xbytes, p.row0, (p.rows + 31) / 32 * 32, i * QB, to + kProdRows * to_pitch);
                    cp_async_arrive(&lfull[qr % NQ]);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    // no CTA of a cluster leaves, or frees its tensor memory, while another may still reach it
    if (CG == 2 || ks > 1) {
        if (rank && warp == 1) mbar_wait(done, 0, err);      // the leader's last arrival here
        __syncwarp();
        // (those that did not wait for the start yet)
        if (CG == 1 && (warp < 2 || warp >= 10 || first >= ntiles)) cluster_wait();
        __syncwarp();
        if (CG == 2 && threadIdx.x == 0 && *abort_flag) store_there(in_rank((const void *)abort_flag, 1 - rank), 1u);
        cluster_sync_all();
        // a wait ran out in one of a pair or both: operands may be on their way to either
        if (CG == 2 && *abort_flag) {
            if (rank == 0 && threadIdx.x == 0) settle_pair<S, TN>(gr, nw, first, step, nst, issued_here, *issued, full, err);
            __syncwarp();
            cluster_sync_all();
        }
        if (S::kSplit && warp == 4 && lane == 0 && lost != kNoTile)
            settle_parts<TN>(gr, nw, first, step, ntiles, ks, part, lost, sent, pfull, err);
    }
    if (warp == 1) {
        tc_fence_after();
        prod_tmem_free<CG>(tmem_base);
    }
}

#endif  // __CUDACC__

// Host: 2-D map of rows of `row_bytes`, `pitch` bytes apart, in boxes of 128 bytes x box_rows with the 128-byte swizzle.
bool make_tmap_rows(CUtensorMap *tm, const void *base, uint64_t rows, uint64_t row_bytes, uint64_t pitch,
                    uint32_t box_rows, bool two_byte);
// The same of bytes, in boxes of box_bytes (32, with the swizzle of that width, or 16), rows without gaps.
bool make_tmap_scales(CUtensorMap *tm, const void *base, uint64_t rows, uint64_t row_bytes, uint32_t box_bytes,
                      uint32_t box_rows);
int device_sms();
constexpr int kProdDevices = 64;

// What a product runs as: tiles of `rows` rows of x by 128 weight rows, or by 256 on a pair of CTAs; K in ks parts.
struct ProdPlan {
    int rows, pair, ks;
};
ProdPlan plan_product(bool fp4, int groups, int M, int N, int K);

#ifdef __CUDACC__
// x: rows x_pitch bytes apart; w: [groups * N] rows without gaps.
template <int KIND, int TN, int CG = 1>
cudaError_t launch_product(const ProdArgs &a0, const void *x, int64_t x_pitch, const void *w, int ks, cudaStream_t st) {
    using S = ProdShape<KIND, TN, CG>;
    static std::atomic<uint64_t> attr_set{0};
    const auto kern = product_kernel<KIND, TN, CG>;
    cudaError_t e = set_smem_limit_once((const void *)kern, (int)S::kSmem, attr_set);
    if (e != cudaSuccess) return e;
    ProdArgs a = a0;
    a.hold = products_held();
    // (every part has work)
    constexpr int kBatchK = (KIND == PROD_16 ? 64 : 256) * S::kBatch;
    const int most_ks = (a.K + kBatchK - 1) / kBatchK;
    a.ks = !S::kSplit ? 1 : ks < most_ks ? ks : most_ks;
    a.wide = a.y_type != MOE_T_F32 && (uintptr_t)a.y % 16 == 0 && (a.M == 1 || a.y_ld % 8 == 0);
    const uint64_t row = KIND == PROD_16 ? (uint64_t)a.K * 2 : (uint64_t)a.K / 2;
    CUtensorMap tw, tx;
    if (!make_tmap_rows(&tw, w, (uint64_t)a.groups * a.N, row, row, kProdRows, KIND == PROD_16) ||
        !make_tmap_rows(&tx, x, a.M, row, a.M > 1 ? x_pitch : row, S::kBox, KIND == PROD_16))
        return cudaErrorInvalidValue;
    CUtensorMap tws = tw, txs = tx;
    if constexpr (S::kFp4) {
        const uint64_t srow = a.K / (KIND == PROD_NVFP4 ? 16 : 32);
        if (a.s_copy >= 16 &&
            (!make_tmap_scales(&tws, a.ws, (uint64_t)a.groups * a.N, srow, S::kBatchBytes, kProdRows) ||
             !make_tmap_scales(&txs, a.xs, a.M, srow, S::kBatchBytes, S::kScaleBox)))
            return cudaErrorInvalidValue;
    }
    const int64_t nw = (a.N + CG * kProdRows - 1) / (CG * kProdRows);
    // a tile of every group may be ragged
    const int64_t most = ((int64_t)a.M / TN + (a.groups < a.M ? a.groups : a.M)) * nw;
    cudaLaunchConfig_t cfg{};
    const int width = CG * a.ks;                 // CTAs of a cluster
    cfg.gridDim = dim3(width * 1024);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = width;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = width == 1 ? 1 : 2;
    // no more clusters than the device holds at once (fewer than the SMs suggest: a cluster's CTAs lie in one group of SMs)
    static std::atomic<int> known[kProdDevices][kMostParts + 1];
    int dev = 0, n = device_sms();
    if (n < 1 || cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    if (width > 1) {
        n = dev < kProdDevices ? known[dev][width].load(std::memory_order_relaxed) : 0;
        if (n < 1) {
            cudaLaunchConfig_t ask = cfg;
            ask.attrs = attr + 1;
            ask.numAttrs = 1;
            if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &ask)) != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
            if (dev < kProdDevices) known[dev][width].store(n, std::memory_order_relaxed);
        }
    }
    cfg.gridDim = dim3((unsigned)(most < n ? most : n) * width);
    return cudaLaunchKernelEx(&cfg, kern, tw, tx, tws, txs, a);
}
#endif

}  // namespace moe
