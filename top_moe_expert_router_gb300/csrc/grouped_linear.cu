// grouped_linear.cu — y[r] = W[e(r)] x[r] + b[e(r)] for rows grouped by expert,
// operands in bf16 or f16 (the kernel: products.cuh), and what the products
// share on the host.
#include "products.cuh"

namespace moe {

static std::atomic<int> prod_hold{0};
int products_held() { return prod_hold.load(std::memory_order_relaxed); }
void hold_products(int hold) { prod_hold.store(hold, std::memory_order_relaxed); }

cudaError_t linear_fp4_errors(cudaStream_t st, uint32_t *bits);  // linear_fp4.cu

// Reads and clears the current device's error bits, after `st`'s work.
cudaError_t products_errors(cudaStream_t st, uint32_t *bits) {
    uint32_t fp4 = 0;
    cudaError_t e = prod_take_errors(st, bits);
    if (e == cudaSuccess) e = linear_fp4_errors(st, &fp4);
    *bits |= fp4;
    return e;
}

bool make_tmap_rows(CUtensorMap *tm, const void *base, uint64_t rows, uint64_t row_bytes, uint64_t pitch,
                    uint32_t box_rows, bool two_byte) {
    auto enc = get_encode();
    if (!enc) return false;
    const uint32_t es = two_byte ? 2 : 1;
    cuuint64_t dims[2] = {row_bytes / es, rows};
    cuuint64_t strides[1] = {pitch};
    cuuint32_t box[2] = {128 / es, box_rows};
    cuuint32_t estr[2] = {1, 1};
    // (rows that do not begin on lines of 128 bytes: what lies beside a box is rarely wanted. 5003 rows by 12 experts of
    // 2712 x 2712: 83 -> 74 us)
    const auto promote = pitch % 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    return enc(tm, two_byte ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, promote,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_tmap_scales(CUtensorMap *tm, const void *base, uint64_t rows, uint64_t row_bytes, uint32_t box_bytes,
                      uint32_t box_rows) {
    auto enc = get_encode();
    if (!enc) return false;
    cuuint64_t dims[2] = {row_bytes, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_bytes, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The current device's SMs, asked for once a device.
int device_sms() {
    constexpr int kMax = 64;
    static std::atomic<int> known[kMax];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < kMax && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < kMax) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// The plan with the shortest estimate, for a GB300 (152 SMs, 6.6 TB/s). The groups' sizes are on the device: as many as there
// can be are taken to share the rows. (Where few of many groups have rows, the tiles are then smaller than theirs would
// be: 8192 rows of 16 experts of 1536 x 4096, bf16 / NVFP4, 68 / 31 us, told among 256 experts 110 / 54; with 64 experts of
// 256 150 / 58 for 145 / 50.) Measured, a stage of a tile (K = 64, of 4-bit operands 256) takes
//   16 bits: 120 ns, or 6.3 ns for every KB that passes through shared memory, or what its MMAs take; a pair's at least 190
//   4 bits:  215 to 236 ns, a pair's 235 to 313
// and splitting K costs 2 us. The weights come no faster than from memory, which it takes about 120 CTAs to keep busy; read
// again for more tiles along a group's rows, mostly from L2, they count a quarter.
// Against each plan forced (20 dense and 15 grouped shapes, 1 to 32768 rows): within 6 % of the best. Few rows, us: 1 x 4096
// x 4096 bf16 whole K 11.4, in four parts 9.1; 200 x 4096 x 4096 bf16 tiles of 32 rows 21.2, of 64 14.5, pairs of 256 22.7;
// 1000 rows 61 / 41 / 26; NVFP4 1000 x 4096 x 4096 tiles of 32 rows 38, of 128 17.9, pairs 20.3; 4096 rows 132 / 48 / 43.
ProdPlan plan_product(bool fp4, int groups, int M, int N, int K) {
    static const ProdPlan shapes16[] = {{32, 0, 1}, {64, 0, 1}, {128, 0, 1}, {128, 1, 1}, {256, 1, 1}};
    static const ProdPlan shapes4[] = {{32, 0, 1}, {64, 0, 1}, {128, 0, 1}, {192, 1, 1}};
    const ProdPlan *shapes = fp4 ? shapes4 : shapes16;
    const int n_shapes = fp4 ? 4 : 5;
    const int used = groups < M ? groups : M, stages = fp4 ? (K + 255) / 256 : (K + 63) / 64;
    const double rows = (double)M / used;                    // of a group
    const double wbytes = (double)used * N * K * (fp4 ? 0.5625 : 2.0);
    ProdPlan best = shapes[0];
    double least = 1e30;
    for (int i = 0; i < n_shapes; ++i) {
        const ProdPlan &s = shapes[i];
        const int ctas = s.pair ? 2 : 1;
        // tiles along a group's rows: groups of several sizes end in a tile that is half full
        const double along = groups == 1 ? (M + s.rows - 1) / s.rows
                                         : rows <= 0.75 * s.rows ? 1.0 : rows / s.rows + 0.5;
        const double tiles = used * along * ((N + 128 * ctas - 1) / (128 * ctas)), full = rows / along;
        double ns;
        if (fp4) {
            ns = s.pair ? 235 + 78 * full / s.rows : 215 + s.rows / 6;
        } else {
            const double mma = 4 * (full < 92 ? 46 : full / 2) / 1.9 * 1.08, kb = 16 + s.rows / ctas / 8.0;
            ns = s.pair ? 190 : 120;
            ns = ns > mma ? ns : mma;
            ns = ns > 6.3 * kb ? ns : 6.3 * kb;
        }
        for (int ks = 1; ks <= (s.rows == 32 ? kMostParts : 1); ++ks) {
            const int slots = 152 / (ctas * ks), part = ((stages + 1) / 2 + ks - 1) / ks * 2;
            if (ks > 1 && (tiles > slots || part * (ks - 1) >= stages)) break;
            const double rounds = tiles <= slots ? 1 : (double)(int64_t)((tiles + slots - 1) / slots);
            const double busy = (tiles < slots ? tiles : slots) * ctas * ks;
            const double memory = wbytes * (0.75 + 0.25 * along) / (6600.0 * (busy < 120 ? busy / 120 : 1));
            double t = rounds * (ks > 1 ? part : stages) * ns;
            t = (t > memory ? t : memory) + rounds * 150 + (ks > 1 ? 2000 : 0);
            if (t < 0.98 * least) {
                least = t;
                best = {s.rows, s.pair, ks};
            }
        }
    }
    return best;
}

cudaError_t launch_grouped_linear(const ProdArgs &a, const void *x, int64_t x_ld, const void *w, cudaStream_t st) {
    const ProdPlan p = plan_product(false, a.groups, a.M, a.N, a.K);
    if (p.rows == 32) return launch_product<PROD_16, 32>(a, x, 2 * x_ld, w, p.ks, st);
    if (p.rows == 64) return launch_product<PROD_16, 64>(a, x, 2 * x_ld, w, 1, st);
    if (p.rows == 128 && !p.pair) return launch_product<PROD_16, 128>(a, x, 2 * x_ld, w, 1, st);
    if (p.rows == 128) return launch_product<PROD_16, 128, 2>(a, x, 2 * x_ld, w, 1, st);
    return launch_product<PROD_16, 256, 2>(a, x, 2 * x_ld, w, 1, st);
}

}  // namespace moe
