// grouped_linear.cu — y[r] = W[e(r)] x[r] + b[e(r)] for rows grouped by expert,
// operands in bf16 or f16 (the kernel: products.cuh), and what the products
// share on the host.
#include <stdio.h>
#include <stdlib.h>
#include "products.cuh"

namespace moe {

static std::atomic<int> prod_hold{0};
bool products_held() { return prod_hold.load(std::memory_order_relaxed) != 0; }
void hold_products(bool hold) { prod_hold.store(hold, std::memory_order_relaxed); }

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
    return enc(tm, two_byte ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
               const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

cudaError_t launch_grouped_linear(const ProdArgs &a, const void *x, int64_t x_ld, const void *w, cudaStream_t st) {
    static const char *env = getenv("MOE_PLAN");
    int tn = 0, ks = 1, per = a.M / (a.groups < a.M ? a.groups : a.M);
    if (env) sscanf(env, "%d,%d", &tn, &ks);
    if (!tn) tn = a.M <= 32 || per <= 16 ? 32 : per <= 64 ? 128 : a.N <= 128 ? 128 : 256;
    if (tn == 32) return launch_product<PROD_16, 32>(a, x, 2 * x_ld, w, ks, st);
    if (tn == 64) return launch_product<PROD_16, 64>(a, x, 2 * x_ld, w, ks, st);
    if (tn == 128) return launch_product<PROD_16, 128>(a, x, 2 * x_ld, w, ks, st);
    if (tn == 129) return launch_product<PROD_16, 128, 2>(a, x, 2 * x_ld, w, ks, st);
    return launch_product<PROD_16, 256, 2>(a, x, 2 * x_ld, w, ks, st);
}

}  // namespace moe
