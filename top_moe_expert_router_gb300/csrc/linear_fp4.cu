// linear_fp4.cu — y[r] = W[e(r)] x[r] + b[e(r)] where both operands are
// microscaled 4-bit floats, for one matrix or for rows grouped by expert (the
// kernel: products.cuh). The products of two codes and their block scales are
// formed and summed by the tensor cores (kind::mxf4nvf4: E4M3 scales per 16,
// kind::mxf4: powers of two per 32), in fp32; the second scales of x and W, and
// the bias, belong to the epilogue.
#include "products.cuh"

namespace moe {

cudaError_t linear_fp4_errors(cudaStream_t st, uint32_t *bits) { return prod_take_errors(st, bits); }

template <int KIND>
static cudaError_t launch_kind(const ProdArgs &a, const uint8_t *xq, const uint8_t *wq, cudaStream_t st) {
    const int64_t pitch = a.K / 2;
    const ProdPlan p = plan_product(true, a.groups, a.M, a.N, a.K);
    if (p.rows == 32) return launch_product<KIND, 32>(a, xq, pitch, wq, p.ks, st);
    if (p.rows == 64) return launch_product<KIND, 64>(a, xq, pitch, wq, 1, st);
    if (p.rows == 128) return launch_product<KIND, 128>(a, xq, pitch, wq, 1, st);
    return launch_product<KIND, 192, 2>(a, xq, pitch, wq, 1, st);
}

cudaError_t launch_linear_fp4(ProdArgs a, bool nvfp4, const uint8_t *xq, const uint8_t *wq, cudaStream_t st) {
    const uintptr_t at = (uintptr_t)a.xs | (uintptr_t)a.ws | (uintptr_t)(a.K / (nvfp4 ? 16 : 32));
    a.s_copy = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 2;
    return nvfp4 ? launch_kind<PROD_NVFP4>(a, xq, wq, st) : launch_kind<PROD_MXFP4>(a, xq, wq, st);
}

}  // namespace moe
