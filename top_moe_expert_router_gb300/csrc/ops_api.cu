// ops_api.cu — C entries (include/moe.h) of the operators around the expert
// layer: argument checks on the host, then one launch or two on the caller's
// stream.
#include <limits.h>
#include <math.h>

#include "ops.cuh"
#include "ops_api.h"

namespace moe {

moe_status check_route_desc(const moe_route_desc *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->E < 1 || d->top_k < 1 || d->top_k > d->E || d->n_groups < 1 || d->topk_groups < 1 ||
        d->topk_groups > d->n_groups || d->E % d->n_groups || !isfinite(d->scale) ||
        (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID) ||
        (d->group_rule != MOE_GROUP_MAX && d->group_rule != MOE_GROUP_TOP2) || ((uintptr_t)d->bias & 3u))
        return MOE_ERR_INVALID_ARG;
    if (d->E / d->n_groups * d->topk_groups < d->top_k) return MOE_ERR_INVALID_ARG;
    if (d->E > kRouteMaxE || d->top_k > kRouteMaxK || d->n_groups > kRouteMaxGroups) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

RouteArgs route_args(const moe_route_desc &d) {
    RouteArgs a{};
    a.E = d.E;
    a.k = d.top_k;
    a.sigmoid = d.score == MOE_SCORE_SIGMOID;
    a.bias = d.bias;
    a.groups = d.n_groups;
    a.keep = d.topk_groups;
    a.top2 = d.group_rule == MOE_GROUP_TOP2;
    a.renorm = d.renormalise != 0;
    a.scale = d.scale;
    a.nsplit = 1;
    a.perm_fill = -1;
    return a;
}

}  // namespace moe

namespace {

using namespace moe;

bool misaligned(const void *p, unsigned a) { return ((uintptr_t)p & (a - 1u)) != 0; }
int type_size(moe_dtype t) { return t == MOE_T_F32 ? 4 : t == MOE_T_E4M3 ? 1 : 2; }
bool is_float_type(moe_dtype t) { return t == MOE_T_BF16 || t == MOE_T_F16 || t == MOE_T_F32; }
moe_status status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

moe_status moe_route_logits_workspace_size(const moe_route_desc *desc, int T, size_t *bytes) {
    const moe_status s = check_route_desc(desc);
    if (s != MOE_OK) return s;
    if (!bytes || T < 0) return MOE_ERR_INVALID_ARG;
    if (T > kRouteMaxT) return MOE_ERR_UNSUPPORTED;
    *bytes = T ? route_scratch_bytes(T, desc->E) : 0;
    return MOE_OK;
}

moe_status moe_route_logits(const moe_route_desc *desc, const void *logits, moe_dtype type, int64_t row_stride, int T,
                            int32_t *ids, float *w, int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *pos,
                            void *workspace, size_t ws_bytes, void *stream) {
    const moe_status s = check_route_desc(desc);
    if (s != MOE_OK) return s;
    if (!is_float_type(type)) return MOE_ERR_UNSUPPORTED;
    if (T < 0) return MOE_ERR_INVALID_ARG;
    if (T > kRouteMaxT) return MOE_ERR_UNSUPPORTED;
    for (const void *p : {(const void *)counts, (const void *)offsets, (const void *)perm, (const void *)pos,
                          (const void *)ids, (const void *)w})
        if (misaligned(p, 4)) return MOE_ERR_INVALID_ARG;
    if (misaligned(workspace, 16)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {
        if (counts && cudaMemsetAsync(counts, 0, sizeof(int32_t) * (size_t)desc->E, st) != cudaSuccess)
            return MOE_ERR_CUDA;
        if (offsets && cudaMemsetAsync(offsets, 0, sizeof(int32_t) * ((size_t)desc->E + 1), st) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!logits || !ids || !w || misaligned(logits, (unsigned)type_size(type)) || row_stride < desc->E)
        return MOE_ERR_INVALID_ARG;
    RouteArgs a = route_args(*desc);
    a.logits = logits;
    a.type = type;
    a.stride = row_stride;
    a.T = T;
    a.ids = ids;
    a.w = w;
    a.counts = counts;
    a.offsets = offsets;
    a.perm = perm;
    a.pos = pos;
    if (counts || offsets || perm || pos) {
        const size_t need = route_scratch_bytes(T, desc->E);
        if (need && (!workspace || ws_bytes < need)) return MOE_ERR_INVALID_ARG;
        a.chunk_cnt = (uint16_t *)workspace;
    }
    return status_of(launch_route_logits(a, st, nullptr));
}

moe_status moe_add_rmsnorm(const moe_norm_args *n, void *stream) {
    if (!n || n->T < 0 || n->d < 1 || !(n->eps >= 0.f) || !isfinite(n->eps)) return MOE_ERR_INVALID_ARG;
    if (!is_float_type(n->type) || (n->out_type != n->type && n->out_type != MOE_T_E4M3)) return MOE_ERR_UNSUPPORTED;
    if (n->d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
    const bool e4m3 = n->out_type == MOE_T_E4M3;
    const int group = n->group ? n->group : n->d;
    if (n->group < 0 || (e4m3 ? n->d % group != 0 : n->group != 0)) return MOE_ERR_INVALID_ARG;
    if (e4m3 && n->d / group > 4096) return MOE_ERR_UNSUPPORTED;
    if (n->T == 0) return MOE_OK;
    const unsigned es = (unsigned)type_size(n->type);
    if (!n->x || !n->out || (e4m3 && !n->scales)) return MOE_ERR_INVALID_ARG;
    if (misaligned(n->x, es) || misaligned(n->res, es) || misaligned(n->sum, es) || misaligned(n->gain, es) ||
        misaligned(n->out, (unsigned)type_size(n->out_type)) || misaligned(n->scales, 4))
        return MOE_ERR_INVALID_ARG;
    if (n->x_stride < n->d || n->out_stride < n->d || (n->res && n->res_stride < n->d) ||
        (n->sum && n->sum_stride < n->d) || (e4m3 && n->scales_stride < n->d / group))
        return MOE_ERR_INVALID_ARG;
    // in place means the same rows; the E4M3 codes of one would lie over another's elements
    if (n->sum == n->out) return MOE_ERR_INVALID_ARG;
    struct { const void *in; int64_t ld; } in[2] = {{n->x, n->x_stride}, {n->res, n->res_stride}};
    for (const auto &i : in) {
        if (!i.in) continue;
        if (n->out == i.in && (e4m3 || (n->T > 1 && n->out_stride != i.ld))) return MOE_ERR_INVALID_ARG;
        if (n->sum == i.in && n->T > 1 && n->sum_stride != i.ld) return MOE_ERR_INVALID_ARG;
    }
    NormArgs a{};
    a.x = n->x;
    a.res = n->res;
    a.gain = n->gain;
    a.sum = n->sum;
    a.out = n->out;
    a.scales = n->scales;
    a.x_ld = n->x_stride;
    a.res_ld = n->res_stride;
    a.sum_ld = n->sum_stride;
    a.out_ld = n->out_stride;
    a.scales_ld = n->scales_stride;
    a.T = n->T;
    a.d = n->d;
    a.group = group;
    a.eps = n->eps;
    a.type = n->type;
    a.e4m3 = e4m3;
    return status_of(launch_add_rmsnorm(a, (cudaStream_t)stream));
}

moe_status moe_linear_w4(const moe_w4_args *l, void *stream) {
    if (!l || l->M < 0 || l->N < 1 || l->K < 1) return MOE_ERR_INVALID_ARG;
    if (l->fmt != MOE_W4_NVFP4 && l->fmt != MOE_W4_INT4) return MOE_ERR_UNSUPPORTED;
    if (l->M > kW4MaxM || l->N > kW4MaxN || l->K > kW4MaxK || l->K % 32) return MOE_ERR_UNSUPPORTED;
    if (l->x_type != MOE_T_BF16 && l->x_type != MOE_T_F16 && l->x_type != MOE_T_E4M3) return MOE_ERR_UNSUPPORTED;
    if (!is_float_type(l->y_type)) return MOE_ERR_UNSUPPORTED;
    const bool nvfp4 = l->fmt == MOE_W4_NVFP4;
    if (nvfp4) {
        if (l->group != 16) return MOE_ERR_UNSUPPORTED;
    } else {
        if ((l->group != 32 && l->group != 64 && l->group != 128) ||
            (l->s_type != MOE_T_BF16 && l->s_type != MOE_T_F16))
            return MOE_ERR_UNSUPPORTED;
        if (l->K % l->group) return MOE_ERR_INVALID_ARG;
    }
    const bool e4m3 = l->x_type == MOE_T_E4M3;
    const int xg = l->x_group ? l->x_group : l->K;
    if (e4m3) {
        if (l->x_group < 0 || l->K % xg) return MOE_ERR_INVALID_ARG;
        if (l->x_group % 128 && xg != l->K) return MOE_ERR_UNSUPPORTED;
    }
    if (l->M == 0) return MOE_OK;
    if (!l->q || !l->s || !l->x || !l->y || (nvfp4 && !l->g) || (e4m3 && !l->x_scales)) return MOE_ERR_INVALID_ARG;
    if (misaligned(l->q, 16) || misaligned(l->s, 2) || misaligned(l->g, 4) || misaligned(l->bias, 4) ||
        misaligned(l->x, (unsigned)type_size(l->x_type)) || misaligned(l->y, (unsigned)type_size(l->y_type)) ||
        misaligned(l->x_scales, 4))
        return MOE_ERR_INVALID_ARG;
    if (l->x_stride < l->K || l->y_stride < l->N || (e4m3 && l->x_scales_stride < l->K / xg)) return MOE_ERR_INVALID_ARG;
    W4Args a{};
    a.q = l->q;
    a.s = l->s;
    a.g = l->g;
    a.z = nvfp4 ? nullptr : l->z;
    a.x = l->x;
    a.xs = l->x_scales;
    a.bias = l->bias;
    a.y = l->y;
    a.x_ld = l->x_stride;
    a.xs_ld = l->x_scales_stride;
    a.y_ld = l->y_stride;
    a.M = l->M;
    a.N = l->N;
    a.K = l->K;
    a.group = l->group;
    a.xgroup = xg;
    a.nvfp4 = nvfp4;
    a.s_type = l->s_type;
    a.x_type = l->x_type;
    a.y_type = l->y_type;
    return status_of(launch_linear_w4(a, (cudaStream_t)stream));
}

moe_status moe_linear_w4_status(void *stream) {
    uint32_t bits = 0;
    if (linear_w4_errors((cudaStream_t)stream, &bits) != cudaSuccess) return MOE_ERR_CUDA;
    return bits & ERRBIT_TIMEOUT ? MOE_ERR_TIMEOUT : MOE_OK;
}

moe_status moe_debug_hold_linear_w4(int hold) {
    hold_linear_w4(hold != 0);
    return MOE_OK;
}

}  // extern "C"
