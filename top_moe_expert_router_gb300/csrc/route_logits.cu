// route_logits.cu — routing of tokens to experts from given logits: softmax or
// sigmoid scores, a per-expert bias that only steers the choice, group-limited
// choice, top-k, weights (renormalised or not), and the token permutation.
//
//   p[e] = softmax(l)[e] or 1 / (1 + exp(-l[e])),   c[e] = p[e] + bias[e]
//   group score = the best c of the group, or the sum of its two best
//   ids = the k best c within the `keep` best groups, by descending c
//   w[j] = scale * p[ids[j]] (/ sum of the chosen p)
// Every tie goes to the lower index. An expert whose logit or bias is NaN or
// -inf is never chosen (and has no part in the softmax where it is the
// logit); +inf counts as the largest finite float. Slots for which no expert
// is left hold id -1, weight 0 and position -1.
//
// The choice is that of 64-bit scores: 32 bits order two experts whose scores
// differ by less than a few 2^-24 by chance. 64-bit arithmetic for every
// expert would cost about 40 operations each at 1/64 of the fp32 rate, so each
// token is chosen in 32 bits first, with a bound on the error of every score
// it compared; only where two neighbours of the resulting order (or the
// border of the kept groups) lie closer than that bound is the token chosen
// again in 64 bits. Without a bias the order of the scores is that of the
// logits, which needs neither.
//
// One warp per token; lane l holds the EPL consecutive experts from l * EPL
// on, so that among equal keys the lowest lane and slot is the lowest id.
#include <math.h>

#include "ops.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kSelThreads = 256;

__device__ __forceinline__ float load_logit(const void *p, int64_t i, moe_dtype t) {
    if (t == MOE_T_F32) return __ldg((const float *)p + i);
    if (t == MOE_T_BF16) return __uint_as_float((uint32_t)__ldg((const uint16_t *)p + i) << 16);
    return __half2float(__ushort_as_half(__ldg((const uint16_t *)p + i)));
}

// A lane's EPL logits, experts e0 .. e0 + EPL - 1 (NaN past E).
template <int EPL>
__device__ __forceinline__ void load_lane(const RouteArgs &a, int64_t row, int e0, float l[EPL]) {
    if (a.vec) {  // E % EPL == 0 and every lane's first logit aligned
        if (e0 >= a.E) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) l[i] = NAN;
            return;
        }
        if (a.type == MOE_T_F32) {
            const float *p = (const float *)a.logits + row + e0;
            if constexpr (EPL >= 4) {
#pragma unroll
                for (int i = 0; i < EPL; i += 4) {
                    const float4 v = __ldg((const float4 *)(p + i));
                    l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i) l[i] = __ldg(p + i);
            }
            return;
        }
        const uint16_t *p = (const uint16_t *)a.logits + row + e0;
        uint32_t u[(EPL + 1) / 2];
        if constexpr (EPL >= 8) {
#pragma unroll
            for (int i = 0; i < EPL / 2; i += 4) {
                const uint4 v = __ldg((const uint4 *)(p + 2 * i));
                u[i] = v.x, u[i + 1] = v.y, u[i + 2] = v.z, u[i + 3] = v.w;
            }
        } else if constexpr (EPL == 4) {
            const uint2 v = __ldg((const uint2 *)p);
            u[0] = v.x, u[1] = v.y;
        } else if constexpr (EPL == 2) {
            u[0] = __ldg((const uint32_t *)p);
        } else {
            u[0] = __ldg(p);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const uint32_t h = (i & 1) ? u[i / 2] >> 16 : u[i / 2] & 0xFFFFu;
            l[i] = a.type == MOE_T_BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((uint16_t)h));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = e0 + i;
        l[i] = e < a.E ? load_logit(a.logits, row + e, a.type) : NAN;
        if (a.nsplit > 1 && e < a.E)
            for (int s = 1; s < a.nsplit; ++s) l[i] += ((const float *)a.logits)[row + s * a.split_stride + e];
    }
}

// Order-preserving unsigned keys; 0 marks "no candidate".
__device__ __forceinline__ uint32_t key_of(float f) { return order_key(f); }
__device__ __forceinline__ uint64_t key_of(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f == 0.0 ? 0.0 : f);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = __reduce_max_sync(kFull, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kFull, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}
template <typename S>
__device__ __forceinline__ S warp_add(S v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ float score_exp(float x) { return expf(x); }
__device__ __forceinline__ double score_exp(double x) { return exp(x); }

template <typename S>
struct KeyOf;
template <>
struct KeyOf<float> { using T = uint32_t; };
template <>
struct KeyOf<double> { using T = uint64_t; };

// What one pass over a token leaves in lane j < k: the j-th pick.
struct Pick {
    int id;        // -1: none left
    float l;       // its logit
    bool close;    // 32-bit pass: some comparison was within the error of the scores (warp-uniform)
};

// One choice of a token in arithmetic S. l: the lane's cleaned logits (dead:
// -inf); lmax: the largest live logit of the token (finite if any is live).
// lbuf: this warp's room for E scores of S.
template <int EPL, typename S>
__device__ __forceinline__ Pick choose(const RouteArgs &a, const float (&l)[EPL], float lmax, int lane, float *lbuf) {
    using Key = typename KeyOf<S>::T;
    constexpr bool k32 = sizeof(S) == 4;
    const int e0 = lane * EPL;
    const bool staged = a.keep < a.groups;
    const bool by_logit = a.bias == nullptr;             // the picks' order needs no score
    const bool need_p = !by_logit || (staged && a.top2);
    S p[EPL];
    S z = 1;
    if (need_p) {
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) p[i] = (S)1 / ((S)1 + score_exp(-(S)l[i]));
        } else {
            S s = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                p[i] = l[i] > -INFINITY ? score_exp((S)l[i] - (S)lmax) : (S)0;
                s += p[i];
            }
            z = warp_add(s);
            if (z == 0) z = 1;  // no live expert
#pragma unroll
            for (int i = 0; i < EPL; ++i) p[i] = p[i] / z;
        }
    }
    // bound on the error of a 32-bit score: sigmoid within 4 ulp; softmax: the
    // exponent's argument is off by up to 2^-24 |l - lmax|, which costs
    // exp(-t) t 2^-24 <= 0.37 * 2^-24 of the largest score, and the sum of up
    // to 512 terms carries about 25 roundings
    // (err <= 2^-20 of 1, or 2^-18 of the largest score 1 / z, for either)
    const S err = a.sigmoid ? (S)0x1p-20f : (S)0x1p-18f / z;
    S c[EPL];
    uint32_t on = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        c[i] = need_p ? p[i] : (S)l[i];
        bool live = l[i] > -INFINITY;
        if (!by_logit && live) {
            const float b = __ldg(a.bias + e0 + i);
            live = b > -INFINITY;                        // also false for NaN
            c[i] += (S)fminf(b, 3.402823466e38f);
        }
        on |= live ? 1u << i : 0u;
    }
    bool close = false;
    if (staged) {
        const bool exact = by_logit && !a.top2;
        const int gs = a.E / a.groups;
        // best and second best of every group: lane g walks group g
        S *buf = reinterpret_cast<S *>(lbuf);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e0 + i < a.E) buf[e0 + i] = ((on >> i) & 1u) ? c[i] : (S)-INFINITY;
        __syncwarp();
        S b1 = -INFINITY, b2 = -INFINITY;
        if (lane < a.groups)
            for (int i = 0; i < gs; ++i) {
                const S v = buf[lane * gs + i];
                if (v > b1) {
                    b2 = b1;
                    b1 = v;
                } else if (v > b2) {
                    b2 = v;
                }
            }
        __syncwarp();
        S score = b1;
        if (a.top2 && b2 > (S)-INFINITY) score = b1 + b2;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const S o = __shfl_sync(kFull, score, g);
            rank += (o > score || (o == score && g < lane)) ? 1 : 0;
        }
        const bool kept = lane < a.groups && rank < a.keep && b1 > (S)-INFINITY;
        const uint32_t mask = __ballot_sync(kFull, kept);
        if (k32 && !exact) {
            // the border: the worst kept group against the best one left out;
            // two scores make a group's, each rounded once more with its bias
            S lo = kept ? score : (S)INFINITY;
            S hi = (lane < a.groups && !kept) ? score : (S)-INFINITY;
            S mag = lane < a.groups && b1 > (S)-INFINITY ? fabs(b1) + (b2 > (S)-INFINITY ? fabs(b2) : (S)0) : (S)0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const S vl = __shfl_xor_sync(kFull, lo, o), vh = __shfl_xor_sync(kFull, hi, o);
                const S vm = __shfl_xor_sync(kFull, mag, o);
                lo = vl < lo ? vl : lo;
                hi = vh > hi ? vh : hi;
                mag = vm > mag ? vm : mag;
            }
            const S tol = (S)4 * err + (S)0x1p-21f * mag;
            close = hi > (S)-INFINITY && lo - hi <= tol;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (e0 + i >= a.E || !((mask >> ((e0 + i) / gs)) & 1u)) on &= ~(1u << i);
            if (by_logit) c[i] = (S)l[i];
        }
    }
    Key key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = ((on >> i) & 1u) ? key_of(c[i]) : (Key)0;
    Pick r{-1, -INFINITY, false};
    S mine = 0;
    const int npick = k32 && !by_logit ? a.k + 1 : a.k;  // one more: the border
    for (int j = 0; j < npick; ++j) {
        Key bk = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < EPL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = i;
            }
        const Key m = warp_max(bk);
        if (m == 0) break;
        const int win = __ffs(__ballot_sync(kFull, bk == m)) - 1;
        float lw = 0.f;
        S cw = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i == bi) {
                lw = l[i];
                cw = c[i];
                if (lane == win) key[i] = 0;
            }
        const int id = __shfl_sync(kFull, e0 + bi, win);
        lw = __shfl_sync(kFull, lw, win);
        cw = __shfl_sync(kFull, cw, win);
        if (lane == j) {
            r.id = id;
            r.l = lw;
            mine = cw;
        }
    }
    if (k32 && !by_logit) {
        const int nid = __shfl_down_sync(kFull, r.id, 1);
        const float nl = __shfl_down_sync(kFull, r.l, 1);
        const S nc = __shfl_down_sync(kFull, mine, 1);
        if (lane < a.k && nid >= 0) {
            const S tol = (S)2 * err + (S)0x1p-22f * (fabs(mine) + fabs(nc));
            if (mine - nc <= tol && !(r.l == nl && __ldg(a.bias + r.id) == __ldg(a.bias + nid))) close = true;
        }
        close = __any_sync(kFull, close);
        if (lane == a.k) r.id = -1;
    }
    r.close = close;
    return r;
}

// The 64-bit choice, out of line: few tokens take it.
template <int EPL>
__device__ __noinline__ Pick choose_again(const RouteArgs &a, const float (&l)[EPL], float lmax, int lane, float *lbuf) {
    return choose<EPL, double>(a, l, lmax, lane, lbuf);
}

// The weight of lane j's pick (lanes >= k or without a pick: 0).
template <int EPL>
__device__ __forceinline__ float pick_weight(const RouteArgs &a, const float (&l)[EPL], float lmax, const Pick &r,
                                             int lane) {
    const bool on = r.id >= 0;
    float w = 0.f;
    if (a.renorm) {
        float top = on ? r.l : -INFINITY;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
        // sigmoid(l) = exp(l) to within exp(-60) below -60: the quotient is
        // then that of the exponentials, which does not underflow
        if (on) w = a.sigmoid && top >= -60.f ? 1.f / (1.f + expf(-r.l)) : expf(r.l - top);
        const float s = warp_add(w);
        if (on) w = w / s;
    } else if (a.sigmoid) {
        if (on) w = 1.f / (1.f + expf(-r.l));
    } else {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s += l[i] > -INFINITY ? expf(l[i] - lmax) : 0.f;
        s = warp_add(s);
        if (on) w = expf(r.l - lmax) / s;
    }
    return on ? w * a.scale : 0.f;
}

// One CTA per chunk of tokens: ids and weights, and the chunk's count of every expert.
template <int EPL>
__global__ void __launch_bounds__(kSelThreads) route_select_kernel(RouteArgs a) {
    __shared__ int32_t cnt[kRouteMaxE];
    __shared__ __align__(8) float lbuf[kSelThreads / 32][2 * kRouteMaxE];  // a warp's scores (up to 64 bits each)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int e = tid; e < a.E; e += kSelThreads) cnt[e] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * a.chunk, t1 = min(t0 + a.chunk, a.T);
    for (int t = t0 + warp; t < t1; t += kSelThreads / 32) {
        float l[EPL];
        load_lane<EPL>(a, (int64_t)t * a.stride, lane * EPL, l);
        float lmax = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            l[i] = l[i] > -INFINITY ? fminf(l[i], 3.402823466e38f) : -INFINITY;  // NaN and -inf: dead
            lmax = fmaxf(lmax, l[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(kFull, lmax, o));
        Pick r = choose<EPL, float>(a, l, lmax, lane, lbuf[warp]);
        if (r.close) r = choose_again<EPL>(a, l, lmax, lane, lbuf[warp]);
        const float w = pick_weight<EPL>(a, l, lmax, r, lane);
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = r.id;
            a.w[(size_t)t * a.k + lane] = w;
            if (r.id >= 0) atomicAdd(&cnt[r.id], 1);
        }
    }
    if (!a.chunk_cnt) return;
    __syncthreads();
    for (int e = tid; e < a.E; e += kSelThreads) a.chunk_cnt[(size_t)blockIdx.x * a.E + e] = cnt[e];
}

// Exclusive scan of a[0..n) (n <= kRouteMaxE) by one warp; returns the total.
__device__ int warp_scan(const int32_t *a, int32_t *out, int n, int lane) {
    constexpr int P = kRouteMaxE / 32;
    int v[P], local = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        v[i] = lane * P + i < n ? a[lane * P + i] : 0;
        local += v[i];
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    int run = incl - local;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (lane * P + i < n) out[lane * P + i] = run;
        run += v[i];
    }
    return __shfl_sync(kFull, incl, 31);
}

constexpr int kPermThreads = 512;
constexpr int kPermSmem = 2 * kRouteMaxE * (kRouteMaxT / kRouteMaxChunks / 32) * 4;  // both tables at the largest chunk

// One CTA per chunk: the rows of its pairs. Expert e's rows are offsets[e] ..,
// its tokens ascending: row = offsets[e] + (pairs of e in earlier chunks) +
// (tokens of e earlier in the chunk), the last from a bitmap of the chunk's
// tokens per expert, so the result does not depend on the order of threads.
__global__ void __launch_bounds__(kPermThreads) route_permute_kernel(RouteArgs a, int nch) {
    extern __shared__ uint32_t bm[];                 // [E][words] bitmaps, then [E][words] pairs in earlier words
    __shared__ int32_t tot[kRouteMaxE], base[kRouteMaxE], off[kRouteMaxE + 1], tmp[kRouteMaxE];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.E, words = a.chunk / 32, c = blockIdx.x;
    uint32_t *before = bm + (size_t)E * words;
    for (int i = tid; i < E * words; i += kPermThreads) bm[i] = 0u;
    pdl_wait();
    for (int e = tid; e < E; e += kPermThreads) {
        int pre = 0, all = 0;
#pragma unroll 8
        for (int ch = 0; ch < nch; ++ch) {
            const int v = __ldcg(a.chunk_cnt + (size_t)ch * E + e);
            all += v;
            pre += ch < c ? v : 0;
        }
        tot[e] = all;
        base[e] = pre;
    }
    __syncthreads();
    const int t0 = c * a.chunk, nt = min(a.chunk, a.T - t0);
    const int32_t *ids = a.ids + (size_t)t0 * a.k;
    for (int i = tid; i < nt * a.k; i += kPermThreads) {
        const int e = __ldcg(ids + i), t = i / a.k;
        if (e >= 0) atomicOr(&bm[e * words + (t >> 5)], 1u << (t & 31));
    }
    if (warp == 0) {
        const int total = warp_scan(tot, off, E, lane);
        if (lane == 0) off[E] = total;
        if (c == 0 && a.uniq) {
            for (int e = lane; e < E; e += 32) tmp[e] = tot[e] > 0 ? 1 : 0;
            __syncwarp();
            const int nu = warp_scan(tmp, tmp, E, lane);
            __syncwarp();
            for (int e = lane; e < E; e += 32)
                if (tot[e] > 0) a.uniq[tmp[e]] = e;
            __syncwarp();
            for (int e = lane; e < E; e += 32) tmp[e] = (tot[e] + 127) >> 7;
            __syncwarp();
            const int ntile = warp_scan(tmp, tmp, E, lane);
            __syncwarp();
            for (int e = lane; e < E; e += 32) a.tile_off[e] = tmp[e];
            if (lane == 0) {
                a.tile_off[E] = ntile;
                *a.n_uniq = nu;
                *a.n_tiles = ntile;
            }
        }
    }
    __syncthreads();
    for (int e = tid; e < E; e += kPermThreads) {
        uint32_t run = 0;
        for (int w = 0; w < words; ++w) {
            before[e * words + w] = run;
            run += __popc(bm[e * words + w]);
        }
        if (c == 0) {
            if (a.counts) a.counts[e] = tot[e];
            if (a.offsets) a.offsets[e] = off[e];
        }
    }
    if (c == 0 && tid == 0 && a.offsets) a.offsets[E] = off[E];
    __syncthreads();
    for (int i = tid; i < nt * a.k; i += kPermThreads) {
        const int e = __ldcg(ids + i), t = i / a.k;
        int row = -1;
        if (e >= 0) {
            const int w = e * words + (t >> 5);
            row = off[e] + base[e] + (int)before[w] + __popc(bm[w] & ((1u << (t & 31)) - 1u));
            if (a.perm) a.perm[row] = t0 + t;
        }
        if (a.pos) a.pos[(size_t)t0 * a.k + i] = row;
    }
    if (a.perm)
        for (int64_t i = off[E] + (int64_t)c * kPermThreads + tid; i < (int64_t)a.T * a.k; i += (int64_t)nch * kPermThreads)
            a.perm[i] = a.perm_fill;
}

template <int EPL>
cudaError_t launch_select(const RouteArgs &a, int nch, cudaStream_t st) {
    route_select_kernel<EPL><<<nch, kSelThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route_logits(RouteArgs a, cudaStream_t st, int *launches) {
    a.chunk = route_chunk_tokens(a.T);
    const int nch = (a.T + a.chunk - 1) / a.chunk;
    const bool permute = a.counts || a.offsets || a.perm || a.pos || a.uniq;
    if (!permute) a.chunk_cnt = nullptr;
    const int epl = a.E <= 32 ? 1 : a.E <= 64 ? 2 : a.E <= 128 ? 4 : a.E <= 256 ? 8 : 16;
    const int size = a.type == MOE_T_F32 ? 4 : 2;
    const int align = epl * size < 16 ? epl * size : 16;
    a.vec = a.nsplit == 1 && a.E % epl == 0 && (uintptr_t)a.logits % align == 0 && (a.stride * size) % align == 0;
    cudaError_t e = epl == 1   ? launch_select<1>(a, nch, st)
                    : epl == 2 ? launch_select<2>(a, nch, st)
                    : epl == 4 ? launch_select<4>(a, nch, st)
                    : epl == 8 ? launch_select<8>(a, nch, st)
                               : launch_select<16>(a, nch, st);
    if (launches) ++*launches;
    if (e != cudaSuccess || !permute) return e;
    const size_t smem = (size_t)2 * a.E * (a.chunk / 32) * 4;
    static std::atomic<uint64_t> attr_set{0};
    e = set_smem_limit_once((const void *)route_permute_kernel, kPermSmem, attr_set);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(nch);
    cfg.blockDim = dim3(kPermThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (launches) ++*launches;
    return cudaLaunchKernelEx(&cfg, route_permute_kernel, a, nch);
}

}  // namespace moe
