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
// logits, which needs no score at all.
//
// One warp per token; lane l holds the EPL consecutive experts from l * EPL
// on. The (k + 1)-th largest of the lanes' maxima is a lower bound of the
// (k + 1)-th best expert: the few experts that reach it (about 13 for k = 8) are
// gathered one to a lane, in order of their ids, and ranked by comparing each
// with all. That takes half the instructions of k rounds of "best of all". Where
// over 32 reach it (the live experts lie in few lanes) they are spread first: 140
// tokens of 272 experts, 3 of 8 groups kept, 42 -> 14 us (always spreading where
// few lanes are kept: 30011 tokens of 160 experts, 47 -> 51 us).
// The kernel is bound by its instructions: 1060 a token for 160 experts in 8
// groups (30011 tokens: 47 us, of it 12 of permutation; issue slots 59 % used).
#include <math.h>

#include "ops.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kSelThreads = 1024, kPermThreads = 512;
constexpr int kSelSmem = 32 * (2 * kRouteMaxE + 192) * 4;              // 32 warps' scores
constexpr int kPermSmem = 2 * kRouteMaxE * ((kRouteMaxT / kRouteMaxChunks + 47) / 32) * 4;  // both tables at the largest chunk

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

// Order-preserving unsigned keys; 0, that of -inf, marks "no candidate". Both
// zeros have the same. Not for NaN.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);
    return (u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u)) - 0x007FFFFFu;
}
__device__ __forceinline__ float value_of(uint32_t key) { return key_value(key + 0x007FFFFFu); }
__device__ __forceinline__ uint64_t key_of(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f == 0.0 ? 0.0 : f);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
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
// NaN and -inf as -inf, +inf as the largest finite float (fmaxf takes NaN for the other operand).
__device__ __forceinline__ float clean(float f) { return fminf(fmaxf(f, -INFINITY), 3.402823466e38f); }
// load_lane, cleaned.
template <int EPL>
__device__ __forceinline__ void load_clean(const RouteArgs &a, int64_t row, int e0, float l[EPL]) {
    load_lane<EPL>(a, row, e0, l);
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = clean(l[i]);
}

// What a choice leaves in a lane: an expert, its logit and its place among the
// picks (the first k count).
struct Pick {
    int id;        // -1: none
    float l;
    int rank;
};

// The logit of expert e of a row (lane by lane), cleaned as in the kernel.
__device__ __forceinline__ float one_logit(const RouteArgs &a, int64_t row, int e) {
    float l = load_logit(a.logits, row + e, a.type);
    for (int s = 1; s < a.nsplit; ++s) l += ((const float *)a.logits)[row + s * a.split_stride + e];
    return fminf(l, 3.402823466e38f);
}

// The `want`-th largest of the lanes' largest keys: at most the want-th largest
// key of all. 1 where fewer lanes have any.
template <int EPL>
__device__ __forceinline__ uint32_t lane_bound(const uint32_t (&key)[EPL], int want) {
    uint32_t top = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) top = max(top, key[i]);
    uint32_t m = 0u;
    for (int j = 0; j < want;) {
        m = __reduce_max_sync(kFull, top);
        const bool hit = top == m;               // no key left: every lane, and the loop ends
        j += __popc(__ballot_sync(kFull, hit));
        if (hit) top = 0u;
    }
    return max(m, 1u);
}

// Gathers the experts whose keys reach `bound`, ids ascending, one to a lane
// (key 0: none), and returns how many they are; over 32 (many equal keys),
// nothing is gathered.
template <int EPL>
__device__ __forceinline__ int gather_from(const uint32_t (&key)[EPL], uint32_t bound, int lane, uint2 *cand,
                                           uint32_t *my_key, int *my_id) {
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) cnt += key[i] >= bound ? 1 : 0;
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    const int n = __shfl_sync(kFull, incl, 31);
    *my_key = 0u;
    *my_id = -1;
    if (n > 32) return n;
    __syncwarp();
    uint2 *at = cand + (incl - cnt);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (key[i] >= bound) *at++ = make_uint2(key[i], (uint32_t)(lane * EPL + i));
    __syncwarp();
    if (lane < n) {
        const uint2 v = cand[lane];
        *my_key = v.x;
        *my_id = (int)v.y;
    }
    return n;
}

// The rest of gather_spread: cand holds the live keys, behind them (at cand + E)
// room for 32 pairs.
struct Gathered {
    uint32_t bound, key;
    int n, id;
};
__device__ __noinline__ Gathered gather_live(const uint2 *cand, uint2 *out, int live, int want, float slack, float rel,
                                             int lane) {
    uint32_t top[1] = {0u};
    for (int p = lane; p < live; p += 32) top[0] = max(top[0], cand[p].x);
    Gathered r;
    r.bound = lane_bound<1>(top, want);
    if (slack >= 0.f && r.bound > 1u) {
        const float x = value_of(r.bound);
        r.bound = max(key_of(x - (slack + rel * fabsf(x))), 1u);
    }
    r.n = 0;
    for (int p0 = 0; p0 < live; p0 += 32) {
        const uint2 v = p0 + lane < live ? cand[p0 + lane] : make_uint2(0u, 0u);
        const uint32_t hits = __ballot_sync(kFull, v.x >= r.bound);
        const int to = r.n + __popc(hits & ((1u << lane) - 1u));
        if (v.x >= r.bound && to < 32) out[to] = v;
        r.n += __popc(hits);
    }
    __syncwarp();
    const bool mine = r.n <= 32 && lane < r.n;
    r.key = mine ? out[lane].x : 0u;
    r.id = mine ? (int)out[lane].y : -1;
    return r;
}

// gather_from for keys that lie in few lanes (kept groups, or E much below 32
// EPL), where the lanes' maxima say little: the live keys are first spread over
// all lanes, item 32 j + lane in order of the ids. The bound: the `want`-th largest
// of those lanes' maxima, less slack + rel |bound| where slack is not negative.
// cand: room for E pairs and 32 more.
template <int EPL>
__device__ __forceinline__ Gathered gather_spread(const RouteArgs &a, const uint32_t (&key)[EPL], int want, float slack,
                                                  float rel, int lane, uint2 *cand) {
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) cnt += key[i] != 0u ? 1 : 0;
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    __syncwarp();
    uint2 *at = cand + (incl - cnt);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (key[i] != 0u) *at++ = make_uint2(key[i], (uint32_t)(lane * EPL + i));
    __syncwarp();
    return gather_live(cand, cand + a.E, __shfl_sync(kFull, incl, 31), want, slack, rel, lane);
}

// The place of a lane's key among n gathered ones; ties to the lower lane.
__device__ __forceinline__ int rank_of(uint32_t key, int n, int lane) {
    int rank = __popc(__match_any_sync(kFull, key) & ((1u << lane) - 1u));
    for (int j = 0; j < n; ++j) rank += __shfl_sync(kFull, key, j) > key ? 1 : 0;
    return rank;
}

// The scores of a lane's experts in 32 bits (c; -inf: not to be chosen), and a
// bound on the error of a score. `scored`: false where the order of the logits
// serves.
//
// Errors. Sigmoid by the fast exponential and reciprocal: the exponent's
// relative error of (2 + 1.2 |l|) 2^-23 enters the score times p (1 - p), at
// most 0.64 * 2^-23; with the sum's and the reciprocal's roundings under
// 2.2 * 2^-23: 2^-21 is allowed. Softmax, relative to a score p = exp(-t) / z, t
// its logit's distance from the largest: its term's (2 + 1.2 t) 2^-23 and the
// rounding of t, 0.5 t 2^-23; z's, a mean of the same over the terms (t weighted
// with exp(-t) is at most 3.9 for 512 of them: 8.7 * 2^-23) and 25 roundings; the
// quotient's 2 * 2^-23: under (26 + 1.7 t) 2^-23. own_err allows (32 + 1.9 t)
// 2^-23, and 2^-18 / z is above that for every t. The bias adds a rounding of
// 2^-24 of the sum.
template <int EPL>
__device__ __forceinline__ float score_lane(const RouteArgs &a, const float (&l)[EPL], float lmax, int e0, bool scored,
                                            float (&c)[EPL]) {
    if (!scored) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = l[i];
        return 0.f;
    }
    float err;
    if (a.sigmoid) {
        err = 0x1p-21f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = l[i] > -INFINITY ? __fdividef(1.f, 1.f + __expf(-l[i])) : -INFINITY;
    } else {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            c[i] = __expf(l[i] - lmax);          // (a token without any expert: NaN, and all -inf below)
            s += c[i];
        }
        s = warp_add(s);
        const float inv_z = s > 0.f ? 1.f / s : 1.f;
        err = 0x1p-18f * inv_z;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = l[i] > -INFINITY ? c[i] * inv_z : -INFINITY;
    }
    if (a.bias) {
        float b[EPL];
        if (a.vec_bias && EPL >= 4 && e0 < a.E) {
#pragma unroll
            for (int i = 0; i + 3 < EPL; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(a.bias + e0 + i));
                b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) b[i] = e0 + i < a.E ? __ldg(a.bias + e0 + i) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] += clean(b[i]);
    }
    return err;
}

__device__ __forceinline__ float own_err(const RouteArgs &a, float err, float l, float lmax) {
    const float t = fminf(lmax - l, 1e3f);       // (the exponential is 0 from 104 on)
    return a.sigmoid ? err : err * __expf(-t) * (1.f + 0.06f * t) + 1e-37f;
}

// The best (a.top2: two best) of every group, with the lpg lanes of a group (a
// power of two). Where the groups are whole lanes (a.direct) those lanes hold the
// group themselves; else 32 / groups lanes or fewer walk it in shared memory
// (element e lies at e + e / 32: groups a multiple of 32 apart would share a bank).
template <int EPL, typename S>
__device__ __forceinline__ void group_best(const RouteArgs &a, const S (&c)[EPL], int lane, S *buf, S &b1, S &b2) {
    const int e0 = lane * EPL, gs = a.E / a.groups, lpg = a.lanes_per_group, sub = lane & (lpg - 1), g = lane / lpg;
    constexpr bool kPad = sizeof(S) == 4;        // doubles: room for E of them only
    S m1 = (S)-INFINITY, m2 = (S)-INFINITY;
    auto take = [&](S v) {
        if (a.top2) {
            const S low = m1 < v ? m1 : v;
            m2 = m2 > low ? m2 : low;
        }
        m1 = m1 > v ? m1 : v;
    };
    if (a.direct) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) take(c[i]);
    } else {
        __syncwarp();
        S *at = buf + e0 + (kPad ? e0 >> 5 : 0);  // EPL divides 32
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (kPad || e0 + i < a.E) at[i] = c[i];
        __syncwarp();
        if (g < a.groups)
            for (int e = g * gs + sub; e < g * gs + gs; e += lpg) take(buf[e + (kPad ? e >> 5 : 0)]);
    }
    for (int o = lpg >> 1; o > 0; o >>= 1) {
        const S v = __shfl_xor_sync(kFull, m1, o);
        if (a.top2) {
            const S v2 = __shfl_xor_sync(kFull, m2, o);
            m2 = m2 > v2 ? m2 : v2;
        }
        take(v);
    }
    b1 = m1, b2 = m2;
}

// Whether this lane's group is among the `keep` best by `score`; the ballot has
// a kept group's bits at its lanes.
template <typename S>
__device__ __forceinline__ bool group_kept(const RouteArgs &a, S score, bool any, int lane) {
    const int lpg = a.lanes_per_group, sub = lane & (lpg - 1), g = lane / lpg;
    int rank = 0;                                         // each lane compares with every lpg-th group
    for (int o0 = 0; o0 < a.groups; o0 += lpg) {
        const int o = o0 + sub;
        const S v = __shfl_sync(kFull, score, (o * lpg) & 31);
        rank += o < a.groups && (v > score || (v == score && o < g)) ? 1 : 0;
    }
    for (int o = lpg >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(kFull, rank, o);
    return g < a.groups && rank < a.keep && any;
}

// Bits of a lane's experts that lie in kept groups.
template <int EPL>
__device__ __forceinline__ uint32_t in_kept_groups(const RouteArgs &a, bool kept, int e0) {
    if (a.direct) return kept ? kFull : 0u;
    const int gs = a.E / a.groups, lpg = a.lanes_per_group;
    const uint32_t mask = __ballot_sync(kFull, kept);
    if (gs >= EPL) {                             // two groups at most
        const int g = (int)(((uint32_t)e0 * a.group_inv) >> 22), rem = (g + 1) * gs - e0;
        const uint32_t first = rem >= 32 ? kFull : (1u << rem) - 1u;
        return (((mask >> ((g * lpg) & 31)) & 1u) ? first : 0u) | (((mask >> (((g + 1) * lpg) & 31)) & 1u) ? ~first : 0u);
    }
    uint32_t in = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const uint32_t gi = ((uint32_t)(e0 + i) * a.group_inv) >> 22;  // (e0 + i) / group size
        in |= ((mask >> ((gi * lpg) & 31u)) & 1u) << i;
    }
    return in;
}

// The largest upper end of the scores of the experts that `in` says (a lane's bits) less the gathered ones (`id`, one a
// lane or -1); -inf where there are none. One copy of the code: few tokens come here.
template <int EPL>
__device__ __noinline__ float upper_end_of_rest(const RouteArgs &a, int64_t row, float lmax, int lane, uint32_t in, int id,
                                                int n) {
    float l[EPL], c[EPL];
    load_clean<EPL>(a, row, lane * EPL, l);
    const float err = score_lane<EPL>(a, l, lmax, lane * EPL, true, c);
    for (int j = 0; j < n; ++j) {
        const int i = __shfl_sync(kFull, id, j) - lane * EPL;
        if (i >= 0 && i < EPL) in &= ~(1u << i);
    }
    float hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (((in >> i) & 1u) && c[i] > -INFINITY) hi = fmaxf(hi, c[i] + own_err(a, err, l[i], lmax) + 0x1p-22f * fabsf(c[i]));
    return value_of(__reduce_max_sync(kFull, key_of(hi)));
}

constexpr int kAll = -1, kGroups = -2;

// The choice in 32 bits; *close (warp-uniform) says that some comparison was
// within the error of what was compared, or that over 32 experts tied; *again
// then: kGroups, the groups' border was close; n (>= 0), only some of the n
// gathered experts were, which no other can reach; kAll, anything else. buf: room
// for E + E / 32 floats, and for 32 pairs.
template <int EPL>
__device__ __forceinline__ Pick choose_fast(const RouteArgs &a, const float (&l)[EPL], float lmax, int64_t row, int lane,
                                            float *buf, bool *close, int *again) {
    const int e0 = lane * EPL;
    const bool staged = a.keep < a.groups, by_logit = a.bias == nullptr;
    float c[EPL];
    const float err = score_lane<EPL>(a, l, lmax, e0, !by_logit || (staged && a.top2), c);
    bool near = false, near_groups = false;
    uint32_t in = kFull;
    if (staged) {
        float b1, b2;
        group_best<EPL, float>(a, c, lane, buf, b1, b2);
        const bool any = b1 > -INFINITY, is_group = lane / a.lanes_per_group < a.groups;
        const float score = a.top2 && b2 > -INFINITY ? b1 + b2 : b1;
        const bool kept = group_kept(a, score, any, lane);
        if (!by_logit || a.top2) {
            // the border: the worst kept group against the best one left out;
            // two scores make a group's, each rounded once more with its bias
            const uint32_t lo = ~__reduce_max_sync(kFull, kept ? ~key_of(score) : 0u);
            const uint32_t hi = __reduce_max_sync(kFull, is_group && any && !kept ? key_of(score) : 0u);
            const uint32_t mag = __reduce_max_sync(
                kFull, any ? __float_as_uint(fabsf(b1) + (b2 > -INFINITY ? fabsf(b2) : 0.f)) : 0u);
            near_groups = hi != 0u && !(value_of(lo) - value_of(hi) > 4.f * err + 0x1p-22f * __uint_as_float(mag));
        }
        in = in_kept_groups<EPL>(a, kept, e0);
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = ((in >> i) & 1u) ? (by_logit ? l[i] : c[i]) : -INFINITY;
    }
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = key_of(c[i]);
    uint32_t mine;
    Pick r{-1, -INFINITY, 0};
    uint32_t bound = lane_bound<EPL>(key, a.k + 1);
    uint2 *cand = reinterpret_cast<uint2 *>(buf);
    int n = gather_from<EPL>(key, bound, lane, cand, &mine, &r.id);
    if (EPL > 1 && n > 32) {
        const Gathered s = gather_spread<EPL>(a, key, a.k + 1, -1.f, 0.f, lane, cand);
        bound = s.bound, mine = s.key, n = s.n, r.id = s.id;
    }
    near |= n > 32;
    bool within = false;
    r.rank = rank_of(mine, min(n, 32), lane);
    if (r.id >= 0) r.l = one_logit(a, row, r.id);
    if (!by_logit) {
        // Each pick against all that follow it. A softmax score's error grows with the score, so an expert that a bias
        // holds back to far below the picks may belong above them while the one next to them does not: the next one
        // is taken with the largest error of all, and only where that does not do, each with its own (30011 tokens of
        // 160 experts with a bias: 40.4 us, 43.5 with the second step for every token).
        __syncwarp();
        const bool one = r.id >= 0;
        const float own = one ? own_err(a, err, r.l, lmax) : 0.f, v = value_of(mine);
        const float most = a.sigmoid ? err : __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(own)));
        if (one) buf[r.rank] = v;
        __syncwarp();
        bool next = false;
        if (one && r.rank < a.k && r.rank + 1 < n) {
            const float x = buf[r.rank + 1];
            next = !(v - x > own + most + 0x1p-22f * fmaxf(fabsf(v), fabsf(x)));
        }
        if (!a.sigmoid && __any_sync(kFull, next)) {
            if (one) buf[32 + r.rank] = own;
            __syncwarp();
            // lane r: the lower end of the score at rank r against the largest upper end behind it
            const float u = lane < n ? buf[lane] : -INFINITY;
            const float slack = lane < n ? buf[32 + lane] + 0x1p-22f * fabsf(u) : 0.f;
            float hi = u + slack;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) hi = fmaxf(hi, __shfl_down_sync(kFull, hi, o));  // (past the warp: itself)
            const float behind = __shfl_down_sync(kFull, hi, 1);
            next = lane < a.k && lane + 1 < n && !(u - slack > behind);
        }
        near |= next;
        // what was not gathered lies below the bound, its error below the largest; else, for a softmax, each with its own
        if (n > 0 && n <= 32) {
            const float w = buf[min(n, a.k) - 1], x = value_of(bound);
            within = bound == 1u || w - x > 2.f * err + 0x1p-22f * fmaxf(fabsf(w), fabsf(x));
            if (!a.sigmoid && !within) {
                const float lo = one && r.rank < a.k ? v - (own + 0x1p-22f * fabsf(v)) : INFINITY;
                within = value_of(__reduce_min_sync(kFull, key_of(lo))) >
                         upper_end_of_rest<EPL>(a, row, lmax, lane, in, r.id, n);
                near |= !within;
            }
        }
    }
    *close = __any_sync(kFull, near) || near_groups;
    *again = near_groups ? kGroups : within ? n : kAll;
    return r;
}

// One copy of the code, and loops that stay loops: the 64-bit steps run for few
// tokens, by warps that find none of it in the instruction cache (1225 tokens of
// 455 experts, some decided in 64 bits: 41 us with the sum unrolled over 16 experts
// a lane, 32 us so, 19 us where no token is close).
__device__ __noinline__ double exp64(double x) { return exp(x); }

// The softmax's sum in 64 bits (1 where no expert is live).
__device__ __noinline__ double sum64(const RouteArgs &a, int64_t row, float lmax, int lane) {
    double s = 0.0;
    auto load = [&](int e) {
        if (e >= a.E) return -INFINITY;
        float l = load_logit(a.logits, row + e, a.type);
        for (int i = 1; i < a.nsplit; ++i) l += ((const float *)a.logits)[row + i * a.split_stride + e];
        return l;
    };
    float next = load(lane);
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) {
        const float l = next;
        next = load(e + 32);
        if (l > -INFINITY) s += exp64((double)fminf(l, 3.402823466e38f) - (double)lmax);
    }
    s = warp_add(s);
    return s > 0.0 ? s : 1.0;
}

// A score in 64 bits.
__device__ __forceinline__ double score64(const RouteArgs &a, float l, float lmax, double z, int e) {
    double p;
    const double x = exp64(a.sigmoid ? -(double)l : (double)l - (double)lmax);
    p = a.sigmoid ? 1.0 / (1.0 + x) : x / z;
    return a.bias ? p + (double)fminf(__ldg(a.bias + e), 3.402823466e38f) : p;
}

// The choice in 64 bits of every expert, for tokens where over 32 of them tie
// or nearly do. buf: room for E doubles.
template <int EPL>
__device__ __noinline__ Pick choose_general(const RouteArgs &a, int64_t row, float lmax, int lane, float *buf) {
    const int e0 = lane * EPL;
    const bool staged = a.keep < a.groups, by_logit = a.bias == nullptr;
    float l[EPL], c[EPL];
    load_clean<EPL>(a, row, e0, l);
    const bool scored = !by_logit || (staged && a.top2);
    score_lane<EPL>(a, l, lmax, e0, scored, c);
    double z = 1.0, d[EPL];
    if (scored && !a.sigmoid) z = sum64(a, row, lmax, lane);
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = scored && c[i] > -INFINITY ? score64(a, l[i], lmax, z, e0 + i) : (double)c[i];
    if (staged) {
        double b1, b2;
        group_best<EPL, double>(a, d, lane, reinterpret_cast<double *>(buf), b1, b2);
        const bool kept = group_kept(a, a.top2 && b2 > -INFINITY ? b1 + b2 : b1, b1 > -INFINITY, lane);
        const uint32_t in = in_kept_groups<EPL>(a, kept, e0);
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] = ((in >> i) & 1u) ? (by_logit ? (double)l[i] : d[i]) : -INFINITY;
    }
    uint64_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = d[i] > -INFINITY ? key_of(d[i]) : 0ull;
    Pick r{-1, -INFINITY, lane};
    for (int j = 0; j < a.k; ++j) {
        uint64_t bk = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < EPL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = i;
            }
        const uint64_t m = warp_max(bk);
        if (m == 0) break;
        const int win = __ffs(__ballot_sync(kFull, bk == m)) - 1;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i == bi && lane == win) key[i] = 0;
        const int id = __shfl_sync(kFull, e0 + bi, win);
        if (lane == j) r.id = id;
    }
    if (r.id >= 0) r.l = one_logit(a, row, r.id);
    return r;
}

// The choice in 64 bits, of those scores that can matter: one that lies further
// below its group's second best, or below the k-th pick, in 32 bits than the
// errors allow is left out; the others are gathered one to a lane. buf: room for
// E + E / 32 floats, and for 32 doubles and 32 words behind 32 pairs.
template <int EPL>
__device__ __noinline__ Pick choose_exact(const RouteArgs &a, int64_t row, float lmax, int lane, float *buf,
                                          bool near_groups) {
    const int e0 = lane * EPL, gs = a.E / a.groups;
    const bool staged = a.keep < a.groups, by_logit = a.bias == nullptr;
    const bool scored = !by_logit || (staged && a.top2);
    float l[EPL], c[EPL];
    load_clean<EPL>(a, row, e0, l);
    const float err = score_lane<EPL>(a, l, lmax, e0, scored, c);
    uint32_t in = kFull, key[EPL], mine;
    uint2 *cand = reinterpret_cast<uint2 *>(buf);
    double z = 1.0;
    if (scored && !a.sigmoid) z = sum64(a, row, lmax, lane);
    Pick r{-1, -INFINITY, lane};
    if (staged) {
        float f1, f2;
        group_best<EPL, float>(a, c, lane, buf, f1, f2);
        if (!near_groups) {                               // the 32-bit choice of the groups stands
            const float score = a.top2 && f2 > -INFINITY ? f1 + f2 : f1;
            in = in_kept_groups<EPL>(a, group_kept(a, score, f1 > -INFINITY, lane), e0);
        } else {
            const float thr = a.top2 ? f2 : f1;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t gi = ((uint32_t)min(e0 + i, a.E - 1) * a.group_inv) >> 22;
                const float tg = __shfl_sync(kFull, thr, (gi * a.lanes_per_group) & 31);
                const bool below = tg - c[i] > 2.f * err + 0x1p-21f * fmaxf(fabsf(tg), fabsf(c[i]));
                key[i] = c[i] > -INFINITY && !below ? 1u : 0u;
            }
            const int n = gather_from<EPL>(key, 1u, lane, cand, &mine, &r.id);
            if (n > 32) return choose_general<EPL>(a, row, lmax, lane, buf);
            double *val = reinterpret_cast<double *>(buf + 64);
            int *grp = reinterpret_cast<int *>(buf + 128);
            if (r.id >= 0) {
                val[lane] = score64(a, one_logit(a, row, r.id), lmax, z, r.id);
                grp[lane] = r.id / gs;
            }
            __syncwarp();
            double b1 = -INFINITY, b2 = -INFINITY;       // lane g: group g
            for (int j = 0; j < n; ++j) {
                const double v = val[j];
                if (grp[j] == lane) {
                    if (v > b1) b2 = b1, b1 = v;
                    else if (v > b2) b2 = v;
                }
            }
            const double score = a.top2 && b2 > -INFINITY ? b1 + b2 : b1;
            int rank = 0;
            for (int g = 0; g < a.groups; ++g) {
                const double o = __shfl_sync(kFull, score, g);
                rank += o > score || (o == score && g < lane) ? 1 : 0;
            }
            const uint32_t mask = __ballot_sync(kFull, lane < a.groups && rank < a.keep && b1 > -INFINITY);
            in = 0u;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t gi = ((uint32_t)(e0 + i) * a.group_inv) >> 22;
                in |= ((mask >> (gi & 31u)) & 1u) << i;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = ((in >> i) & 1u) ? key_of(by_logit ? l[i] : c[i]) : 0u;
    const Gathered s = gather_spread<EPL>(a, key, a.k, by_logit ? -1.f : 2.f * err, 0x1p-20f, lane, cand);
    const int n = s.n;
    mine = s.key, r.id = s.id;
    if (n > 32) return choose_general<EPL>(a, row, lmax, lane, buf);
    if (r.id >= 0) r.l = one_logit(a, row, r.id);
    if (by_logit) {
        r.rank = rank_of(mine, n, lane);
        return r;
    }
    const uint64_t k64 = r.id >= 0 ? key_of(score64(a, r.l, lmax, z, r.id)) : 0ull;
    r.rank = 0;
    for (int j = 0; j < n; ++j) {
        const uint64_t o = __shfl_sync(kFull, k64, j);
        r.rank += o > k64 - (j < lane ? 1ull : 0ull) ? 1 : 0;
    }
    return r;
}

// The places of n gathered experts by their scores in 64 bits.
__device__ __noinline__ int rank_exact(const RouteArgs &a, int64_t row, float lmax, int id, float l, int n, int lane) {
    const double z = a.sigmoid ? 1.0 : sum64(a, row, lmax, lane);
    const uint64_t k64 = id >= 0 ? key_of(score64(a, l, lmax, z, id)) : 0ull;
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const uint64_t o = __shfl_sync(kFull, k64, j);
        rank += o > k64 - (j < lane ? 1ull : 0ull) ? 1 : 0;
    }
    return rank;
}

// 1 / (1 + exp(-l)) with divisors of 1 to 2 (the fast division gives 0 for one past 2^126).
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return __fdividef(l < 0.f ? e : 1.f, 1.f + e);
}

// The weight of a lane's pick (`on`: it is one of the first k).
template <int EPL>
__device__ __forceinline__ float pick_weight(const RouteArgs &a, const float (&l)[EPL], float lmax, const Pick &r,
                                             bool on) {
    float w = 0.f;
    if (a.renorm) {
        // relative to the largest chosen score: at most 1, and their sum is
        // taken in fixed point, 2^-27, where it is 1 to 16
        const float top = value_of(__reduce_max_sync(kFull, on ? key_of(r.l) : 0u));
        // of two sigmoids: exp(l - top) (1 + exp(top)) / (1 + exp(l)) for a negative top, where every factor stays in
        // range however far below zero the logits lie
        if (on)
            w = !a.sigmoid   ? expf(r.l - top)
                : top < 0.f ? expf(r.l - top) * __fdividef(1.f + expf(top), 1.f + expf(r.l))
                            : (1.f + expf(-top)) * sigmoid(r.l);
        const uint32_t s = __reduce_add_sync(kFull, __float2uint_rn(w * 0x1p27f));
        w *= __fdividef(0x1p27f, (float)s);
    } else if (a.sigmoid) {
        if (on) w = sigmoid(r.l);
    } else {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s += __expf(l[i] - lmax);  // within 2^-20 of the sum
        s = warp_add(s);
        if (on) w = expf(r.l - lmax) / s;
    }
    return on ? w * a.scale : 0.f;
}

// ids and weights of a chunk's tokens, one warp per token, and the chunk's
// count of every expert in cnt. lbuf: 2 E + 192 floats per warp.
template <int EPL>
__device__ __forceinline__ void select_chunk(const RouteArgs &a, int c, int32_t *cnt, float *lbuf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    const int t0 = c * a.chunk, t1 = min(t0 + a.chunk, a.T);
    lbuf += warp * (2 * a.E + 192);
    for (int t = t0 + warp; t < t1; t += nw) {
        const int64_t row = (int64_t)t * a.stride;
        float l[EPL];
        load_clean<EPL>(a, row, lane * EPL, l);
        float lmax = 0.f;
        if (!a.sigmoid) {                                 // the softmax's largest logit
            float m = l[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
            lmax = value_of(__reduce_max_sync(kFull, key_of(m)));
        }
        bool close;
        int again;
        Pick r = choose_fast<EPL>(a, l, lmax, row, lane, lbuf, &close, &again);
        if (close) {
            if (again >= 0) r.rank = rank_exact(a, row, lmax, r.id, r.l, again, lane);
            else r = choose_exact<EPL>(a, row, lmax, lane, lbuf, again == kGroups);
        }
        const bool picked = r.id >= 0 && r.rank < a.k;
        const float w = pick_weight<EPL>(a, l, lmax, r, picked);
        int32_t *ids = a.ids + (size_t)t * a.k;
        float *ws = a.w + (size_t)t * a.k;
        if (picked) {
            ids[r.rank] = r.id;
            ws[r.rank] = w;
            atomicAdd(&cnt[r.id], 1);
        }
        const int n_picked = __popc(__ballot_sync(kFull, picked));
        if (lane < a.k && lane >= n_picked) {
            ids[lane] = -1;
            ws[lane] = 0.f;
        }
    }
}

// What a permutation keeps in shared memory besides its bitmaps.
struct PermSmem {
    int32_t tot[kRouteMaxE];       // all pairs of every expert
    int32_t base[kRouteMaxE];      // those in earlier chunks
    int32_t own[kRouteMaxE];       // those of this chunk
    int32_t off[kRouteMaxE + 1];
    int32_t wsum[kSelThreads / 32];
};

// Exclusive scan of v over the CTA's threads; *total their sum. Every thread calls it.
__device__ __forceinline__ int block_scan(int v, int32_t *wsum, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    const int s = lane < nw ? wsum[lane] : 0;
    int si = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, si, o);
        if (lane >= o) si += y;
    }
    *total = __shfl_sync(kFull, si, 31);
    return incl - v + __shfl_sync(kFull, si - s, warp);
}

// The chunk's tokens per expert as bitmaps bm[E][words] (cleared by the
// caller), the pairs in earlier words (bm + E * words), and the chunk's counts.
__device__ __forceinline__ void chunk_bitmaps(const RouteArgs &a, int c, PermSmem &sm, uint32_t *bm) {
    const int tid = threadIdx.x, nth = blockDim.x, E = a.E, words = (a.chunk + 31) / 32;
    const int t0 = c * a.chunk, nt = max(0, min(a.chunk, a.T - t0));
    const int32_t *ids = a.ids + (size_t)t0 * a.k;
    for (int i = tid; i < nt * a.k; i += nth) {
        const int e = __ldcg(ids + i), t = i / a.k;
        if (e >= 0) atomicOr(&bm[e * words + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    uint32_t *before = bm + E * words;
    for (int e = tid; e < E; e += nth) {
        uint32_t run = 0;
        for (int w = 0; w < words; ++w) {
            before[e * words + w] = run;
            run += __popc(bm[e * words + w]);
        }
        sm.own[e] = run;
    }
}

// offsets from sm.tot (every thread of the CTA, after its own writes of tot); returns the total.
__device__ __forceinline__ int expert_offsets(const RouteArgs &a, PermSmem &sm) {
    const int tid = threadIdx.x, nth = blockDim.x, E = a.E;
    __syncthreads();
    int run = 0, total;
    for (int e0 = 0; e0 < E; e0 += nth) {
        const int e = e0 + tid;
        const int o = block_scan(e < E ? sm.tot[e] : 0, sm.wsum, &total);
        if (e < E) sm.off[e] = run + o;
        run += total;
    }
    if (tid == 0) sm.off[E] = run;
    __syncthreads();
    return run;
}

// The rows of a chunk's pairs. Expert e's rows are offsets[e] .., its tokens
// ascending: row = offsets[e] + (pairs in earlier chunks) + (tokens of e earlier
// in the chunk), the last from the bitmaps, so the result does not depend on
// the order of threads.
__device__ __forceinline__ void place_chunk(const RouteArgs &a, int c, const PermSmem &sm, const uint32_t *bm) {
    const int tid = threadIdx.x, nth = blockDim.x, words = (a.chunk + 31) / 32;
    const uint32_t *before = bm + a.E * words;
    const int t0 = c * a.chunk, nt = max(0, min(a.chunk, a.T - t0));
    const int32_t *ids = a.ids + (size_t)t0 * a.k;
    for (int i = tid; i < nt * a.k; i += nth) {
        const int e = __ldcg(ids + i), t = i / a.k;
        int row = -1;
        if (e >= 0) {
            const int w = e * words + (t >> 5);
            row = sm.off[e] + sm.base[e] + (int)before[w] + __popc(bm[w] & ((1u << (t & 31)) - 1u));
            if (a.perm) a.perm[row] = t0 + t;
        }
        if (a.pos) a.pos[(size_t)t0 * a.k + i] = row;
    }
}

// The rest of the outputs, by CTA `b` of `nb`: the rows of perm past the last
// pair; the first CTA the counts, the offsets and a layer's tables.
__device__ __forceinline__ void finish_route(const RouteArgs &a, int b, int nb, int pairs, PermSmem &sm) {
    const int tid = threadIdx.x, nth = blockDim.x, E = a.E;
    if (a.perm)
        for (int64_t i = pairs + (int64_t)b * nth + tid; i < (int64_t)a.T * a.k; i += (int64_t)nb * nth)
            a.perm[i] = a.perm_fill;
    if (b != 0) return;
    for (int e = tid; e <= E; e += nth) {
        if (a.counts && e < E) a.counts[e] = sm.tot[e];
        if (a.offsets) a.offsets[e] = sm.off[e];
    }
    if (!a.uniq) return;
    int nu = 0, ntile = 0, total;
    for (int e0 = 0; e0 < E; e0 += nth) {
        const int e = e0 + tid, n = e < E ? sm.tot[e] : 0;
        const int u = block_scan(n > 0 ? 1 : 0, sm.wsum, &total);
        if (n > 0) a.uniq[nu + u] = e;
        nu += total;
        const int o = block_scan((n + 127) >> 7, sm.wsum, &total);
        if (e < E) a.tile_off[e] = ntile + o;
        ntile += total;
    }
    if (tid == 0) {
        a.tile_off[E] = ntile;
        *a.n_uniq = nu;
        *a.n_tiles = ntile;
    }
}

__device__ __forceinline__ int ld_cluster(const int32_t *p, int rank) {
    uint32_t ra;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ra) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Large batches, first launch: the choice, and the counts of every chunk in
// rows of `ep` (E rounded up to 8).
template <int EPL>
__global__ void __launch_bounds__(kSelThreads) route_select_kernel(const __grid_constant__ RouteArgs a, int ep) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int32_t cnt[kRouteMaxE];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    select_chunk<EPL>(a, blockIdx.x, cnt, reinterpret_cast<float *>(smem));
    if (!a.chunk_cnt) return;
    __syncthreads();
    for (int e = threadIdx.x; e < ep; e += blockDim.x)
        a.chunk_cnt[(size_t)blockIdx.x * ep + e] = e < a.E ? (uint16_t)cnt[e] : (uint16_t)0;
}

// Second launch: every CTA sums the count rows of all chunks and of those before
// its own, and places its chunk's pairs. All CTAs read the same rows at once, so
// their latency counts: with 512 threads a thread's loads (8 at 4096 tokens of
// 256 experts) are one batch, 2 us, with 256 threads two, 4 to 8 us. (Sums split
// over a cluster of 8 and joined through distributed shared memory: 4 us longer,
// two barriers and 16 remote loads a thread.)
__global__ void __launch_bounds__(kPermThreads) route_permute_kernel(const __grid_constant__ RouteArgs a, int rows, int ep) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ PermSmem sm;
    __shared__ __align__(16) int32_t sums[2][8 * kPermThreads];  // [all, before][row group][ep]
    uint32_t *bm = reinterpret_cast<uint32_t *>(smem);
    const int tid = threadIdx.x, E = a.E, words = (a.chunk + 31) / 32, c = blockIdx.x;
    for (int i = tid; i < E * words; i += kPermThreads) bm[i] = 0u;
    __syncthreads();
    pdl_wait();
    const int nv = ep / 8, per = kPermThreads / nv;      // row groups of nv threads, 8 experts each
    if (tid < per * nv) {
        int all[8], pre[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) all[i] = pre[i] = 0;
#pragma unroll 8
        for (int r = tid / nv; r < rows; r += per) {
            const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(a.chunk_cnt + (size_t)r * ep) + tid % nv);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int n = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
                all[i] += n;
                pre[i] += r < c ? n : 0;
            }
        }
        int4 *s0 = reinterpret_cast<int4 *>(sums[0] + 8 * tid), *s1 = reinterpret_cast<int4 *>(sums[1] + 8 * tid);
        s0[0] = make_int4(all[0], all[1], all[2], all[3]), s0[1] = make_int4(all[4], all[5], all[6], all[7]);
        s1[0] = make_int4(pre[0], pre[1], pre[2], pre[3]), s1[1] = make_int4(pre[4], pre[5], pre[6], pre[7]);
    }
    chunk_bitmaps(a, c, sm, bm);                         // (a barrier within)
    for (int e = tid; e < E; e += kPermThreads) {
        int all = 0, pre = 0;
        for (int g = 0; g < per; ++g) {
            all += sums[0][g * ep + e];
            pre += sums[1][g * ep + e];
        }
        sm.tot[e] = all;
        sm.base[e] = pre;
    }
    const int total = expert_offsets(a, sm);
    place_chunk(a, c, sm, bm);
    finish_route(a, c, rows, total, sm);
}

// Small batches: both steps in one launch, the chunks of one cluster, which
// read each other's counts through distributed shared memory.
template <int EPL>
__global__ void __launch_bounds__(kSelThreads) route_fused_kernel(const __grid_constant__ RouteArgs a, int nch) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int32_t cnt[kRouteMaxE];
    __shared__ PermSmem sm;
    const int tid = threadIdx.x, E = a.E, c = blockIdx.x;
    select_chunk<EPL>(a, c, cnt, reinterpret_cast<float *>(smem));
    const bool permute = a.counts || a.offsets || a.perm || a.pos || a.uniq;
    if (!permute) return;
    __syncthreads();
    uint32_t *bm = reinterpret_cast<uint32_t *>(smem);   // over the warps' scores
    if (nch > 1) cluster_arrive();                       // cnt is complete
    for (int i = tid; i < E; i += blockDim.x) bm[i] = 0u;
    __syncthreads();
    chunk_bitmaps(a, c, sm, bm);
    if (nch > 1) cluster_wait();
    for (int e = tid; e < E; e += blockDim.x) {
        int tot = sm.own[e], base = 0;
        if (nch > 1) {
            tot = 0;
            for (int r = 0; r < nch; ++r) {
                const int v = ld_cluster(&cnt[e], r);
                tot += v;
                base += r < c ? v : 0;
            }
        }
        sm.tot[e] = tot;
        sm.base[e] = base;
    }
    if (nch > 1) cluster_arrive();
    const int total = expert_offsets(a, sm);
    place_chunk(a, c, sm, bm);
    finish_route(a, c, nch, total, sm);
    if (nch > 1) cluster_wait();                         // no CTA leaves while another may read its counts
}

template <int EPL>
cudaError_t launch_epl(RouteArgs a, cudaStream_t st, int *launches) {
    const bool permute = a.counts || a.offsets || a.perm || a.pos || a.uniq;
    a.chunk = route_chunk_tokens(a.T);
    const int rows = (a.T + a.chunk - 1) / a.chunk;
    const size_t per_warp = (size_t)(2 * a.E + 192) * 4;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.stream = st;
    cfg.gridDim = dim3(rows);
    if (launches) ++*launches;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (rows <= kRouteFusedChunks) {
        static std::atomic<uint64_t> set{0};
        const cudaError_t e = set_smem_limit_once((const void *)route_fused_kernel<EPL>, kSelSmem, set);
        if (e != cudaSuccess) return e;
        const int warps = a.T < 8 ? 8 : a.T < 32 ? a.T : 32;  // 8 for the permutation of even one token
        cfg.blockDim = dim3(32 * warps);
        cfg.dynamicSmemBytes = warps * per_warp;              // holds the bitmaps too: 2 E words
        attr[0].val.clusterDim.x = rows;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, route_fused_kernel<EPL>, a, rows);
    }
    if (!permute) a.chunk_cnt = nullptr;
    const int ep = (a.E + 7) & ~7;
    static std::atomic<uint64_t> set_sel{0}, set_perm{0};
    cudaError_t e = set_smem_limit_once((const void *)route_select_kernel<EPL>, kSelSmem, set_sel);
    if (e != cudaSuccess) return e;
    // one token per warp while every chunk has an SM; then half as many warps, two CTAs on an SM
    const int warps = rows <= kRouteMaxChunks / 2 ? 32 : 16;
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = warps * per_warp;
    cfg.numAttrs = 0;
    e = cudaLaunchKernelEx(&cfg, route_select_kernel<EPL>, a, ep);
    if (e != cudaSuccess || !permute) return e;
    e = set_smem_limit_once((const void *)route_permute_kernel, kPermSmem, set_perm);
    if (e != cudaSuccess) return e;
    cfg.blockDim = dim3(kPermThreads);
    cfg.dynamicSmemBytes = (size_t)2 * a.E * ((a.chunk + 31) / 32) * 4;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (launches) ++*launches;
    return cudaLaunchKernelEx(&cfg, route_permute_kernel, a, rows, ep);
}

}  // namespace

cudaError_t launch_route_logits(RouteArgs a, cudaStream_t st, int *launches) {
    const int epl = a.E <= 32 ? 1 : a.E <= 64 ? 2 : a.E <= 128 ? 4 : a.E <= 256 ? 8 : 16;
    const int size = a.type == MOE_T_F32 ? 4 : 2;
    const int align = epl * size < 16 ? epl * size : 16;
    a.vec = a.nsplit == 1 && a.E % epl == 0 && (uintptr_t)a.logits % align == 0 && (a.stride * size) % align == 0;
    const int gs = a.E / a.groups;
    a.group_inv = ((1u << 22) + gs - 1) / gs;
    const int lanes = gs / epl;
    a.direct = gs % epl == 0 && (lanes & (lanes - 1)) == 0;
    a.lanes_per_group = a.direct ? lanes : 1;
    while (!a.direct && 2 * a.lanes_per_group * a.groups <= 32) a.lanes_per_group *= 2;
    a.vec_bias = a.E % epl == 0 && (uintptr_t)a.bias % 16 == 0;
    return epl == 1   ? launch_epl<1>(a, st, launches)
           : epl == 2 ? launch_epl<2>(a, st, launches)
           : epl == 4 ? launch_epl<4>(a, st, launches)
           : epl == 8 ? launch_epl<8>(a, st, launches)
                      : launch_epl<16>(a, st, launches);
}

}  // namespace moe
