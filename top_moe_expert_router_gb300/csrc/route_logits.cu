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
// on. A lane packs its slot into the low 4 bits of each 32-bit key and sorts
// its keys by minima and maxima alone (two instructions a comparator); a pick
// is one warp maximum of the lanes' heads without the slot, the lowest lane
// among equals, and a shift of that lane's list. The 4 bits count in the error
// bound; they are zeros anyway in the keys of 16-bit logits.
#include <math.h>

#include "ops.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kSelThreads = 1024;
constexpr int kSelSmem = 32 * (2 * kRouteMaxE + 2) * 4;               // 32 warps' scores
constexpr int kPermSmem = 2 * kRouteMaxE * (kRouteMaxT / kRouteMaxChunks / 32) * 4;  // both tables at the largest chunk

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
// load_lane, with NaN and -inf as -inf and +inf as the largest finite float.
template <int EPL>
__device__ __forceinline__ void load_clean(const RouteArgs &a, int64_t row, int e0, float l[EPL]) {
    load_lane<EPL>(a, row, e0, l);
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = l[i] > -INFINITY ? fminf(l[i], 3.402823466e38f) : -INFINITY;
}

// What a choice leaves in lane j < k: the j-th pick.
struct Pick {
    int id;        // -1: none left
    float l;       // its logit
};

// The logit of expert e of a row (lane by lane), cleaned as in the kernel.
__device__ __forceinline__ float one_logit(const RouteArgs &a, int64_t row, int e) {
    float l = load_logit(a.logits, row + e, a.type);
    for (int s = 1; s < a.nsplit; ++s) l += ((const float *)a.logits)[row + s * a.split_stride + e];
    return fminf(l, 3.402823466e38f);
}

// Sorts key[0 .. N) in descending order.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&key)[N]) {
    // odd-even merge sort (Batcher)
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint32_t x = key[i + j], y = key[i + j + k];
                        key[i + j] = max(x, y);
                        key[i + j + k] = min(x, y);
                    }
}

// The scores of a lane's experts in 32 bits (c), which of them may be chosen,
// and a bound on the error of a score. `scored`: false where the order of the
// logits serves.
//
// Errors. Sigmoid by the fast exponential and reciprocal: the exponent's
// relative error of (2 + 1.2 |l|) 2^-23 enters the score times p (1 - p), at
// most 0.64 * 2^-23; with the sum's and the reciprocal's roundings under
// 2.2 * 2^-23: 2^-21 is allowed. Softmax: likewise t exp(-t) of a term's
// argument, and about 25 roundings of the sum: 2^-18 of the largest score 1 / z
// is allowed. The bias adds a rounding of 2^-24 of the sum.
struct Scored {
    uint32_t on;
    float err;
};
template <int EPL>
__device__ __forceinline__ Scored score_lane(const RouteArgs &a, const float (&l)[EPL], float lmax, int e0, bool scored,
                                             float (&c)[EPL]) {
    Scored r{0u, 0.f};
#pragma unroll
    for (int i = 0; i < EPL; ++i) r.on |= l[i] > -INFINITY ? 1u << i : 0u;
    if (!scored) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = l[i];
        return r;
    }
    if (a.sigmoid) {
        r.err = 0x1p-21f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] = __fdividef(1.f, 1.f + __expf(-l[i]));
    } else {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            c[i] = ((r.on >> i) & 1u) ? __expf(l[i] - lmax) : 0.f;
            s += c[i];
        }
        s = warp_add(s);
        const float inv_z = s > 0.f ? 1.f / s : 1.f;
        r.err = 0x1p-18f * inv_z;
#pragma unroll
        for (int i = 0; i < EPL; ++i) c[i] *= inv_z;
    }
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if ((r.on >> i) & 1u) {
                const float b = __ldg(a.bias + e0 + i);
                if (b > -INFINITY) c[i] += fminf(b, 3.402823466e38f);
                else r.on &= ~(1u << i);                  // also NaN
            }
    }
    return r;
}

// The two best of every group: lpg lanes (a power of two, 32 / groups at most)
// walk each group and all of them end with its result (element e lies at
// e + e / 32: groups a multiple of 32 apart would share a bank).
template <int EPL, typename S>
__device__ __forceinline__ void group_best(const RouteArgs &a, const S (&c)[EPL], uint32_t on, int lane, S *buf, S &b1,
                                           S &b2) {
    const int e0 = lane * EPL, gs = a.E / a.groups, lpg = a.lanes_per_group, sub = lane & (lpg - 1), g = lane / lpg;
    constexpr int kPad = sizeof(S) == 4 ? 5 : 31;         // no padding for doubles: the room is E of them
    __syncwarp();
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (e0 + i < a.E) buf[e0 + i + ((e0 + i) >> kPad)] = ((on >> i) & 1u) ? c[i] : (S)-INFINITY;
    __syncwarp();
    b1 = b2 = (S)-INFINITY;
    if (g < a.groups)
        for (int i = sub; i < gs; i += lpg) {
            const int e = g * gs + i;
            const S v = buf[e + (e >> kPad)];
            const S low = b1 < v ? b1 : v;
            b2 = b2 > low ? b2 : low;
            b1 = b1 > v ? b1 : v;
        }
    for (int o = lpg >> 1; o > 0; o >>= 1) {
        const S v1 = __shfl_xor_sync(kFull, b1, o), v2 = __shfl_xor_sync(kFull, b2, o);
        const S low = b1 < v1 ? b1 : v1;
        b2 = b2 > v2 ? b2 : v2;
        b2 = b2 > low ? b2 : low;
        b1 = b1 > v1 ? b1 : v1;
    }
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

template <int EPL>
__device__ __forceinline__ uint32_t in_kept_groups(const RouteArgs &a, uint32_t on, uint32_t mask, int e0) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const uint32_t gi = ((uint32_t)(e0 + i) * a.group_inv) >> 22;  // (e0 + i) / group size
        if (e0 + i >= a.E || !((mask >> (gi * a.lanes_per_group)) & 1u)) on &= ~(1u << i);
    }
    return on;
}

// The n largest packed keys of the warp in order: lane j gets the j-th (0: none) and its expert.
template <int EPL>
__device__ __forceinline__ uint32_t pick_packed(const float (&c)[EPL], uint32_t on, int n, int lane, int *id) {
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = ((on >> i) & 1u) ? (order_key(c[i]) & ~15u) | (15u - i) : 0u;
    sort_desc<EPL>(key);
    uint32_t mine = 0u;
    *id = -1;
    for (int j = 0; j < n; ++j) {
        const uint32_t m = __reduce_max_sync(kFull, key[0] >> 4);
        if (m == 0u) break;
        const int win = __ffs(__ballot_sync(kFull, (key[0] >> 4) == m)) - 1;
        const uint32_t h = __shfl_sync(kFull, key[0], win);
        if (lane == j) {
            mine = h;
            *id = win * EPL + 15 - (int)(h & 15u);
        }
        if (lane == win) {
#pragma unroll
            for (int i = 0; i + 1 < EPL; ++i) key[i] = key[i + 1];
            key[EPL - 1] = 0u;
        }
    }
    return mine;
}

// A packed key stands for a score within 2^-19 of it above.
constexpr float kPackSlack = 0x1p-19f;

// The choice in 32 bits; *close (warp-uniform) says that some comparison was
// within the error of what was compared. buf: room for E + E / 32 floats.
template <int EPL>
__device__ __forceinline__ Pick choose_fast(const RouteArgs &a, const float (&l)[EPL], float lmax, int64_t row, int lane,
                                            float *buf, bool *close) {
    const int e0 = lane * EPL;
    const bool staged = a.keep < a.groups, by_logit = a.bias == nullptr;
    float c[EPL];
    const Scored sc = score_lane<EPL>(a, l, lmax, e0, !by_logit || (staged && a.top2), c);
    uint32_t on = sc.on;
    bool near = false;
    if (staged) {
        float b1, b2;
        group_best<EPL, float>(a, c, on, lane, buf, b1, b2);
        const bool any = b1 > -INFINITY, is_group = lane / a.lanes_per_group < a.groups;
        const float score = a.top2 && b2 > -INFINITY ? b1 + b2 : b1;
        const bool kept = group_kept(a, score, any, lane);
        if (!by_logit || a.top2) {
            // the border: the worst kept group against the best one left out;
            // two scores make a group's, each rounded once more with its bias
            float lo = kept ? score : INFINITY;
            float hi = is_group && !kept ? score : -INFINITY;
            float mag = any ? fabsf(b1) + (b2 > -INFINITY ? fabsf(b2) : 0.f) : 0.f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
                hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
                mag = fmaxf(mag, __shfl_xor_sync(kFull, mag, o));
            }
            near = hi > -INFINITY && !(lo - hi > 4.f * sc.err + 0x1p-22f * mag);
        }
        on = in_kept_groups<EPL>(a, on, __ballot_sync(kFull, kept), e0);
        if (by_logit) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = l[i];
        }
    }
    Pick r{-1, -INFINITY};
    const uint32_t mine = pick_packed<EPL>(c, on, a.k + 1, lane, &r.id);  // one more: the border
    if (r.id >= 0) r.l = one_logit(a, row, r.id);
    const uint32_t next = __shfl_down_sync(kFull, mine, 1);
    if (by_logit) {
        // equal but for the slot: ties in 16-bit types, anything in fp32
        near |= lane < a.k && next && a.type == MOE_T_F32 && (next >> 4) == (mine >> 4);
    } else {
        // the score again, without the packed slot; what was not picked lies
        // below the border's key and its slack
        float v = 0.f;
        if (r.id >= 0) {
            v = a.sigmoid ? __fdividef(1.f, 1.f + __expf(-r.l)) : __expf(r.l - lmax) * (sc.err * 0x1p18f);
            v += fminf(__ldg(a.bias + r.id), 3.402823466e38f);
        }
        const float nv = __shfl_down_sync(kFull, v, 1);
        const float x = lane < a.k - 1 ? nv : key_value(next & ~15u);
        const float mag = fmaxf(fabsf(v), fabsf(x));
        near |= lane < a.k && next && !(v - x > 2.f * sc.err + mag * (lane < a.k - 1 ? 0x1p-22f : kPackSlack + 0x1p-22f));
    }
    *close = __any_sync(kFull, near);
    if (lane >= a.k) r.id = -1;
    return r;
}

// A score in 64 bits.
__device__ __forceinline__ double score64(const RouteArgs &a, float l, float lmax, double z, int e) {
    double p = l;
    if (a.sigmoid) p = 1.0 / (1.0 + exp(-(double)l));
    else p = exp((double)l - (double)lmax) / z;
    return a.bias ? p + (double)fminf(__ldg(a.bias + e), 3.402823466e38f) : p;
}

// The choice in 64 bits, of those scores that can matter: in 32 bits first, a
// score that lies further below a group's second best, or below the k-th pick,
// than the errors allow is left out. buf: room for E doubles.
template <int EPL>
__device__ __forceinline__ Pick choose_exact(const RouteArgs &a, const float (&l)[EPL], float lmax, int lane, float *buf) {
    const int e0 = lane * EPL;
    const bool staged = a.keep < a.groups;
    const bool by_logit = a.bias == nullptr;              // the picks' order needs no score
    const bool scored = !by_logit || (staged && a.top2);
    float c[EPL];
    const Scored sc = score_lane<EPL>(a, l, lmax, e0, scored, c);
    uint32_t on = sc.on;
    double z = 1.0;
    if (scored && !a.sigmoid) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s += l[i] > -INFINITY ? exp((double)l[i] - (double)lmax) : 0.0;
        s = warp_add(s);
        if (s > 0.0) z = s;
    }
    double d[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = l[i];
    uint32_t have = 0u;
    auto compute = [&](uint32_t need) {
        need &= ~have;
        have |= need;
        while (__any_sync(kFull, need != 0u)) {
            const int at = need ? __ffs(need) - 1 : 0;
            float la = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == at) la = l[i];
            const double v = score64(a, la, lmax, z, need ? e0 + at : 0);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (need && i == at) d[i] = v;
            need &= need - 1u;
        }
    };
    if (staged) {
        float f1, f2;
        group_best<EPL, float>(a, c, on, lane, buf, f1, f2);
        uint32_t need = on;
        if (scored) {
            const float thr = a.top2 ? f2 : f1;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t gi = ((uint32_t)min(e0 + i, a.E - 1) * a.group_inv) >> 22;
                const float tg = __shfl_sync(kFull, thr, (gi * a.lanes_per_group) & 31);
                if (tg - c[i] > 2.f * sc.err + 0x1p-21f * fmaxf(fabsf(tg), fabsf(c[i]))) need &= ~(1u << i);
            }
            compute(need);
        }
        double b1, b2;
        group_best<EPL, double>(a, d, need, lane, reinterpret_cast<double *>(buf), b1, b2);
        const double score = a.top2 && b2 > -INFINITY ? b1 + b2 : b1;
        const bool kept = group_kept(a, score, b1 > -INFINITY, lane);
        on = in_kept_groups<EPL>(a, on, __ballot_sync(kFull, kept), e0);
    }
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] = c[i] = l[i];
    } else {
        int id;
        const uint32_t mine = pick_packed<EPL>(c, on, a.k, lane, &id);
        const uint32_t last = __shfl_sync(kFull, mine, a.k - 1);
        if (last) {                                       // fewer than k are left: all of them
            const float x = key_value(last & ~15u);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (x - c[i] > 2.f * sc.err + (kPackSlack + 0x1p-21f) * fmaxf(fabsf(x), fabsf(c[i]))) on &= ~(1u << i);
        }
        compute(on);
    }
    uint64_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = ((on >> i) & 1u) ? key_of(d[i]) : 0ull;
    Pick r{-1, -INFINITY};
    for (int j = 0; j < a.k; ++j) {
        uint64_t bk = key[0];
        int bi = 0;
        float lw = l[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i)
            if (key[i] > bk) {
                bk = key[i];
                bi = i;
                lw = l[i];
            }
        const uint64_t m = warp_max(bk);
        if (m == 0) break;
        const int win = __ffs(__ballot_sync(kFull, bk == m)) - 1;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (i == bi && lane == win) key[i] = 0;
        const int id = __shfl_sync(kFull, e0 + bi, win);
        lw = __shfl_sync(kFull, lw, win);
        if (lane == j) r = Pick{id, lw};
    }
    return r;
}

// Out of line: few tokens take it, and it loads its logits again so that the
// caller's stay in registers.
template <int EPL>
__device__ __noinline__ Pick choose_again(const RouteArgs &a, int64_t row, float lmax, int lane, float *lbuf) {
    float l[EPL];
    load_clean<EPL>(a, row, lane * EPL, l);
    return choose_exact<EPL>(a, l, lmax, lane, lbuf);
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
        for (int i = 0; i < EPL; ++i) s += l[i] > -INFINITY ? __expf(l[i] - lmax) : 0.f;  // within 2^-20 of the sum
        s = warp_add(s);
        if (on) w = expf(r.l - lmax) / s;
    }
    return on ? w * a.scale : 0.f;
}

// ids and weights of a chunk's tokens, one warp per token, and the chunk's
// count of every expert in cnt. lbuf: 2 E + 2 floats per warp.
template <int EPL>
__device__ __forceinline__ void select_chunk(const RouteArgs &a, int c, int32_t *cnt, float *lbuf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
    __syncthreads();
    const int t0 = c * a.chunk, t1 = min(t0 + a.chunk, a.T);
    lbuf += warp * (2 * a.E + 2);
    for (int t = t0 + warp; t < t1; t += nw) {
        const int64_t row = (int64_t)t * a.stride;
        float l[EPL];
        load_clean<EPL>(a, row, lane * EPL, l);
        float lmax = l[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) lmax = fmaxf(lmax, l[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(kFull, lmax, o));
        bool close;
        Pick r = choose_fast<EPL>(a, l, lmax, row, lane, lbuf, &close);
        if (close) r = choose_again<EPL>(a, row, lmax, lane, lbuf);
        const float w = pick_weight<EPL>(a, l, lmax, r, lane);
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = r.id;
            a.w[(size_t)t * a.k + lane] = w;
            if (r.id >= 0) atomicAdd(&cnt[r.id], 1);
        }
    }
}

// What a permutation keeps in shared memory besides its bitmaps.
struct PermSmem {
    int32_t tot[kRouteMaxE];       // all pairs of every expert
    int32_t base[kRouteMaxE];      // those in earlier chunks
    int32_t own[kRouteMaxE];       // those of this chunk
    int32_t off[kRouteMaxE + 1];
    int32_t part[2][kRouteMaxE];   // this CTA's share of the counts' sums: all, earlier clusters'
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
    const int tid = threadIdx.x, nth = blockDim.x, E = a.E, words = a.chunk / 32;
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

// The rows of a chunk's pairs, from sm.tot and sm.base. Expert e's rows are
// offsets[e] .., its tokens ascending: row = offsets[e] + (pairs in earlier
// chunks) + (tokens of e earlier in the chunk), the last from the bitmaps, so
// the result does not depend on the order of threads.
__device__ __forceinline__ void place_chunk(const RouteArgs &a, int c, int nch, PermSmem &sm, const uint32_t *bm) {
    const int tid = threadIdx.x, nth = blockDim.x, E = a.E, words = a.chunk / 32;
    const uint32_t *before = bm + E * words;
    const int t0 = c * a.chunk, nt = max(0, min(a.chunk, a.T - t0));
    const int32_t *ids = a.ids + (size_t)t0 * a.k;
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
    if (a.perm)
        for (int64_t i = run + (int64_t)c * nth + tid; i < (int64_t)a.T * a.k; i += (int64_t)nch * nth)
            a.perm[i] = a.perm_fill;
    if (c != 0) return;
    for (int e = tid; e <= E; e += nth) {
        if (a.counts && e < E) a.counts[e] = sm.tot[e];
        if (a.offsets) a.offsets[e] = sm.off[e];
    }
    if (!a.uniq) return;
    int nu = 0, ntile = 0;
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

// Large batches, first launch: the choice, and the counts of every 32 tokens
// in rows of `ep` (E rounded up to 8).
template <int EPL>
__global__ void __launch_bounds__(kSelThreads) route_select_kernel(RouteArgs a, int ep) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ int32_t cnt[kRouteMaxE];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    select_chunk<EPL>(a, blockIdx.x, cnt, reinterpret_cast<float *>(smem));
    if (!a.chunk_cnt) return;
    __syncthreads();
    for (int e = threadIdx.x; e < ep; e += blockDim.x)
        a.chunk_cnt[(size_t)blockIdx.x * ep + e] = e < a.E ? (uint16_t)cnt[e] : (uint16_t)0;
}

// Second launch, clusters of 8 CTAs, a chunk of tokens each: every CTA sums an
// eighth of the count rows (all of them, and those before its cluster), the
// CTAs add up their sums and their own chunks' counts through distributed
// shared memory, and each places its pairs.
__global__ void __launch_bounds__(kSelThreads) route_permute_kernel(RouteArgs a, int rows, int ep) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ PermSmem sm;
    uint32_t *bm = reinterpret_cast<uint32_t *>(smem);
    const int tid = threadIdx.x, E = a.E, c = blockIdx.x, rank = c & 7, words = a.chunk / 32;
    for (int i = tid; i < E * words; i += kSelThreads) bm[i] = 0u;
    for (int e = tid; e < E; e += kSelThreads) sm.part[0][e] = sm.part[1][e] = 0;
    __syncthreads();
    pdl_wait();
    {
        const int nv = ep / 8, v = tid % nv, per = kSelThreads / nv;
        const int first = (int)((int64_t)rank * rows / 8), last = (int)((int64_t)(rank + 1) * rows / 8);
        const int before = (c - rank) * words;           // rows ahead of this cluster's chunks
        int all[8], pre[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) all[i] = pre[i] = 0;
        if (tid < per * nv) {
#pragma unroll 4
            for (int r = first + tid / nv; r < last; r += per) {
                const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(a.chunk_cnt + (size_t)r * ep) + v);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int n = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
                    all[i] += n;
                    pre[i] += r < before ? n : 0;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (all[i]) {
                    atomicAdd(&sm.part[0][8 * v + i], all[i]);
                    if (pre[i]) atomicAdd(&sm.part[1][8 * v + i], pre[i]);
                }
        }
    }
    chunk_bitmaps(a, c, sm, bm);
    cluster_arrive();
    cluster_wait();
    for (int e = tid; e < E; e += kSelThreads) {
        int tot = 0, base = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            tot += ld_cluster(&sm.part[0][e], q);
            base += ld_cluster(&sm.part[1][e], q);
            if (q < rank) base += ld_cluster(&sm.own[e], q);
        }
        sm.tot[e] = tot;
        sm.base[e] = base;
    }
    cluster_arrive();
    place_chunk(a, c, gridDim.x, sm, bm);
    cluster_wait();                                      // no CTA leaves while another may read its sums
}

// Small batches: both steps in one launch, the chunks of one cluster, which
// read each other's counts through distributed shared memory.
template <int EPL>
__global__ void __launch_bounds__(kSelThreads) route_fused_kernel(RouteArgs a, int nch) {
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
    place_chunk(a, c, nch, sm, bm);
    if (nch > 1) cluster_wait();                         // no CTA leaves while another may read its counts
}

template <int EPL>
cudaError_t launch_epl(RouteArgs a, cudaStream_t st, int *launches) {
    const bool permute = a.counts || a.offsets || a.perm || a.pos || a.uniq;
    const int rows = (a.T + 31) / 32;
    const size_t per_warp = (size_t)(2 * a.E + 2) * 4;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    cfg.stream = st;
    a.chunk = 32;
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
    // one token per warp while the SMs hold all chunks; then half as many warps, two CTAs on an SM
    const int warps = rows <= 152 ? 32 : 16;
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = warps * per_warp;
    cfg.numAttrs = 0;
    e = cudaLaunchKernelEx(&cfg, route_select_kernel<EPL>, a, ep);
    if (e != cudaSuccess || !permute) return e;
    e = set_smem_limit_once((const void *)route_permute_kernel, kPermSmem, set_perm);
    if (e != cudaSuccess) return e;
    a.chunk = route_chunk_tokens(a.T);
    const int nch = (a.T + a.chunk - 1) / a.chunk;
    cfg.gridDim = dim3((nch + 7) / 8 * 8);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)2 * a.E * (a.chunk / 32) * 4;
    attr[0].val.clusterDim.x = 8;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
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
    a.lanes_per_group = 1;
    while (2 * a.lanes_per_group * a.groups <= 32) a.lanes_per_group *= 2;
    return epl == 1   ? launch_epl<1>(a, st, launches)
           : epl == 2 ? launch_epl<2>(a, st, launches)
           : epl == 4 ? launch_epl<4>(a, st, launches)
           : epl == 8 ? launch_epl<8>(a, st, launches)
                      : launch_epl<16>(a, st, launches);
}

}  // namespace moe
