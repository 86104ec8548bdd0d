"""Timed cases of the operators around the expert layer: routing from logits,
residual + RMSNorm with an 8-bit output, and products with 4-bit weights.

``listed()`` and ``draw()`` give cases, ``prepare()`` a case's inputs on the
GPU, ``run()`` one pass: the plain form in elementary torch operations, or,
with ``own`` set, the framework's kernels. ``exact()`` is the definition in 64
bits, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _route(T, E, k, dtype, score, bias, groups, keep, rule, renorm, scale, masked):
    return {"op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "score": score, "bias": bias, "groups": groups,
            "keep": keep, "rule": rule, "renorm": renorm, "scale": scale, "masked": masked}


def _norm(T, d, dtype, res, out, group):
    return {"op": "norm", "T": T, "d": d, "dtype": dtype, "res": res, "out": out, "group": group}


def _w4(M, N, K, fmt, group, zeros, x, xgroup, out, bias):
    return {"op": "w4", "M": M, "N": N, "K": K, "fmt": fmt, "group": group, "zeros": zeros, "x": x, "xgroup": xgroup,
            "out": out, "bias": bias}


def listed():
    cases = [
        # one decode token of a 256-expert layer: sigmoid scores, a balance bias, 4 of 8 groups
        ("route_token", _route(1, 256, 8, "f32", "sigmoid", True, 8, 4, "top2", True, 2.5, False)),
        # a batch of decode tokens, softmax over 128 experts, bf16 logits
        ("route_batch", _route(48, 128, 8, "bf16", "softmax", False, 1, 1, "max", True, 1.0, False)),
        # a prompt of the prefill workload's length, as the first case otherwise
        ("route_prompt", _route(4096, 256, 8, "f32", "sigmoid", True, 8, 4, "top2", True, 2.5, False)),
        # a long packed batch with an odd length: groups by their best expert, weights not renormalised,
        # some experts switched off
        ("route_long", _route(30011, 160, 6, "bf16", "softmax", False, 8, 3, "max", False, 16.0, True)),
        # one decode token at the layer's hidden size, blocks of 128 in 8 bits
        ("norm_token", _norm(1, 4096, "bf16", True, "e4m3", 128)),
        # a ragged batch at a size that no vector width divides evenly among threads, one scale a row
        ("norm_ragged", _norm(777, 5000, "f16", True, "e4m3", 0)),
        # the prefill workload's prompt
        ("norm_prompt", _norm(4096, 4096, "bf16", True, "e4m3", 128)),
        # a long batch at the largest hidden size of the layer, 16-bit output
        ("norm_long", _norm(16384, 8192, "bf16", True, "bf16", 0)),
        # one decode token through a square projection at the layer's hidden size
        ("w4_token", _w4(1, 4096, 4096, "nvfp4", 16, False, "bf16", 0, "bf16", False)),
        # a few decode tokens through a wide projection with integer codes and zero points
        ("w4_batch", _w4(8, 12288, 4096, "int4", 128, True, "f16", 0, "f16", True)),
        # sixteen tokens as the norm's 8-bit output hands them over
        ("w4_fp8", _w4(16, 8192, 4096, "nvfp4", 16, False, "e4m3", 128, "bf16", False)),
        # an output head over a large vocabulary, 32-bit logits
        ("w4_head", _w4(4, 131072, 4096, "nvfp4", 16, False, "bf16", 0, "f32", False)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "w4"])
    if op == "route":
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 4, 8])
        size = _log(rng, 4, 512 // groups) if groups > 1 else _log(rng, 8, 512)
        keep = rng.randint(1, groups)
        k = rng.randint(2, min(16, size * keep))
        bias = rng.random() < 0.5
        return _route(_log(rng, 1, 30000), groups * size, k, rng.choice(["bf16", "f16", "f32"]), score, bias, groups, keep,
                      rng.choice(["max", "top2"]), rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.3)
    if op == "norm":
        d = _log(rng, 64, 12000)
        if rng.random() < 0.6:
            d = (d + 127) // 128 * 128
        out = rng.choice(["same", "e4m3", "e4m3"])
        group = rng.choice([0, 128, 64]) if out == "e4m3" else 0
        if group and d % group:
            group = 0
        dtype = rng.choice(["bf16", "f16", "f32"])
        T = min(_log(rng, 1, 16384), (1 << 27) // d // (2 if dtype == "f32" else 1))
        return _norm(T, d, dtype, rng.random() < 0.8, dtype if out == "same" else out, group)
    fmt = rng.choice(["nvfp4", "int4"])
    group = 16 if fmt == "nvfp4" else rng.choice([32, 64, 128])
    K = max(1, _log(rng, 256, 12000) // 128) * 128 if rng.random() < 0.6 else max(group, 32) * (_log(rng, 256, 12000) // max(group, 32))
    x = rng.choice(["bf16", "f16", "e4m3"])
    xgroup = rng.choice([0, 128]) if x == "e4m3" and K % 128 == 0 else 0
    M = _log(rng, 1, 64)
    N = min(_log(rng, 64, 131072), (1 << 31) // K // max(4, M))
    return _w4(M, N, K, fmt, group, fmt == "int4" and rng.random() < 0.7, x, xgroup,
               rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.3)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _prepare_route(c, g):
    T, E, k = c["T"], c["E"], c["k"]
    logits = 1.5 * _randn(g, T, E) + 0.7 * _randn(g, E)
    if c["masked"]:
        logits.masked_fill_(torch.rand(T, E, generator=g, device="cuda") < 0.05, -math.inf)
        logits[1:][-1:] = -math.inf                 # a padding row behind the tokens
    i32 = {"dtype": torch.int32, "device": "cuda"}
    return {"logits": logits.to(_T[c["dtype"]]), "bias": 0.1 * _randn(g, E) if c["bias"] else None,
            "out": {"ids": torch.empty((T, k), **i32), "w": torch.empty((T, k), device="cuda"),
                    "counts": torch.empty(E, **i32), "offsets": torch.empty(E + 1, **i32),
                    "perm": torch.empty(T * k, **i32), "pos": torch.empty((T, k), **i32)}}


def _prepare_norm(c, g):
    T, d, t = c["T"], c["d"], _T[c["dtype"]]
    hot = 1 + 8 * (torch.rand(d, generator=g, device="cuda") < 0.01).float()   # a few channels stand out
    x = (_randn(g, T, d) * hot).to(t)
    group = c["group"] or d
    return {"x": x, "res": (_randn(g, T, d) * hot * 2).to(t) if c["res"] else None,
            "gain": (1 + 0.2 * _randn(g, d)).to(t), "sum": torch.empty_like(x) if c["res"] else None,
            "out": torch.empty((T, d), dtype=_T[c["out"]], device="cuda"),
            "scales": torch.empty((T, d // group), device="cuda") if c["out"] == "e4m3" else None}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quant_nvfp4(W):
    """Blocks of 16: an E4M3 scale each, one fp32 scale for all; codes by the nearest value."""
    N, K = W.shape
    g = W.abs().max() / (6 * 448)
    b = W.view(N, K // 16, 16)
    s = (b.abs().amax(2) / 6 / g).to(torch.float8_e4m3fn)
    r = (b / (s.float() * g).clamp_min(1e-30)[:, :, None]).view(N, K)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(r.abs(), mids, out_int32=True).to(torch.uint8) | ((r < 0).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.view(torch.uint8), g.reshape(1)


def _quant_int4(W, group, zeros, t):
    N, K = W.shape
    b = W.view(N, K // group, group)
    if zeros:
        lo, hi = b.amin(2).clamp_max(0), b.amax(2).clamp_min(0)
        s = ((hi - lo) / 15).to(t)
        z = (-lo / s.float()).round().clamp(0, 15)
    else:
        s = (b.abs().amax(2) / 7).to(t)
        z = torch.full_like(s, 8, dtype=torch.float32)
    code = (b / s.float()[:, :, None] + z[:, :, None]).round().clamp(0, 15).to(torch.uint8).view(N, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), s, z.to(torch.uint8) if zeros else None


def _prepare_w4(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    W = 0.02 * _randn(g, N, K)
    if c["fmt"] == "nvfp4":
        q, s, gs = _quant_nvfp4(W)
        z = None
    else:
        q, s, z = _quant_int4(W, c["group"], c["zeros"], _T["f16" if c["x"] == "f16" else "bf16"])
        gs = None
    del W
    x = _randn(g, M, K)
    xs = None
    if c["x"] == "e4m3":
        n = c["xgroup"] or K
        b = x.view(M, K // n, n)
        xs = b.abs().amax(2) / 448
        x = (b / xs[:, :, None]).view(M, K)
    return {"x": x.to(_T[c["x"]]), "x_scales": xs, "q": q, "s": s, "g": gs, "z": z,
            "bias": 0.1 * _randn(g, N) if c["bias"] else None,
            "out": torch.empty((M, N), dtype=_T[c["out"]], device="cuda")}


def prepare(case, seed):
    g = _gen(seed)
    made = {"route": _prepare_route, "norm": _prepare_norm, "w4": _prepare_w4}[case["op"]](case, g)
    return dict(made, case=case)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_route(c, st):
    T, E, k = c["T"], c["E"], c["k"]
    l = st["logits"].double()                                   # 64 bits: scores next to the border
    live = ~(torch.isnan(l) | (l == -math.inf))
    l = l.clamp(max=torch.finfo(torch.float32).max)
    top = torch.where(live, l, -math.inf).amax(1, keepdim=True)
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        e = torch.where(live, torch.exp(l - torch.where(live.any(1, keepdim=True), top, 0.0)), 0.0)
        p = e / e.sum(1, keepdim=True)
    biased = p + st["bias"].double() if st["bias"] is not None else p
    if c["groups"] > 1:
        G, gs = c["groups"], E // c["groups"]
        by = biased if c["rule"] == "top2" or st["bias"] is not None else l
        grouped = torch.where(live, by, -math.inf).view(T, G, gs)
        best = grouped.sort(dim=2, descending=True).values
        score = best[:, :, 0]
        if c["rule"] == "top2" and gs > 1:
            score = score + torch.where(best[:, :, 1] > -math.inf, best[:, :, 1], 0.0)
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        live_k = live & kept[:, :, None].expand(T, G, gs).reshape(T, E)
    else:
        live_k = live
    choice = torch.where(live_k, l if st["bias"] is None else biased, -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    on = live_k.gather(1, ids)
    w = torch.where(on, p.gather(1, ids), 0.0)
    if c["renorm"]:
        if c["score"] == "sigmoid":
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        else:
            lk = torch.where(on, l.gather(1, ids), -math.inf)
            first = lk.amax(1, keepdim=True)
            e = torch.where(on, torch.exp(lk - torch.where(first > -math.inf, first, 0.0)), 0.0)
            w = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    w = (w * c["scale"]).float()
    key = torch.where(on, ids, E).view(-1)
    order = key.sort(stable=True)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    perm = torch.where(order.values < E, order.indices // k, -1)
    pos = torch.empty_like(key).scatter_(0, order.indices, torch.arange(T * k, device=key.device))
    pos = torch.where(key < E, pos, -1).view(T, k)
    i = torch.int32
    return {"ids": torch.where(on, ids, -1).to(i), "w": w, "counts": counts.to(i), "offsets": offsets.to(i),
            "perm": perm.to(i), "pos": pos.to(i)}


def _plain_norm(c, st):
    x = st["x"]
    s = x if st["res"] is None else (x.float() + st["res"].float()).to(x.dtype)
    v = s.float()
    y = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6) * st["gain"].float()
    out = {"sum": s} if st["res"] is not None else {}
    if c["out"] != "e4m3":
        return dict(out, y=y.to(x.dtype))
    T, d = y.shape
    b = y.view(T, -1, c["group"] or d)
    scale = b.abs().amax(2) / 448
    scale = torch.where(scale > 0, scale, 1.0)
    return dict(out, y=(b / scale[:, :, None]).view(T, d).to(torch.float8_e4m3fn), scales=scale)


def _plain_w4(c, st):
    M, N, K = c["M"], c["N"], c["K"]
    q = st["q"]
    codes = torch.stack((q & 15, q >> 4), 2).view(N, K)
    if c["fmt"] == "nvfp4":
        table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=q.device)
        W = table[codes.int()].view(N, K // 16, 16) * st["s"].view(torch.float8_e4m3fn).float()[:, :, None] * st["g"]
    else:
        z = st["z"].float() if st["z"] is not None else torch.full_like(st["s"], 8.0, dtype=torch.float32)
        W = (codes.float().view(N, -1, c["group"]) - z[:, :, None]) * st["s"].float()[:, :, None]
    x = st["x"].float()
    if st["x_scales"] is not None:
        x = (x.view(M, -1, c["xgroup"] or K) * st["x_scales"][:, :, None]).view(M, K)
    y = x @ W.view(N, K).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(_T[c["out"]])


def _own_route(moe, c, st):
    return moe.route_logits(st["logits"], c["k"], score=c["score"], bias=st["bias"], n_groups=c["groups"],
                            topk_groups=c["keep"], group_rule=c["rule"], renormalise=c["renorm"], scale=c["scale"],
                            out=st["out"])


def _own_norm(moe, c, st):
    y, s, scales = moe.add_rmsnorm(st["x"], st["res"], st["gain"], eps=1e-6, group=c["group"], sum_out=st["sum"],
                                   out=st["out"], scales=st["scales"])
    got = {"sum": s} if s is not None else {}
    return dict(got, y=y) if scales is None else dict(got, y=y, scales=scales)


def _own_w4(moe, c, st):
    if c["fmt"] == "nvfp4":
        return moe.linear_nvfp4(st["x"], st["q"], st["s"], st["g"], x_scales=st["x_scales"], bias=st["bias"],
                                out=st["out"])
    return moe.linear_int4(st["x"], st["q"], st["s"], st["z"], x_scales=st["x_scales"], bias=st["bias"], out=st["out"])


def run(state):
    c = state["case"]
    if own:
        import top_moe_expert_router_gb300 as moe
        return {"route": _own_route, "norm": _own_norm, "w4": _own_w4}[c["op"]](moe, c, state)
    return {"route": _plain_route, "norm": _plain_norm, "w4": _plain_w4}[c["op"]](c, state)


# ---------------------------------------------------------------------------
# the work a pass cannot do without
# ---------------------------------------------------------------------------
def work(c):
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        # logits (and bias) in; ids, w, perm and pos out, the counts and offsets
        return {"bytes": T * E * _BYTES[c["dtype"]] + (4 * E if c["bias"] else 0) + T * k * 16 + 4 * (2 * E + 1),
                "flops": 4 * T * E}
    if c["op"] == "norm":
        n, b = c["T"] * c["d"], _BYTES[c["dtype"]]
        scales = 4 * c["T"] * (c["d"] // (c["group"] or c["d"])) if c["out"] == "e4m3" else 0
        return {"bytes": n * b * (3 if c["res"] else 1) + c["d"] * b + n * _BYTES[c["out"]] + scales, "flops": 6 * n}
    M, N, K = c["M"], c["N"], c["K"]
    if c["fmt"] == "nvfp4":
        weights = N * K // 2 + N * K // 16
    else:
        weights = N * K // 2 + N * (K // c["group"]) * (3 if c["zeros"] else 2)
    xs = 4 * M * (K // (c["xgroup"] or K)) if c["x"] == "e4m3" else 0
    return {"bytes": weights + M * K * _BYTES[c["x"]] + xs + M * N * _BYTES[c["out"]] + (4 * N if c["bias"] else 0),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(c, st):
    """Token by token in numpy: sorted by (-choice, index)."""
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    L = st["logits"].float().cpu().numpy().astype(np.float64)
    bias = np.zeros(E) if st["bias"] is None else st["bias"].cpu().numpy().astype(np.float64)
    index = np.arange(E)
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = L[t]
        on = np.isfinite(l) | (l == np.inf)
        l = np.minimum(l, np.finfo(np.float32).max)
        if not on.any():
            continue
        with np.errstate(over="ignore"):
            if c["score"] == "sigmoid":
                p = np.where(on, 1 / (1 + np.exp(-l)), 0.0)
            else:
                p = np.where(on, np.exp(l - l[on].max()), 0.0)
                p = p / math.fsum(p)
        plain_order = st["bias"] is None
        choice = p + bias
        if G > 1:
            n = E // G
            totals = np.full(G, -np.inf)
            for j in range(G):
                vals = (l if plain_order and c["rule"] == "max" else choice)[j * n:(j + 1) * n][on[j * n:(j + 1) * n]]
                if vals.size:
                    vals = np.sort(vals)[::-1]
                    totals[j] = vals[0] if c["rule"] == "max" else vals[:2].sum()
            keep = sorted(range(G), key=lambda j: (-totals[j], j))[:c["keep"]]
            on = on & np.isin(index // n, keep)
        by = l if plain_order else choice
        order = index[on][np.lexsort((index[on], -by[on]))][:k]
        ids[t, :order.size] = order
        if order.size:
            if not c["renorm"]:
                got = p[order]
            elif c["score"] == "softmax":
                got = np.exp(l[order] - l[order].max())
                got = got / math.fsum(got)
            else:
                got = p[order] / math.fsum(p[order])
            w[t, :order.size] = got * c["scale"]
    counts = np.bincount(ids[ids >= 0], minlength=E).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    perm, pos = np.full(T * k, -1, np.int32), np.full((T, k), -1, np.int32)
    tt, jj = np.nonzero(ids >= 0)
    e = ids[tt, jj]
    order = np.lexsort((tt, e))
    perm[:order.size] = tt[order]
    pos[tt[order], jj[order]] = np.arange(order.size)
    return {"ids": ids, "w": w, "counts": counts, "offsets": offsets, "perm": perm, "pos": pos}


def _exact_norm(c, st):
    x = st["x"].double()
    out = {}
    if st["res"] is not None:
        x = x + st["res"].double()
        out["sum"] = x
        x = x.to(st["x"].dtype).double()           # the norm is of the stored sum
    y = x * (torch.einsum("td,td->t", x, x) / c["d"] + 1e-6).pow(-0.5)[:, None] * st["gain"].double()
    if c["out"] != "e4m3":
        return dict(out, y=y)
    n = c["group"] or c["d"]
    scale = torch.stack([b.abs().max(1).values for b in y.split(n, 1)], 1) / 448
    scale = scale + (scale == 0).double()
    return dict(out, y=y / scale.repeat_interleave(n, 1), scales=scale)


def _exact_w4(c, st):
    M, N, K = c["M"], c["N"], c["K"]
    x = st["x"].double()
    if st["x_scales"] is not None:
        x = x * st["x_scales"].double().repeat_interleave(c["xgroup"] or K, 1)
    y = torch.empty(M, N, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 26) // K)
    for n0 in range(0, N, step):
        q = st["q"][n0:n0 + step].long()
        w = torch.empty(q.shape[0], K, dtype=torch.float64, device=x.device)
        for half in (0, 1):
            code = q >> 4 if half else q & 15
            if c["fmt"] == "nvfp4":
                e, m = (code >> 1) & 3, (code & 1).double()
                v = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e.double() - 1))
                w[:, half::2] = torch.where(code >= 8, -v, v)
            else:
                w[:, half::2] = code.double()
        if c["fmt"] == "nvfp4":
            b = st["s"][n0:n0 + step].long()
            e, m = (b >> 3) & 15, (b & 7).double()
            s = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e.double() - 7)) * st["g"].double()
            w *= s.repeat_interleave(16, 1)
        else:
            z = st["z"][n0:n0 + step].double().repeat_interleave(c["group"], 1) if st["z"] is not None else 8.0
            w = (w - z) * st["s"][n0:n0 + step].double().repeat_interleave(c["group"], 1)
        y[:, n0:n0 + step] = torch.einsum("mk,nk->mn", x, w)
    return y if st["bias"] is None else y + st["bias"].double()


def exact(case, seed):
    if case["op"] == "w4" and case["M"] * case["N"] * case["K"] > 4 << 30:
        return None                                 # over about 20 seconds
    st = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "w4": _exact_w4}[case["op"]](case, st)
