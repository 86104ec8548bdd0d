"""Timed cases of the products on 4-bit floats and of the products by expert:
quantisation of tokens to microscaled 4-bit floats (and back), dense products of
two such matrices, and products grouped by expert with ragged sizes, in 16 bits
and in 4.

``listed()`` and ``draw()`` give cases, ``prepare()`` a case's inputs on the
GPU, ``run()`` one pass: the plain form in elementary torch operations, or,
with ``own`` set, the framework's kernels. ``exact()`` is the definition in 64
bits, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False

_T = {"bf16": torch.bfloat16, "f16": torch.float16}
_BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _quant(T, K, R, dtype, fmt, up):
    """R: rows gathered from the T tokens, 0 for all of them in order. up: silu(x) * up is what is quantised."""
    return {"op": "quant", "T": T, "K": K, "R": R, "dtype": dtype, "fmt": fmt, "up": up}


def _linear(M, N, K, dtype, fmt, bias):
    return {"op": "linear", "M": M, "N": N, "K": K, "dtype": dtype, "fmt": fmt, "bias": bias}


def _group(op, R, E, A, N, K, dtype, fmt, bias, skew):
    """R rows for A of E experts, the more unevenly the larger skew is."""
    return {"op": op, "R": R, "E": E, "A": A, "N": N, "K": K, "dtype": dtype, "fmt": fmt, "bias": bias, "skew": skew}


def listed():
    cases = [
        # one decode token at the layer's hidden size
        ("quant_token", _quant(1, 4096, 0, "bf16", "nvfp4", False)),
        # a ragged batch with rows that are no whole number of 256-column stages, blocks of 32
        ("quant_ragged", _quant(777, 5056, 0, "f16", "mxfp4", False)),
        # the prefill workload's prompt, each token gathered to its eight experts' rows
        ("quant_gather", _quant(4096, 4096, 32768, "bf16", "nvfp4", False)),
        # the activation between an expert's products: silu(gate) * up of those rows
        ("quant_silu", _quant(32768, 1536, 0, "bf16", "nvfp4", True)),
        # one decode token through a square projection, its quantisation among the pass
        ("linear_token", _linear(1, 4096, 4096, "bf16", "nvfp4", False)),
        # a batch of decode tokens through a wide projection
        ("linear_batch", _linear(48, 12288, 4096, "f16", "mxfp4", True)),
        # a prompt through a wide projection at the largest hidden size of the layer
        ("linear_long", _linear(8192, 16384, 8192, "bf16", "nvfp4", False)),
        # the gate product of one decode token's eight experts
        ("group_token", _group("group", 8, 256, 8, 1536, 4096, "bf16", "", False, 0.0)),
        # the gate product of the prefill workload: 4096 tokens, eight experts each, uneven loads
        ("group_prompt", _group("group", 32768, 256, 256, 1536, 4096, "bf16", "", False, 0.3)),
        # few wide experts with biases and an odd length
        ("group_ragged", _group("group", 5003, 12, 11, 2712, 2712, "f16", "", True, 0.3)),
        # the down product of sixteen decode tokens with 4-bit experts
        ("group4_batch", _group("group4", 128, 256, 96, 4096, 1536, "bf16", "nvfp4", False, 0.2)),
        # the gate product of the prefill workload with 4-bit experts
        ("group4_prompt", _group("group4", 32768, 256, 256, 1536, 4096, "bf16", "nvfp4", False, 0.3)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "group", "group4"])
    dtype, fmt = rng.choice(["bf16", "f16"]), rng.choice(["nvfp4", "mxfp4"])
    if op == "quant":
        K = 64 * _log(rng, 1, 200)
        T = min(_log(rng, 1, 32768), (1 << 26) // K)
        up = rng.random() < 0.35
        R = 0 if up or rng.random() < 0.5 else min(T * rng.randint(1, 8), (1 << 27) // K)
        return _quant(T, K, R, dtype, fmt, up)
    if op == "linear":
        M, K = _log(rng, 1, 8192), 64 * _log(rng, 2, 128)
        N = min(_log(rng, 64, 32768), (1 << 37) // (M * K), (1 << 28) // K)
        return _linear(M, N, K, dtype, fmt, rng.random() < 0.3)
    E, R = _log(rng, 4, 256), _log(rng, 1, 32768)
    K = 64 * _log(rng, 2, 64) if op == "group4" else 8 * _log(rng, 16, 512)
    N = min(_log(rng, 64, 4096), (1 << 30) // (E * K))
    A = rng.randint((min(E, R) + 1) // 2, min(E, R))
    return _group(op, R, E, A, N, K, dtype, fmt if op == "group4" else "", rng.random() < 0.3, rng.choice([0.0, 0.3, 0.6]))


# ---------------------------------------------------------------------------
# 4-bit floats in elementary operations: codes e2m1 (two to a byte, the low nibble first), a scale per block of
# 16 (E4M3) or 32 (a power of two), and for blocks of 16 a second scale
# ---------------------------------------------------------------------------
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _codes(r):
    """The nearest of the eight magnitudes, at the middle between two the one with the even code; the sign in bit 3."""
    a = r.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5).to(torch.uint8))
    code |= (r < 0).to(torch.uint8) << 3
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _power(e):
    """2 ** e of whole numbers e in [-127, 127], as the bits of a float."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _row_scale(x):
    """The smallest power of two g with max|x| / (6 * 448) <= g, 1 for a row of zeros."""
    m, e = torch.frexp(x.abs().amax(-1) / (6 * 448))
    return torch.where(m > 0, _power(torch.where(m == 0.5, e - 1, e).clamp_min(-100)), 1.0)


def _quantise(x, fmt, g=None):
    """x [..., K] in 32 bits -> codes [..., K/2], scales [..., K/block] as bytes. g: the second scale, by rows."""
    b = x.unflatten(-1, (-1, _BLOCK[fmt]))
    top = b.abs().amax(-1)
    if fmt == "nvfp4":
        s = (top / 6 / g[..., None]).to(torch.float8_e4m3fn)
        unit, s = s.float() * g[..., None], s.view(torch.uint8)
    else:
        e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
        e = torch.where(top > 0, e, -127)
        unit, s = _power(e), (e + 127).to(torch.uint8)
    r = torch.where(unit[..., None] > 0, b / unit[..., None], 0.0)
    return _codes(r.flatten(-2)), s


def _values(q, s, g, fmt):
    """What codes and scales stand for, in 32 bits. g: the second scale, by rows, or None."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=q.device)
    v = table[torch.stack((q & 15, q >> 4), -1).flatten(-2).int()].unflatten(-1, (-1, _BLOCK[fmt]))
    if fmt == "nvfp4":
        unit = s.view(torch.float8_e4m3fn).float() * g[..., None]
    else:
        unit = _power(s.int() - 127)
    return (v * unit[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _tokens(g, T, K):
    """Activations: a few channels stand out."""
    return _randn(g, T, K) * (1 + 8 * (torch.rand(K, generator=g, device="cuda") < 0.01).float())


def _weights(g, E, N, K, fmt):
    """E matrices in 4 bits: codes [E, N, K/2], scales [E, N, K/block], and for blocks of 16 one scale a matrix."""
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // _BLOCK[fmt], dtype=torch.uint8, device="cuda")
    gs = torch.empty(E, device="cuda") if fmt == "nvfp4" else None
    for at in range(0, E, 32):
        W = 0.02 * _randn(g, min(32, E - at), N, K)
        if gs is not None:
            gs[at:at + 32] = W.abs().amax((1, 2)) / (6 * 448)
        q[at:at + 32], s[at:at + 32] = _quantise(W, fmt, None if gs is None else gs[at:at + 32, None].expand(-1, N))
    return q, s, gs


def _prepare_quant(c, g):
    T, K, t = c["T"], c["K"], _T[c["dtype"]]
    R = c["R"] or T
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32) if c["R"] else None
    return {"x": _tokens(g, T, K).to(t), "up": _randn(g, T, K).to(t) if c["up"] else None, "rows": rows,
            "codes": (torch.empty(R, K // 2, dtype=torch.uint8, device="cuda"),
                      torch.empty(R, K // _BLOCK[c["fmt"]], dtype=torch.uint8, device="cuda"),
                      torch.empty(R, device="cuda") if c["fmt"] == "nvfp4" else None),
            "out": torch.empty(R, K, dtype=t, device="cuda")}


def _prepare_linear(c, g):
    M, N, K, t = c["M"], c["N"], c["K"], _T[c["dtype"]]
    q, s, gs = _weights(g, 1, N, K, c["fmt"])
    return {"x": _tokens(g, M, K).to(t), "q": q[0], "s": s[0], "g": gs,
            "bias": 0.1 * _randn(g, N) if c["bias"] else None, "out": torch.empty(M, N, dtype=t, device="cuda")}


def _prepare_group(c, g, seed):
    R, E, A, N, K, t = c["R"], c["E"], c["A"], c["N"], c["K"], _T[c["dtype"]]
    r = np.random.RandomState(int(seed) % (1 << 32))
    share = (1.0 + np.arange(A)) ** -c["skew"]
    counts = 1 + r.multinomial(R - A, r.permutation(share / share.sum()))
    used = np.sort(r.choice(E, A, replace=False))
    per = np.zeros(E, np.int64)
    per[used] = counts
    st = {"offsets": torch.from_numpy(np.concatenate([[0], np.cumsum(per)]).astype(np.int32)).cuda(),
          "used": torch.from_numpy(used).cuda(), "most": int(counts.max()),
          "bias": 0.1 * _randn(g, E, N) if c["bias"] else None, "out": torch.empty(R, N, dtype=t, device="cuda")}
    if c["op"] == "group":
        w = torch.empty(E, N, K, dtype=t, device="cuda")
        for at in range(0, E, 32):
            w[at:at + 32] = 0.02 * _randn(g, min(32, E - at), N, K)
        return dict(st, x=_tokens(g, R, K).to(t), w=w)
    x = _tokens(g, R, K).to(t).float()              # quantised once for all of a layer's products
    xg = _row_scale(x) if c["fmt"] == "nvfp4" else None
    xq, xs = _quantise(x, c["fmt"], xg)
    q, s, gs = _weights(g, E, N, K, c["fmt"])
    return dict(st, x=(xq, xs, xg), q=q, s=s, g=gs)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quant":
        made = _prepare_quant(case, g)
    elif case["op"] == "linear":
        made = _prepare_linear(case, g)
    else:
        made = _prepare_group(case, g, seed)
    return dict(made, case=case)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_quantised(x, fmt):
    g = _row_scale(x) if fmt == "nvfp4" else None
    return *_quantise(x, fmt, g), g


def _plain_quant(c, st):
    x = st["x"] if st["rows"] is None else st["x"][st["rows"].long()]
    x = x.float()
    if st["up"] is not None:
        x = x / (1 + torch.exp(-x)) * st["up"].float()
    return _values(*_plain_quantised(x, c["fmt"]), c["fmt"]).to(st["x"].dtype)


def _plain_linear(c, st):
    x = _values(*_plain_quantised(st["x"].float(), c["fmt"]), c["fmt"])
    y = x @ _values(st["q"], st["s"], None if st["g"] is None else st["g"].expand(c["N"]), c["fmt"]).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(st["x"].dtype)


def _plain_group(c, st):
    """The used experts' rows padded to the longest group, one product for each expert."""
    if c["op"] == "group":
        x, w = st["x"].float(), st["w"][st["used"]].float()
    else:
        x = _values(*st["x"], c["fmt"])
        g = None if st["g"] is None else st["g"][st["used"], None].expand(-1, c["N"])
        w = _values(st["q"][st["used"]], st["s"][st["used"]], g, c["fmt"])
    first = st["offsets"][st["used"]].long()
    r = torch.arange(c["R"], device=x.device)
    e = torch.searchsorted(first, r, right=True) - 1            # a row's place among the used experts
    at = e * st["most"] + r - first[e]
    padded = torch.zeros(c["A"] * st["most"], c["K"], device=x.device)
    padded[at] = x
    y = torch.bmm(padded.view(c["A"], st["most"], c["K"]), w.transpose(1, 2))
    if st["bias"] is not None:
        y = y + st["bias"][st["used"]][:, None, :]
    return y.view(-1, c["N"])[at].to(_T[c["dtype"]])


def _own_quant(moe, c, st):
    codes = moe.quantize_fp4(st["x"], c["fmt"], up=st["up"], rows=st["rows"], out=st["codes"])
    return moe.dequantize_fp4(*codes, out=st["out"])


def _own_linear(moe, c, st):
    return moe.linear_fp4(st["x"], st["q"], st["s"], st["g"], bias=st["bias"], out=st["out"])


def _own_group(moe, c, st):
    if c["op"] == "group":
        return moe.grouped_linear(st["x"], st["w"], st["offsets"], bias=st["bias"], out=st["out"])
    return moe.grouped_linear_fp4(st["x"], st["q"], st["s"], st["g"], st["offsets"], bias=st["bias"], out=st["out"])


def run(state):
    c = state["case"]
    if own:
        import top_moe_expert_router_gb300 as moe
        return {"quant": _own_quant, "linear": _own_linear}.get(c["op"], _own_group)(moe, c, state)
    return {"quant": _plain_quant, "linear": _plain_linear}.get(c["op"], _plain_group)(c, state)


# ---------------------------------------------------------------------------
# the work a pass cannot do without
# ---------------------------------------------------------------------------
def _fp4_bytes(rows, K, fmt):
    return rows * (K // 2 + K // _BLOCK[fmt])


def work(c):
    if c["op"] == "quant":
        R = c["R"] or c["T"]
        g = 4 * R if c["fmt"] == "nvfp4" else 0
        # the tokens (and rows) in; codes, scales and the values that they stand for out
        return {"bytes": c["T"] * c["K"] * (4 if c["up"] else 2) + 4 * c["R"] + _fp4_bytes(R, c["K"], c["fmt"]) + g
                + 2 * R * c["K"], "flops": 4 * R * c["K"]}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * M * K + _fp4_bytes(N, K, c["fmt"]) + 2 * M * N + (4 * N if c["bias"] else 0),
                "flops": 2 * M * N * K}
    R, A, N, K = c["R"], c["A"], c["N"], c["K"]
    if c["op"] == "group":
        operands = 2 * R * K + 2 * A * N * K
    else:
        operands = _fp4_bytes(R, K, c["fmt"]) + _fp4_bytes(A * N, K, c["fmt"]) + (4 * R + 4 * A if c["fmt"] == "nvfp4" else 0)
    return {"bytes": operands + 2 * R * N + 4 * (c["E"] + 1) + (4 * A * N if c["bias"] else 0), "flops": 2 * R * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_power(v):
    """2 ** v of whole numbers v, as the bits of a double."""
    return ((v.long() + 1023) << 52).view(torch.float64)


def _exact_exponent(v):
    """floor(log2 v) of positive doubles."""
    return (v.contiguous().view(torch.int64) >> 52) - 1023


def _exact_step(v, least, bits):
    """v rounded to a float of so many bits behind the leading one, with steps no smaller than 2^least."""
    step = _exact_power((_exact_exponent(v.abs().clamp_min(1e-300)) - bits).clamp_min(least))
    return torch.round(v / step) * step                         # (to even)


def _exact_rounded(x, fmt):
    """x in doubles -> what its 4-bit form stands for."""
    K, n = x.shape[-1], _BLOCK[fmt]
    top = torch.stack([b.abs().max(-1).values for b in x.split(n, -1)], -1)
    if fmt == "nvfp4":
        r = x.abs().max(-1, keepdim=True).values / 2688
        e = _exact_exponent(r.clamp_min(1e-300))
        e = e + (_exact_power(e) < r).long()
        g = torch.where(r > 0, _exact_power(e.clamp_min(-100)), 1.0)
        unit = _exact_step(top / (6 * g), -9, 3).clamp_max(448) * g
    else:
        e = (_exact_exponent(top.clamp_min(1e-300)) - 2).clamp(-127, 127)
        unit = _exact_power(torch.where(top > 0, e, -127))
    unit = unit.repeat_interleave(n, -1)[..., :K]
    v = x / torch.where(unit > 0, unit, 1.0)
    return torch.where(unit > 0, _exact_step(v, -1, 1).clamp(-6, 6) * unit, 0.0)


def _exact_values(q, s, g, fmt):
    """Codes and scales by their fields. g: one scale a row, one for all, or None."""
    v = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    for half in (0, 1):
        code = (q >> 4 if half else q & 15).long()
        e, m = (code >> 1) & 3, (code & 1).double()
        a = torch.where(e == 0, m / 2, (1 + m / 2) * _exact_power(e - 1))
        v[..., half::2] = torch.where(code >= 8, -a, a)
    b = s.long()
    if fmt == "nvfp4":
        e, m = (b >> 3) & 15, (b & 7).double()
        unit = torch.where(e == 0, m / 512, (1 + m / 8) * _exact_power(e - 7)) * g.double().reshape(-1, 1)
    else:
        unit = _exact_power(b - 127)
    return v * unit.repeat_interleave(_BLOCK[fmt], -1)


def _exact_quant(c, st):
    step = max(1, (1 << 26) // c["K"])
    R, done = c["R"] or c["T"], []
    for at in range(0, R, step):
        pick = slice(at, at + step) if st["rows"] is None else st["rows"][at:at + step].long()
        x = st["x"][pick].double()
        if st["up"] is not None:
            x = x * torch.sigmoid(x) * st["up"][pick].double()
        done.append(_exact_rounded(x, c["fmt"]))
    return torch.cat(done)


def _exact_linear(c, st):
    y = torch.einsum("mk,nk->mn", _exact_rounded(st["x"].double(), c["fmt"]),
                     _exact_values(st["q"], st["s"], st["g"], c["fmt"]))
    return y if st["bias"] is None else y + st["bias"].double()


def _exact_group(c, st):
    off = st["offsets"].tolist()
    y = torch.empty(c["R"], c["N"], dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        if c["op"] == "group":
            x, w = st["x"][lo:hi].double(), st["w"][e].double()
        else:
            xg, g = st["x"][2], st["g"]
            x = _exact_values(st["x"][0][lo:hi], st["x"][1][lo:hi], None if xg is None else xg[lo:hi], c["fmt"])
            w = _exact_values(st["q"][e], st["s"][e], None if g is None else g[e], c["fmt"])
        y[lo:hi] = torch.einsum("mk,nk->mn", x, w)
        if st["bias"] is not None:
            y[lo:hi] += st["bias"][e].double()
    return y


def exact(case, seed):
    st = prepare(case, seed)
    return {"quant": _exact_quant, "linear": _exact_linear}.get(case["op"], _exact_group)(case, st)
