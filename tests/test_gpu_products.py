"""4-bit floats, their products, and products grouped by expert on the GPU, each
against a plain implementation in 64 bits. Codes and scales are compared
exactly. A product is held to the rounding of its result (half a step of the
output's type) plus that of its sum: n terms added in fp32, each addition (or
alignment of a term in the tensor cores) off by at most 2^-23 of the sum of
magnitudes, so n * 2^-23 * sum |x w|."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}
INF, NAN = math.inf, math.nan


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# ---------------------------------------------------------------------------
# the definitions
# ---------------------------------------------------------------------------
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
E4M3 = torch.tensor([((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16) for m in range(8)],
                    dtype=torch.float64)[:127]                     # 127: NaN


def power(e):
    """2 ** e of whole numbers, as the bits of doubles (pow is off by a step)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def nearest(v, table):
    """Index of the nearest table entry for v >= 0 (doubles), ties to the even index, saturating."""
    t = table.to(v.device)
    mid = (t[1:] + t[:-1]) / 2
    i = torch.bucketize(v, mid)                                    # v <= mid[i]: a tie counts as below
    tie = (i < mid.numel()) & (v == mid[i.clamp_max(mid.numel() - 1)])
    return torch.where(tie & (i % 2 == 1), i + 1, i)


def ref_quantise(x, fmt):
    """x [R, K] doubles -> magnitudes with signs, scale bytes, g."""
    R, K = x.shape
    n = BLOCK[fmt]
    b = x.view(R, K // n, n)
    finite = torch.isfinite(x)
    top = b.abs().amax(2)
    if fmt == "nvfp4":
        ok = finite.all(1)
        big = torch.where(ok, x.abs().amax(1), 0.0)
        m, e = torch.frexp(big / torch.full_like(big, 2688.0))       # (a quotient by a number is a product)
        g = torch.where(m > 0, power(torch.where(m == 0.5, e - 1, e).clamp_min(-100)), 1.0)
        s = nearest(torch.where(ok[:, None], top, 0.0) / (6 * g[:, None]), E4M3)
        unit = E4M3.to(x.device)[s] * g[:, None]
        live = ok[:, None].expand_as(unit) & (unit > 0)
        g = torch.where(ok, g, NAN)
    else:
        ok = finite.view(R, K // n, n).all(2)
        m, ex = torch.frexp(torch.where(ok, top, 0.0))
        e = torch.where(m > 0, (ex - 3).clamp(-127, 127), torch.full_like(ex, -127))
        s = torch.where(ok, e + 127, torch.full_like(e, 255)).long()
        unit = torch.where(ok, power(e), 0.0)
        live, g = ok, None
    r = torch.where(live[..., None], b / torch.where(live, unit, 1.0)[..., None], 0.0)
    r = torch.where(live[..., None], r, 0.0)
    return (torch.sign(r) * E2M1.to(x.device)[nearest(r.abs(), E2M1)]).view(R, K), s.to(torch.uint8), g


def code_values(q):
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    v = E2M1.to(q.device)[c & 7]
    return torch.where(c >= 8, -v, v)


def values(q, s, g, fmt):
    """What codes and scales [.., K/2], [.., K/n] stand for, in doubles; g broadcasts over the rows."""
    if fmt == "nvfp4":
        unit = torch.cat([E4M3, torch.tensor([NAN], dtype=torch.float64)]).to(q.device)[s.long() & 127]
        if g is not None:
            unit = unit * g.double()[..., None]
    else:
        unit = torch.where(s == 255, NAN, power(s.long() - 127))
    return code_values(q) * unit.repeat_interleave(BLOCK[fmt], -1)


def check_quantised(got, x, fmt):
    v, s, g = ref_quantise(x.double(), fmt)
    torch.testing.assert_close(got[1], s, rtol=0, atol=0)
    if g is None:
        assert got[2] is None
    else:
        torch.testing.assert_close(got[2].double(), g, rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(code_values(got[0]), v, rtol=0, atol=0)


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------
SIZES = [(1, 64), (3, 128), (1, 4096), (5, 1536), (7, 2048), (4, 2112), (9, 5056), (2, 8192), (3, 16384), (2, 32768),
         (257, 320), (700, 192)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,K", SIZES)
def test_quantize(gpu_lib, R, K, dtype, fmt):
    g = gen(R * 100003 + K)
    x = (randn(g, R, K) * torch.exp(randn(g, R, 1))).to(DT[dtype])
    check_quantised(gpu_lib.quantize_fp4(x, fmt), x, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_special_rows(gpu_lib, dtype, fmt):
    t, K = DT[dtype], 256
    fin = torch.finfo(t)
    g = gen(3)
    rows = [torch.zeros(K, device="cuda"), -torch.zeros(K, device="cuda")]
    for scale in (fin.max / 8, fin.smallest_normal, fin.smallest_normal * fin.eps * 4, 2.0 ** -14, 1.0):
        rows.append((randn(g, K) * scale).clamp(fin.min, fin.max))
    rows.append(torch.full((K,), fin.max, device="cuda"))
    rows.append(torch.where(torch.arange(K, device="cuda") == 77, 1.0, 2.0 ** -12))     # one large, the rest rounds away
    one = torch.zeros(K, device="cuda")
    one[200] = -fin.smallest_normal * fin.eps                                           # the smallest subnormal alone
    rows.append(one)
    for k in (2688.0, 2680.0, 2696.0, 1344.0):                                          # at and beside the steps of g
        r = randn(g, K)
        r[5] = k
        rows.append(r)
    x = torch.stack(rows).to(t)
    check_quantised(gpu_lib.quantize_fp4(x, fmt), x, fmt)
    x = torch.cat([x, x[2:7]])
    x[-5, 3], x[-4, 40], x[-3, 255], x[-2, 0] = INF, -INF, NAN, NAN
    got = gpu_lib.quantize_fp4(x, fmt)
    check_quantised(got, x, fmt)
    y = gpu_lib.dequantize_fp4(*got, dtype=torch.float32)
    n = K if fmt == "nvfp4" else 32
    bad = (~torch.isfinite(x)).view(-1, K // n, n).any(2).repeat_interleave(n, 1)
    assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_at_the_middles(gpu_lib, dtype):
    """Every middle between two codes, exactly and a step beside it, under every mantissa of a block's scale, and block
    maxima at the middles between two scales."""
    t = DT[dtype]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    blocks = []
    for m in range(8, 16):
        for e in (0, 3, -4):
            s = m / 8 * 2.0 ** e
            b = torch.zeros(16, device="cuda")
            b[0] = 6 * s                                            # the block's scale is s (g is 1: a row with 2688)
            b[1:8], b[8:15] = mids * s, -mids * s
            blocks += [b, b * torch.where(torch.arange(16, device="cuda") == 0, 1.0, 1 + 2.0 ** -7),
                       b * torch.where(torch.arange(16, device="cuda") == 0, 1.0, 1 - 2.0 ** -7)]
    for m in range(16, 32):                                         # maxima 6 * (middle between two E4M3 values)
        b = torch.zeros(16, device="cuda")
        b[3] = 6 * m / 16
        b[4] = 1.0
        blocks += [b, b * (1 + 2.0 ** -7), b * (1 - 2.0 ** -7)]
    full = torch.zeros(16, device="cuda")
    full[0] = 2688.0
    blocks += [full] * (-len(blocks) % 4)
    x = torch.cat(blocks)
    x = torch.cat([x, full.repeat(4 * math.ceil((x.numel() + 64) / 64) - x.numel() // 16)])[None].to(t)
    assert x.shape[1] % 64 == 0
    check_quantised(gpu_lib.quantize_fp4(x, "nvfp4"), x, "nvfp4")
    check_quantised(gpu_lib.quantize_fp4(x, "mxfp4"), x, "mxfp4")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_gather_and_strides(gpu_lib, fmt):
    """Rows by index, repeated, in any order and out of range; rows further apart than K, at odd addresses."""
    g = gen(8)
    T, K, R = 50, 448, 300
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
    rows[[3, 100, 299]] = torch.tensor([-1, T, -2 ** 31], dtype=torch.int32, device="cuda")
    on = (rows >= 0) & (rows < T)
    buf = randn(g, T, 600).to(torch.bfloat16)
    for x in (buf[:, :K], buf[:, 1:K + 1], buf[:, 8:K + 8]):
        out = (torch.full((R, K // 2), 0xA5, dtype=torch.uint8, device="cuda"),
               torch.full((R, K // BLOCK[fmt]), 0xA5, dtype=torch.uint8, device="cuda"),
               torch.full((R,), -7.0, device="cuda") if fmt == "nvfp4" else None)
        got = gpu_lib.quantize_fp4(x, fmt, rows=rows, out=out)
        assert got[0] is out[0]
        check_quantised(tuple(None if o is None else o[on] for o in got), x[rows[on].long()], fmt)
        assert (got[0][~on] == 0xA5).all() and (got[1][~on] == 0xA5).all()
        assert got[2] is None or (got[2][~on] == -7).all()
        check_quantised(gpu_lib.quantize_fp4(x, fmt), x, fmt)
    got = gpu_lib.quantize_fp4(buf[:0, :K], fmt, rows=rows)          # no row to gather from: nothing is written
    assert got[0].shape == (R, K // 2)
    assert gpu_lib.quantize_fp4(buf[:0, :K], fmt)[0].shape == (0, K // 2)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("K,with_up", [(4096, False), (4160, False), (4224, True)])
def test_quantize_rows_many_times_the_tokens(gpu_lib, K, with_up, fmt):
    """So many rows that tokens are quantised once and copied: the codes of the tokens themselves, rows out of range as
    they were; also captured, on two streams at once, with scales at any word. (Rows of scales of 16, 4 and 2 bytes.)"""
    g = gen(K)
    T, R, n = 37, 8200, BLOCK[fmt]
    assert R * K >= 1 << 25
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=torch.int32)
    rows[[0, 4000, R - 1]] = torch.tensor([-1, T, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    on = (rows >= 0) & (rows < T)
    at = rows[on].long()
    xs = [randn(g, T, K + 16).to(torch.bfloat16)[:, 3:K + 3] for _ in range(3)]
    xs[1][5, 70] = NAN
    up = randn(g, T, K).to(torch.bfloat16) if with_up else None
    want = [gpu_lib.quantize_fp4(x, fmt, up=up) for x in xs]

    def room():
        s = torch.full((R * (K // n) + 16,), 0xA5, dtype=torch.uint8, device="cuda")[4:4 + R * (K // n)]
        return (torch.full((R, K // 2), 0xA5, dtype=torch.uint8, device="cuda"), s.view(R, K // n),
                torch.full((R,), -7.0, device="cuda") if fmt == "nvfp4" else None)

    def same(got, k):
        for o, w, kept in zip(got, want[k], (0xA5, 0xA5, -7.0)):
            if o is not None:
                assert torch.equal(o[on].view(torch.uint8), w[at].view(torch.uint8)) and (o[~on] == kept).all()

    same(gpu_lib.quantize_fp4(xs[0], fmt, up=up, rows=rows, out=room()), 0)
    new = gpu_lib.quantize_fp4(xs[1], fmt, up=up, rows=rows)
    assert all(o is None or torch.equal(o[on].view(torch.uint8), w[at].view(torch.uint8)) for o, w in zip(new, want[1]))
    outs, streams = [room() for _ in range(6)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        gpu_lib.quantize_fp4(xs[i % 3], fmt, up=up, rows=rows, out=o, stream=streams[i % 2])
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        same(o, i % 3)
    held, graphs = [x.clone() for x in xs[:2]], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu_lib.quantize_fp4(held[i], fmt, up=up, rows=rows, out=outs[i])
        graphs.append(graph)
    for k in range(3):
        for i in range(2):
            held[i].copy_(xs[(k + i) % 3])
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            same(outs[i], (k + i) % 3)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("R,K", [(1, 64), (33, 1536), (5, 4160), (2, 12288)])
def test_quantize_silu(gpu_lib, R, K, dtype, fmt):
    """silu(x) * up in fp32 is off by up to (5 + 1.2 |x|) 2^-23 of itself; scales and codes are those of a value within."""
    g = gen(K)
    x, up = (3 * randn(g, R, K)).to(DT[dtype]), randn(g, R, K + 8).to(DT[dtype])[:, 8:]
    got = gpu_lib.quantize_fp4(x, fmt, up=up)
    xd = x.double()
    v = xd * torch.sigmoid(xd) * up.double()
    off = (5 + 1.2 * xd.abs()) * 2.0 ** -23
    n = BLOCK[fmt]
    lo, hi = v.abs() * (1 - off), v.abs() * (1 + off)
    top = lambda a: a.view(R, K // n, n).amax(2)
    if fmt == "nvfp4":
        gs = [power(torch.frexp(a.amax(1) / 2688).exponent) for a in (lo, hi)]         # (no maximum lies at a power of two)
        assert ((got[2].double() == gs[0]) | (got[2].double() == gs[1])).all()
        gd = got[2].double()[:, None]
        s0, s1 = (nearest(top(a) / (6 * gd), E4M3) for a in (lo, hi))
        unit = E4M3.cuda()[got[1].long()] * gd
    else:
        s0, s1 = ((torch.frexp(top(a)).exponent - 3 + 127) for a in (lo, hi))
        unit = power(got[1].long() - 127)
    s = got[1].long()
    assert ((s >= s0) & (s <= s1)).all()
    unit = unit.repeat_interleave(n, 1)
    live = unit > 0
    unit = torch.where(live, unit, 1.0)
    c = code_values(got[0])
    c0, c1 = (torch.where(live, E2M1.cuda()[nearest(a / unit, E2M1)], 0.0) for a in (lo, hi))
    assert ((c.abs() >= c0) & (c.abs() <= c1)).all()
    assert ((c == 0) | (torch.sign(c) == torch.sign(v))).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_silu_far_below_zero(gpu_lib, dtype, fmt):
    """silu(x) of x below -87.3, less than 2^-119, is 0 whatever it is multiplied by; just above it is not."""
    least, most = torch.finfo(DT[dtype]).min, torch.finfo(DT[dtype]).max
    x = torch.tensor([-87.5, -88.0, -89.0, -100.0, -1000.0, least], device="cuda").repeat_interleave(64).view(6, 64).to(DT[dtype])
    up = torch.full_like(x, most)
    assert (gpu_lib.dequantize_fp4(*gpu_lib.quantize_fp4(x, fmt, up=up), dtype=torch.float32) == 0).all()
    x[:, 5] = -80.0                                          # the largest of its row and block: 6 or 4 times a scale
    q, s, g = gpu_lib.quantize_fp4(x, fmt, up=up)
    c = code_values(q)
    if dtype == "bf16":
        assert (c[:, 5] <= -4).all()
    assert (c[:, :5] == 0).all() and (c[:, 6:] == 0).all()


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_dequantize_every_code_and_scale(gpu_lib, out):
    t = DT[out]
    q = torch.arange(256, dtype=torch.uint8, device="cuda").view(8, 32).repeat(256, 1)             # [2048, 32]
    for fmt in ("nvfp4", "mxfp4"):
        cols = 64 // BLOCK[fmt]
        s = torch.arange(256, dtype=torch.uint8, device="cuda")[:128 if fmt == "nvfp4" else 256]
        s = s.repeat_interleave(8)[:, None].expand(-1, cols).contiguous()
        R = s.shape[0]
        for g in ([None, torch.tensor([0.37], device="cuda"), torch.rand(R, device="cuda") + 0.5] if fmt == "nvfp4" else [None]):
            buf = torch.full((R, 80), 9.0, dtype=t, device="cuda")
            for y in (buf[:, :64], buf[:, 3:67]):
                gpu_lib.dequantize_fp4(q[:R], s, g, out=y)
                want = values(q[:R], s, g if g is None or g.numel() > 1 else g.expand(R), fmt)
                assert torch.equal(torch.isnan(y), torch.isnan(want))
                # s * g and its product with the code, fp32 each, then the output's rounding; results below the normal
                # range of fp32 or of the output are off by half a step there
                tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps + 2.0 ** -149
                big = torch.finfo(t).max
                ok = want.abs() < big
                bound = want.abs() * (2 * 2.0 ** -24 + torch.finfo(t).eps / 2) * 1.001 + tiny
                assert ((y.double() - want).abs()[ok] <= bound[ok]).all()
            assert (buf[:, 67:] == 9).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("R,K", [(1, 64), (3, 1536), (100, 12288), (1300, 1088), (1300, 4160), (1217, 16448), (5000, 64),
                                 (4865, 4160), (6001, 8256)])
def test_dequantize_sizes(gpu_lib, R, K, fmt):
    """Every count of threads a row, and more values than L2 holds; a code times its scales has few enough bits to be exact in
    bf16 and fp32."""
    x = randn(gen(R + K), R, K).to(torch.bfloat16)
    codes = gpu_lib.quantize_fp4(x, fmt)
    want = values(*codes, fmt)
    assert torch.equal(gpu_lib.dequantize_fp4(*codes).double(), want)
    buf = torch.full((R, K + 9), 9.0, device="cuda")
    assert torch.equal(gpu_lib.dequantize_fp4(*codes, out=buf[:, 1:K + 1]).double(), want)
    assert (buf[:, 0] == 9).all() and (buf[:, K + 1:] == 9).all()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def check_product(y, x, w, bias=None):
    """y [M, N] against x [M, K] w [N, K]^T + bias, doubles. A row without NaN in x has none in y."""
    want, mag = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        want, mag = want + bias.double(), mag + bias.double().abs()
    K = x.shape[1]
    # (+ 2: the second scales and the bias; an f16 result may be subnormal)
    bound = torch.finfo(y.dtype).eps / 2 * want.abs() + (K + 4) * 2.0 ** -23 * mag
    bound = bound * (1 + torch.finfo(y.dtype).eps) + (2.0 ** -25 if y.dtype == torch.float16 else 1e-38)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    off = ((y.double() - want).abs() - bound).nan_to_num(-1.0)
    assert (off <= 0).all(), (off.max().item(), (off > 0).sum().item(), (off > 0).nonzero()[:5].tolist())


def quantised(g, moe, fmt, *shape, scale=1.0, g_shape=None):
    """A matrix in 4-bit floats [*shape[:-1], K/2] and what it stands for in doubles."""
    K, n = shape[-1], BLOCK[fmt]
    x = (scale * randn(g, *shape)).to(torch.bfloat16)
    q, s, gs = moe.quantize_fp4(x.view(-1, K), fmt)
    q, s = q.view(*shape[:-1], K // 2), s.view(*shape[:-1], K // n)
    if fmt == "nvfp4":
        if g_shape is not None:
            gs = (torch.rand(g_shape, generator=g, device="cuda") + 0.5) * scale / 448
        else:
            gs = gs.view(shape[:-1])
    return q, s, gs


LINEAR = [
    # M, N, K
    (1, 1, 64), (1, 4096, 4096), (2, 130, 128), (16, 100, 192), (17, 128, 256), (31, 129, 320), (33, 257, 4160),
    (64, 1000, 512), (129, 384, 448), (191, 96, 1024), (193, 640, 2048), (400, 300, 576), (777, 1111, 768),
    (5, 70, 32768), (4096, 4096, 704), (4001, 4090, 448), (3, 4096, 4096), (30, 512, 8192), (20, 900, 3136), (500, 4096, 4096),
    (1000, 4096, 1088),
]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_fp4(gpu_lib, M, N, K, fmt):
    g = gen(M * 7 + N * 11 + K)
    x, w = quantised(g, gpu_lib, fmt, M, K), quantised(g, gpu_lib, fmt, N, K, scale=0.02)
    xv, wv = values(*x, fmt), values(*w, fmt)
    bias = randn(g, N) if M % 2 else None
    for t in ("bf16", "f32") if K < 2048 else ("f16",):
        y = gpu_lib.linear_fp4(x, *w, bias=bias, out_dtype=DT[t])
        assert y.dtype == DT[t]
        check_product(y, xv, wv, bias)
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


def test_linear_fp4_second_scales(gpu_lib):
    """One g for W, one per row of it, none; tokens in 16 bits give the bits of the two calls."""
    g = gen(4)
    M, N, K = 50, 200, 640
    w = randn(g, 1, N, K).to(torch.bfloat16) * 0.1
    q, s, gs = gpu_lib.quantize_nvfp4(w)
    x = randn(g, M, K).to(torch.float16)
    codes = gpu_lib.quantize_fp4(x)
    xv = values(*codes, "nvfp4")
    for wg in (gs, None, torch.rand(N, generator=g, device="cuda")):
        y = gpu_lib.linear_fp4(codes, q[0], s[0], wg, out_dtype=torch.float16)
        check_product(y, xv, values(q[0], s[0], None if wg is None else wg.expand(N), "nvfp4"))
        assert torch.equal(y, gpu_lib.linear_fp4(x, q[0], s[0], wg))
    y = gpu_lib.linear_fp4((codes[0], codes[1], None), q[0], s[0], gs, out_dtype=torch.float32)
    check_product(y, values(codes[0], codes[1], None, "nvfp4"), values(q[0], s[0], gs.expand(N), "nvfp4"))
    wm = gpu_lib.quantize_fp4(w[0], "mxfp4")
    assert torch.equal(gpu_lib.linear_fp4(x, *wm), gpu_lib.linear_fp4(gpu_lib.quantize_fp4(x, "mxfp4"), *wm,
                                                                     out_dtype=torch.float16))


def test_no_rows_and_refusals(gpu_lib):
    x = torch.zeros(0, 128, dtype=torch.bfloat16, device="cuda")
    q, s, gs = gpu_lib.quantize_fp4(torch.ones(70, 128, dtype=torch.bfloat16, device="cuda"))
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert gpu_lib.linear_fp4(x, q, s, gs).shape == (0, 70)
    assert gpu_lib.linear_fp4((q[:0], s[:0], gs[:0]), q, s, gs).shape == (0, 70)
    assert gpu_lib.grouped_linear_fp4(x, q[None], s[None], None, off).shape == (0, 70)
    assert gpu_lib.grouped_linear(x, torch.ones(1, 70, 128, dtype=torch.bfloat16, device="cuda"), off).shape == (0, 70)
    assert gpu_lib.dequantize_fp4(q[:0], s[:0], gs[:0]).shape == (0, 128)
    x = torch.ones(3, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu_lib.MoeError):                     # K no multiple of 64
        gpu_lib.linear_fp4(x[:, :32], q[:, :16].contiguous(), s[:, :2].contiguous(), gs)
    with pytest.raises(gpu_lib.MoeError):                     # x not 16-byte aligned
        gpu_lib.grouped_linear(x[:, 1:121], torch.ones(1, 70, 120, dtype=torch.bfloat16, device="cuda"), off)
    for call in (lambda: gpu_lib.linear_fp4(x, q, s, gs[:3]), lambda: gpu_lib.linear_fp4(x, q, s, gs.half()),
                 lambda: gpu_lib.linear_fp4(x[:, :64], q, s, gs), lambda: gpu_lib.linear_fp4(x.float(), q, s, gs),
                 lambda: gpu_lib.linear_fp4(x, q, s[:60], gs), lambda: gpu_lib.linear_fp4(x, q, s, gs, bias=gs[:9]),
                 lambda: gpu_lib.linear_fp4(x, q, s, gs, out_dtype=torch.float64), lambda: gpu_lib.linear_fp4(x, q[::2], s[::2], None),
                 lambda: gpu_lib.linear_fp4((q, s[:, :4], None), q, s, gs), lambda: gpu_lib.quantize_fp4(x[:, :96]),
                 lambda: gpu_lib.quantize_fp4(x, "fp4"), lambda: gpu_lib.quantize_fp4(x, up=x[:2]),
                 lambda: gpu_lib.quantize_fp4(x, out=(q, s, gs)), lambda: gpu_lib.quantize_fp4(x, rows=off.long()),
                 lambda: gpu_lib.dequantize_fp4(q, s, gs[:7]), lambda: gpu_lib.dequantize_fp4(q, s.cpu(), gs),
                 lambda: gpu_lib.grouped_linear(x, x[None], off[:1]), lambda: gpu_lib.grouped_linear(x, x[None].half(), off),
                 lambda: gpu_lib.grouped_linear(x, x[None], off, out=x.to(torch.float64)),
                 lambda: gpu_lib.grouped_linear_fp4(x, q[None], s[None], gs, off.long())):
        with pytest.raises(ValueError):
            call()
    # g of one column each, where there are as many matrices as that makes scales
    w = gpu_lib.quantize_fp4(torch.ones(4, 128, dtype=torch.bfloat16, device="cuda"))
    off = torch.tensor([0, 1, 1, 2, 3], dtype=torch.int32, device="cuda")
    y = gpu_lib.grouped_linear_fp4(x, w[0][:, None], w[1][:, None], w[2][:, None], off)
    assert torch.equal(y, gpu_lib.grouped_linear_fp4(x, w[0][:, None], w[1][:, None], w[2], off))


def test_linear_fp4_exact_sums(gpu_lib):
    """Small whole numbers: every product and sum is exact, so every result is too, whatever the order."""
    g = gen(5)
    for fmt in ("nvfp4", "mxfp4"):
        n = BLOCK[fmt]
        for M, N, K in ((40, 260, 1088), (300, 130, 320), (3, 1000, 4096)):
            q = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            p = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            if fmt == "nvfp4":                              # scales 1, 1.5, 2, 3, 4: E4M3 bytes
                pick = torch.tensor([0x38, 0x3C, 0x40, 0x44, 0x48], dtype=torch.uint8, device="cuda")
            else:
                pick = torch.tensor([126, 127, 128, 129], dtype=torch.uint8, device="cuda")
            sx = pick[torch.randint(0, pick.numel(), (M, K // n), generator=g, device="cuda")]
            sw = pick[torch.randint(0, pick.numel(), (N, K // n), generator=g, device="cuda")]
            y = gpu_lib.linear_fp4((q, sx, None), p, sw, None, out_dtype=torch.float32)
            want = values(q, sx, None, fmt) @ values(p, sw, None, fmt).t()
            assert torch.equal(y.double(), want)


def offsets_of(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32,
                        device="cuda")


GROUPS = [
    # counts of each group, N, K (multiples of 8; 64 for 4-bit operands)
    ([1], 1, 8), ([5], 130, 72), ([0, 3, 0, 0, 1, 0], 100, 64), ([1] * 8, 1536, 4096), ([16, 17, 31, 32, 33], 384, 200),
    ([0] * 255 + [7], 96, 320), ([130, 1, 0, 300, 64, 65], 257, 448), ([513, 0, 255, 256, 257], 200, 136),
    ([3] * 512, 64, 64), ([0, 0, 0], 128, 128), ([40] * 12, 1000, 1016), ([900, 30], 640, 2048),
    # sums in parts: one tile a cluster, several parts, a last part that is shorter
    ([3], 384, 4096), ([32], 260, 2040), ([9], 4096, 4096),
    # ... and more tiles than the clusters that run at a time
    ([829] + 35 * [1], 100, 8192),
    # tiles of 64 and 128 rows, pairs of CTAs
    ([200], 4096, 1024), ([60, 0, 70], 1024, 1024), ([500, 300], 2048, 512), ([1000], 4096, 640), ([257, 511, 700], 2000, 1032),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped_linear(gpu_lib, counts, N, K, dtype):
    g = gen(N + K + len(counts))
    E, M = len(counts), sum(counts)
    off = offsets_of(counts)
    x, w = randn(g, M, K).to(DT[dtype]), (0.05 * randn(g, E, N, K)).to(DT[dtype])
    bias = randn(g, E, N) if N % 3 else None
    y = gpu_lib.grouped_linear(x, w, off, bias=bias)
    y32 = gpu_lib.grouped_linear(x, w, off, bias=bias, out_dtype=torch.float32)
    assert y.dtype == DT[dtype] and y.shape == (M, N)
    at = 0
    for e, c in enumerate(counts):
        if c and (E < 100 or e % 37 == 5 or e == E - 1):
            for o in (y, y32):
                check_product(o[at:at + c], x[at:at + c].double(), w[e].double(), None if bias is None else bias[e])
        at += c
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("counts,N,K", GROUPS)
def test_grouped_linear_fp4(gpu_lib, counts, N, K, fmt):
    K = (K + 63) // 64 * 64
    g = gen(N + K + len(counts))
    E, M = len(counts), sum(counts)
    off = offsets_of(counts)
    x = quantised(g, gpu_lib, fmt, max(M, 1), K)
    x = tuple(None if v is None else v[:M] for v in x)
    w = quantised(g, gpu_lib, fmt, E, N, K, scale=0.05, g_shape=(E,) if N % 2 else (E, N))
    bias = randn(g, E, N) if N % 3 else None
    y = gpu_lib.grouped_linear_fp4(x, *w, off, bias=bias)
    assert y.dtype == torch.bfloat16 and y.shape == (M, N)
    at = 0
    for e, c in enumerate(counts):
        if c and (E < 100 or e % 37 == 5 or e == E - 1):
            wg = None if w[2] is None else w[2][e].expand(N)
            check_product(y[at:at + c], values(*(None if v is None else v[at:at + c] for v in x), fmt),
                          values(w[0][e], w[1][e], wg, fmt), None if bias is None else bias[e])
        at += c
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


def test_grouped_rows_left_alone(gpu_lib):
    """Rows before the first group and behind the last, columns past N, rows between strides: as they were. Offsets that
    lead out of range or run backwards touch no other memory."""
    g = gen(9)
    M, N, K, E = 90, 70, 128, 4
    xb = randn(g, M + 2, K + 24).to(torch.bfloat16)
    x, w = xb[1:M + 1, 8:K + 8], (0.1 * randn(g, E, N, K)).to(torch.bfloat16)
    off = offsets_of([20, 0, 33, 10], first=7)
    buf = torch.full((M + 2, N + 9), -3.0, dtype=torch.float32, device="cuda")
    y = buf[1:M + 1, 5:N + 5]
    gpu_lib.grouped_linear(x, w, off, out=y)
    o = off.tolist()
    for e in range(E):
        if o[e + 1] > o[e]:
            check_product(y[o[e]:o[e + 1]], x[o[e]:o[e + 1]].double(), w[e].double())
    kept = buf.clone()
    kept[1 + o[0]:1 + o[-1], 5:N + 5] = -3.0
    assert (kept == -3).all()
    xq = gpu_lib.quantize_fp4(x)
    q, s, gs = gpu_lib.quantize_nvfp4(w)
    for bad in ([-9, 3, 2 ** 30, 2 ** 31 - 1, 5], [80, 20, 10, 200, 90], [0, 90, 0, 90, 0], [-2 ** 31, -5, -1, 0, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        buf.fill_(-3.0)
        gpu_lib.grouped_linear(x, w, off, out=y)
        gpu_lib.grouped_linear_fp4(xq, q, s, gs, off, out=y)
        torch.cuda.synchronize()
        kept = buf.clone()
        kept[1:M + 1, 5:N + 5] = -3.0
        assert (kept == -3).all()
    # groups that overlap a thousandfold are more tiles than M rows have: none is taken
    E, M, N = 512, 512, 256
    x, w = randn(g, M, 64).to(torch.bfloat16), randn(g, E, N, 64).to(torch.bfloat16)
    off = torch.tensor([0, M] * (E // 2) + [0], dtype=torch.int32, device="cuda")
    y = torch.full((M, N), -3.0, dtype=torch.float32, device="cuda")
    gpu_lib.grouped_linear(x, w, off, out=y)
    assert (y == -3).all()
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


def test_infinities_and_nan_stay_in_their_rows(gpu_lib):
    g = gen(10)
    counts, N, K = [30, 3, 50], 140, 192
    M, E = sum(counts), len(counts)
    off = offsets_of(counts)
    x, w = randn(g, M, K).to(torch.bfloat16), (0.1 * randn(g, E, N, K)).to(torch.bfloat16)
    clean = gpu_lib.grouped_linear(x, w, off)
    xb, wb = x.clone(), w.clone()
    xb[5, 100], xb[31, 0], xb[82, 191] = NAN, INF, -INF
    wb[0, 139, 64] = NAN
    y = gpu_lib.grouped_linear(xb, wb, off)
    assert torch.isnan(y[5]).all() and torch.isnan(y[:30, 139]).all()
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[[5, 31, 82]] = True
    hit[:30, 139] = True
    assert not torch.isfinite(y[31]).any() and not torch.isfinite(y[82]).any()
    assert torch.equal(y[~hit], clean[~hit])
    for fmt in ("nvfp4", "mxfp4"):
        ws = [v if v is None else v.view(E, N, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(E * N, K), fmt)]
        clean = gpu_lib.grouped_linear_fp4(gpu_lib.quantize_fp4(x, fmt), *ws, off)
        y = gpu_lib.grouped_linear_fp4(gpu_lib.quantize_fp4(xb, fmt), *ws, off)
        bad = torch.zeros(M, dtype=torch.bool, device="cuda")
        bad[[5, 31, 82]] = True
        assert torch.isnan(y[bad]).all()
        assert torch.equal(y[~bad], clean[~bad])


def test_past_32_bits(gpu_lib):
    """Weights past 2^32 elements, results past 2^31."""
    E, N, K = 260, 4096, 4096
    g = gen(11)
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[-1] = 0.02 * randn(g, N, K)
    x = randn(g, 3, K).to(torch.bfloat16)
    off = offsets_of([0] * (E - 1) + [3])
    buf = torch.empty(2 ** 31 + N + 8, dtype=torch.bfloat16, device="cuda")
    y = buf.as_strided((3, N), (2 ** 30, 1), 8)
    gpu_lib.grouped_linear(x, w, off, out=y)
    check_product(y, x.double(), w[-1].double())


def test_same_inputs_same_bits(gpu_lib):
    g = gen(12)
    counts = [100, 3, 0, 270, 1]
    off = offsets_of(counts)
    x, w = randn(g, sum(counts), 512).to(torch.float16), randn(g, 5, 300, 512).to(torch.float16)
    ws = [v if v is None else v.view(5, 300, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(1500, 512))]
    first = gpu_lib.grouped_linear(x, w, off), gpu_lib.grouped_linear_fp4(x, *ws, off)
    for _ in range(5):
        again = gpu_lib.grouped_linear(x, w, off), gpu_lib.grouped_linear_fp4(x, *ws, off)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_streams_and_graphs(gpu_lib):
    """Two streams at once, and graphs that captured the calls, replayed over new inputs."""
    g = gen(13)
    M, N, K, E = 200, 260, 448, 3
    w = (0.1 * randn(g, E, N, K)).to(torch.bfloat16)
    ws = [v.view(E, N, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(E * N, K))]
    off = [offsets_of([150, 0, 50]), offsets_of([1, 100, 60])]
    xs = [randn(g, M, K).to(torch.bfloat16) for _ in range(4)]

    def calls(x, o, stream=None):
        a = gpu_lib.grouped_linear(x, w, o, stream=stream)
        b = gpu_lib.grouped_linear_fp4(x, *ws, o, stream=stream)
        c = gpu_lib.linear_fp4(x, *(v[1] for v in ws), stream=stream)
        return a, b, c, gpu_lib.dequantize_fp4(*gpu_lib.quantize_fp4(x, "mxfp4", stream=stream), stream=stream)

    def same(a, b, rows):
        assert all(torch.equal(u[:n], v[:n]) for u, v, n in zip(a, b, (rows, rows, M, M)))

    want = [[calls(x, o) for o in off] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(20):
        got.append(calls(xs[i % 4], off[i % 2], streams[i % 2]))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        same(o, want[i % 4][i % 2], (200, 161)[i % 2])
    held, graphs = [x.clone() for x in xs[:2]], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = calls(held[i], off[i])
        graphs.append((graph, o))
    for k in range(4):
        for i in range(2):
            held[i].copy_(xs[(k + i) % 4])
            graphs[i][0].replay()
        torch.cuda.synchronize()
        for i in range(2):
            same(graphs[i][1], want[(k + i) % 4][i], (200, 161)[i])
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


@pytest.mark.parametrize("counts,N,K", [([20, 0, 300], 300, 320), ([3, 0, 5], 300, 4096), ([700, 0, 900], 2056, 768),
                                        ([2000, 0, 2500], 2056, 2048), ([6000, 0, 6500], 1000, 64)])
def test_waits_that_run_out(gpu_lib, counts, N, K):
    """Products that copy no operands: NaN in their rows and only there, the status says so once, and the next call is as
    before. (Tiles of one CTA, sums in parts, pairs of CTAs, and many tiles for each.)"""
    g = gen(14)
    off = offsets_of(counts, first=2)
    end = 2 + sum(counts)
    M = end + 8
    x, w = randn(g, M, K).to(torch.bfloat16), randn(g, 3, N, K).to(torch.bfloat16)
    ws = [v.view(3, N, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(3 * N, K))]
    xq = gpu_lib.quantize_fp4(x)
    for call in (lambda o: gpu_lib.grouped_linear(x, w, off, out=o),
                 lambda o: gpu_lib.grouped_linear_fp4(xq, *ws, off, out=o)):
        good = call(torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda"))
        held = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
        gpu_lib.hold_products(True)
        try:
            call(held)
            torch.cuda.synchronize()
        finally:
            gpu_lib.hold_products(False)
        assert torch.isnan(held[2:end]).all() and (held[:2] == 5).all() and (held[end:] == 5).all()
        assert gpu_lib.products_status() == gpu_lib.MOE_ERR_TIMEOUT
        assert gpu_lib.products_status() == gpu_lib.MOE_OK
        assert torch.equal(call(torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")), good)


@pytest.mark.parametrize("counts,N,K,clusters", [
    ([20, 0, 300], 300, 320, (False, False)), ([3, 0, 5], 300, 4096, (True, True)),
    ([700, 0, 900], 2056, 768, (True, False)), ([2000, 0, 2500], 2056, 2048, (True, True)),
    ([829] + 35 * [1], 100, 8192, (True, True))])
def test_waits_that_run_out_in_every_second_cta(gpu_lib, counts, N, K, clusters):
    """As above where only every second CTA copies none: what comes out is right or NaN, and NaN throughout where the CTAs
    of a cluster need each other (of 16-bit operands, of 4-bit ones). Second and last: sums in parts, there with several
    tiles for a CTA; third and fourth: pairs."""
    g = gen(15)
    E, off = len(counts), offsets_of(counts, first=2)
    end = 2 + sum(counts)
    M = end + 8
    x, w = randn(g, M, K).to(torch.bfloat16), randn(g, E, N, K).to(torch.bfloat16)
    ws = [v.view(E, N, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(E * N, K))]
    xq = gpu_lib.quantize_fp4(x)
    for cluster, call in zip(clusters, (lambda o: gpu_lib.grouped_linear(x, w, off, out=o),
                                        lambda o: gpu_lib.grouped_linear_fp4(xq, *ws, off, out=o))):
        good = call(torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda"))
        held = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
        gpu_lib.hold_products(2)
        try:
            call(held)
            torch.cuda.synchronize()
        finally:
            gpu_lib.hold_products(0)
        none = torch.isnan(held)
        assert none.any() and torch.equal(held[~none], good[~none]) and not none[:2].any() and not none[end:].any()
        assert none[2:end].all() or not cluster
        assert gpu_lib.products_status() == gpu_lib.MOE_ERR_TIMEOUT
        assert torch.equal(call(torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")), good)
        assert gpu_lib.products_status() == gpu_lib.MOE_OK


FIRST_USE = """
import torch
import top_moe_expert_router_gb300 as moe
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(40, 512, generator=g, device="cuda").to(torch.bfloat16)
w = (0.1 * torch.randn(3, 300, 512, generator=g, device="cuda")).to(torch.bfloat16)
off = torch.tensor([0, 10, 10, 40], dtype=torch.int32, device="cuda")
def calls():
    q, s, gs = moe.quantize_fp4(w.view(900, 512))
    q, s, gs = q.view(3, 300, 256), s.view(3, 300, 32), gs.view(3, 300)
    return (moe.dequantize_fp4(*moe.quantize_fp4(x, "mxfp4")), moe.grouped_linear(x, w, off),
            moe.grouped_linear_fp4(x, q, s, gs, off), moe.linear_fp4(x, q[1], s[1], gs[1]))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
print("same" if all(torch.equal(a, b) for a, b in zip(got, calls())) else "different")
"""


def test_first_use_of_every_operator_inside_a_capture():
    """A process whose first call of each operator is a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,fmt", [(1, "nvfp4"), (13, "mxfp4"), (300, "nvfp4")])
def test_experts_from_the_operators(gpu_lib, T, fmt):
    """Routing, gathered quantisation, the experts' products in 4 bits and in 16, silu between them, the weighted sum:
    each step against the definition on what the step before gave."""
    g = gen(T)
    E, k, d, I = 32, 4, 512, 320
    x, logits = randn(g, T, d).to(torch.bfloat16), randn(g, T, E)
    r = gpu_lib.route_logits(logits, k)
    off, perm = r["offsets"], r["perm"]
    W = {n: (0.05 * randn(g, E, *s)).to(torch.bfloat16) for n, s in (("gate", (I, d)), ("up", (I, d)), ("down", (d, I)))}
    Q = {n: [v if v is None else v.view(E, w.shape[1], *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(-1, w.shape[2]), fmt)]
         for n, w in W.items()}
    xq = gpu_lib.quantize_fp4(x, fmt, rows=perm)
    check_quantised(xq, x[perm.long()], fmt)
    gate = gpu_lib.grouped_linear_fp4(xq, *Q["gate"], off)
    up = gpu_lib.grouped_linear_fp4(xq, *Q["up"], off)
    hq = gpu_lib.quantize_fp4(gate, fmt, up=up)
    y4 = gpu_lib.grouped_linear_fp4(hq, *Q["down"], off)
    xg = x[perm.long()]
    gate16, up16 = gpu_lib.grouped_linear(xg, W["gate"], off), gpu_lib.grouped_linear(xg, W["up"], off)
    h16 = (torch.nn.functional.silu(gate16.float()) * up16.float()).to(torch.bfloat16)
    y16 = gpu_lib.grouped_linear(h16, W["down"], off)
    o = off.tolist()
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        if o[e + 1] == o[e]:
            continue
        cut = lambda t: tuple(None if v is None else v[rows] for v in t)
        one = lambda n: values(*(None if v is None else v[e] for v in Q[n]), fmt)
        check_product(gate[rows], values(*cut(xq), fmt), one("gate"))
        check_product(up[rows], values(*cut(xq), fmt), one("up"))
        check_product(y4[rows], values(*cut(hq), fmt), one("down"))
        check_product(gate16[rows], xg[rows].double(), W["gate"][e].double())
        check_product(y16[rows], h16[rows].double(), W["down"][e].double())
    # the layer itself on the same weights: its experts are the 16-bit products' (h and the expert outputs rounded
    # to bf16 here, sums fp32 in both: three roundings of 2^-8 a term, on sums that may cancel)
    out = (y16.float()[r["pos"].long()] * r["w"][..., None]).sum(1)
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = r["ids"][t, j]
            gd, ud = W["gate"][e].double() @ x[t].double(), W["up"][e].double() @ x[t].double()
            ref[t] += r["w"][t, j].double() * (W["down"][e].double() @ (gd * torch.sigmoid(gd) * ud))
    assert ((out.double() - ref).norm(dim=1) <= 4 * 2.0 ** -8 * ref.norm(dim=1)).all()
