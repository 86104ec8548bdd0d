"""Products by expert and 4-bit floats where few tests go: sums that have to be
exact in 16 bits, addresses past 32 bits, and how calls end whose waits run out."""
import pytest
import torch

from test_gpu_products import BLOCK, DT, check_product, check_quantised, gen, offsets_of, power, randn, values

pytestmark = pytest.mark.gpu


# counts of each group, N, K: tiles of 32 rows, those with K in parts, of 64 and 128 rows, pairs of CTAs
EXACT = [([1], 100, 40), ([3, 0, 30], 260, 4096), ([1], 4096, 4096), ([829] + 35 * [1], 100, 8192), ([200], 4096, 1024),
         ([60, 0, 70], 1024, 1032), ([500, 300], 2048, 520), ([1000], 4096, 640), ([257, 511, 700], 2000, 1032)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,N,K", EXACT)
def test_grouped_linear_exact_sums(gpu_lib, counts, N, K, dtype):
    """Small whole numbers: sums of up to 8192 products of at most 49 stay below 2^24 in magnitude, so every sum of some of
    them is exact in fp32, and every result is too, whatever the order."""
    g = gen(N + K + len(counts))
    E, M = len(counts), sum(counts)
    assert 49 * K < 1 << 24
    off = offsets_of(counts)
    x = torch.randint(-7, 8, (M, K), generator=g, device="cuda").to(DT[dtype])
    w = torch.randint(-7, 8, (E, N, K), generator=g, device="cuda").to(DT[dtype])
    bias = torch.randint(-9, 10, (E, N), generator=g, device="cuda").float()
    y = gpu_lib.grouped_linear(x, w, off, bias=bias, out_dtype=torch.float32)
    at = 0
    for e, c in enumerate(counts):
        want = x[at:at + c].double() @ w[e].double().t() + bias[e].double()
        assert torch.equal(y[at:at + c].double(), want)
        at += c
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


@pytest.mark.parametrize("fmt,K", [("nvfp4", 4096), ("nvfp4", 4160), ("mxfp4", 4096), ("mxfp4", 4160)])
def test_4bit_weights_past_32_bits(gpu_lib, fmt, K):
    """Codes past 2^32 elements, scales of whole 16 bytes a row (4096 columns) and of words (4160): the first and the last
    expert, whose weights alone are not 0."""
    E, N = 270, 4096
    assert (E - 1) * N * K > 1 << 32
    g = gen(K)
    q = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(E, N, K // BLOCK[fmt], dtype=torch.uint8, device="cuda")
    gs = torch.ones(E, N, device="cuda") if fmt == "nvfp4" else None
    for e in (0, E - 1):
        codes = gpu_lib.quantize_fp4((0.02 * randn(g, N, K)).to(torch.bfloat16), fmt)
        q[e], s[e] = codes[0], codes[1]
        if gs is not None:
            gs[e] = codes[2]
    for first, last in ((3, 5), (150, 170)):
        x = gpu_lib.quantize_fp4(randn(g, first + last, K).to(torch.bfloat16), fmt)
        off = offsets_of([first] + [0] * (E - 2) + [last])
        y = gpu_lib.grouped_linear_fp4(x, q, s, gs, off)
        for e, rows in ((0, slice(0, first)), (E - 1, slice(first, first + last))):
            check_product(y[rows], values(*(None if v is None else v[rows] for v in x), fmt),
                          values(q[e], s[e], None if gs is None else gs[e], fmt))
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


@pytest.mark.parametrize("M", [70, 150, 400])
def test_results_past_32_bits(gpu_lib, M):
    """Rows of y so far apart that its last elements lie past 2^31: tiles of 64 and 128 rows and pairs of CTAs, whole rows of
    16-byte stores and single elements."""
    N, K = 4096, 256
    g = gen(M)
    x, w = randn(g, M, K).to(torch.bfloat16), (0.1 * randn(g, 1, N, K)).to(torch.bfloat16)
    off = offsets_of([M])
    ws = [v.view(1, N, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w[0])]
    want = gpu_lib.grouped_linear(x, w, off), gpu_lib.grouped_linear_fp4(x, *ws, off)
    ld = -(-(2 ** 31 + 9) // (M - 1) // 8) * 8
    buf = torch.empty((M - 1) * ld + N + 8, dtype=torch.bfloat16, device="cuda")
    assert (M - 1) * ld > 1 << 31
    for first in (0, 8, 1):
        y = buf.as_strided((M, N), (ld, 1), first)
        assert (gpu_lib.grouped_linear(x, w, off, out=y) == want[0]).all()
        assert (gpu_lib.grouped_linear_fp4(x, *ws, off, out=y) == want[1]).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantisation_past_32_bits(gpu_lib, fmt):
    """Tokens, codes and values past 2^31 elements, each row by itself and gathered (from few tokens: by way of their codes):
    the rows around that border and the last."""
    K = 4096
    T = (1 << 31) // K + 700
    g = gen(5)
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    for at in range(0, T, 1 << 16):
        x[at:at + (1 << 16)] = randn(g, min(1 << 16, T - at), K)
    look = torch.tensor([0, 1, T // 2, T - 702, T - 701, T - 700, T - 699, T - 2, T - 1], device="cuda")
    pick = lambda t, at: tuple(None if v is None else v[at] for v in t)
    got = gpu_lib.quantize_fp4(x, fmt)
    check_quantised(pick(got, look), x[look], fmt)
    out = gpu_lib.dequantize_fp4(*got)
    assert torch.equal(out[look].double(), values(*pick(got, look), fmt))
    del out, got
    rows = torch.randint(0, T, (T,), generator=g, device="cuda", dtype=torch.int32)
    rows[look] = torch.arange(T - look.numel(), T, device="cuda", dtype=torch.int32)
    got = gpu_lib.quantize_fp4(x, fmt, rows=rows)
    check_quantised(pick(got, look), x[rows[look].long()], fmt)
    few = rows % 512
    got = gpu_lib.quantize_fp4(x[:512], fmt, rows=few)
    check_quantised(pick(got, look), x[few[look].long()], fmt)


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4", "mxfp4"])
def test_pairs_leave_once_their_copies_have_landed(gpu_lib, fmt):
    """Pairs of CTAs of which the second copies no operands: waits run out after 1.5 s, and what the first has issued has
    landed long before. The call takes one such limit, not a second one for copies that nobody issued."""
    g = gen(21)
    counts, N, K = [2000, 0, 2500], 2056, 2048
    off, M = offsets_of(counts), sum(counts)
    x, w = randn(g, M, K).to(torch.bfloat16), (0.1 * randn(g, 3, N, K)).to(torch.bfloat16)
    if fmt == "bf16":
        call = lambda: gpu_lib.grouped_linear(x, w, off)
    else:
        xq = gpu_lib.quantize_fp4(x, fmt)
        ws = [v if v is None else v.view(3, N, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(3 * N, K), fmt)]
        call = lambda: gpu_lib.grouped_linear_fp4(xq, *ws, off)
    good = call()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    gpu_lib.hold_products(2)
    try:
        start.record()
        held = call()
        end.record()
        torch.cuda.synchronize()
    finally:
        gpu_lib.hold_products(0)
    assert torch.isnan(held).all()
    assert start.elapsed_time(end) < 2500
    assert gpu_lib.products_status() == gpu_lib.MOE_ERR_TIMEOUT
    assert torch.equal(call(), good)
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
@pytest.mark.parametrize("counts,N,K,limits", [([3], 384, 4096, 1), ([32], 384, 8192, 1), ([829] + 35 * [1], 100, 8192, 2)])
def test_parts_leave_once_their_sums_have_landed(gpu_lib, counts, N, K, limits, fmt):
    """K in parts, where every second CTA copies no operands: at about the time at which it gives up and sends NaN, the others
    give up waiting for its sums. Whichever comes first, what was sent has landed before a CTA leaves, and nobody waits
    for what was not. With one tile for a CTA that takes one limit of 1.5 s; with several a CTA that still had the sums of the
    first waits once more."""
    g = gen(22)
    E, off, M = len(counts), offsets_of(counts), sum(counts)
    x, w = randn(g, M, K).to(torch.bfloat16), (0.1 * randn(g, E, N, K)).to(torch.bfloat16)
    if fmt == "bf16":
        call = lambda: gpu_lib.grouped_linear(x, w, off)
    else:
        xq = gpu_lib.quantize_fp4(x, fmt)
        ws = [v.view(E, N, *v.shape[1:]) for v in gpu_lib.quantize_fp4(w.view(E * N, K), fmt)]
        call = lambda: gpu_lib.grouped_linear_fp4(xq, *ws, off)
    good = call()
    for _ in range(2):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        gpu_lib.hold_products(2)
        try:
            start.record()
            held = call()
            end.record()
            torch.cuda.synchronize()
        finally:
            gpu_lib.hold_products(0)
        none = torch.isnan(held)
        assert none.all()
        assert start.elapsed_time(end) < 1500 * limits + 1000
        assert gpu_lib.products_status() == gpu_lib.MOE_ERR_TIMEOUT
    assert torch.equal(call(), good)
    assert gpu_lib.products_status() == gpu_lib.MOE_OK


@pytest.mark.parametrize("op", ["grouped_linear", "linear_fp4", "linear_nvfp4"])
def test_every_wait_that_ran_out_is_reported(gpu_lib, op):
    """The status is asked for all the time, on another stream, while one call after the other runs out of its waits: whatever
    the moment at which a bit is set, one of the answers has it."""
    g = gen(23)
    x, w = randn(g, 1, 128).to(torch.bfloat16), randn(g, 1, 64, 128).to(torch.bfloat16)
    hold, status = gpu_lib.hold_products, gpu_lib.products_status
    side, asks = torch.cuda.Stream(), torch.cuda.Stream()
    if op == "grouped_linear":
        call = lambda off=offsets_of([1]): gpu_lib.grouped_linear(x, w, off, stream=side)
    elif op == "linear_fp4":
        xq, ws = gpu_lib.quantize_fp4(x), gpu_lib.quantize_fp4(w[0])
        call = lambda: gpu_lib.linear_fp4(xq, *ws, stream=side)
    else:
        q, s, gs = gpu_lib.quantize_nvfp4(w)
        hold, status = gpu_lib.hold_linear_w4, gpu_lib.linear_w4_status
        call = lambda: gpu_lib.linear_nvfp4(x, q[0], s[0], gs, stream=side)
    good = call()
    torch.cuda.synchronize()
    assert status(asks) == gpu_lib.MOE_OK
    for _ in range(8):
        hold(True)
        try:
            y = call()
        finally:
            hold(False)
        answers = []
        while not side.query():
            answers.append(status(asks))
        answers.append(status(asks))
        assert torch.isnan(y).all() and gpu_lib.MOE_ERR_TIMEOUT in answers
        assert status(asks) == gpu_lib.MOE_OK
    assert torch.equal(call(), good)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scales_of_silu_at_the_middles(gpu_lib, dtype):
    """silu(x) * up where it is exact: x of 32 or more, where 1 + exp(-x) is 1, and so a product of two short values. Block
    maxima at 6 times every middle between two E4M3 values, and at the products next to it."""
    t = DT[dtype]
    xs, ups = [], []
    for m in range(17, 32, 2):                              # middles m / 16, in three binades
        for e in (-3, 0, 4):
            for near in (0.0, 2.0 ** -7, -(2.0 ** -7)):
                x = torch.zeros(16, device="cuda")
                up = torch.zeros(16, device="cuda")
                x[3], up[3] = 32 * m / 16, 6 * 2.0 ** (e - 5) * (1 + near)
                x[7], up[7] = 48.0, 2.0 ** (e - 6)          # 0.75 and 1 in the same binade
                xs.append(x)
                ups.append(up)
    x, up = torch.zeros(16, device="cuda"), torch.zeros(16, device="cuda")
    x[0], up[0] = 64.0, 42.0                                # 2688: g is 1
    fill = 4 - len(xs) % 4
    xs, ups = torch.cat(xs + [x] * fill)[None].to(t), torch.cat(ups + [up] * fill)[None].to(t)
    check_quantised(gpu_lib.quantize_fp4(xs, up=ups), xs.double() * ups.double(), "nvfp4")


@pytest.mark.parametrize("K", [64, 512])
def test_mxfp4_every_pair_of_scales(gpu_lib, K):
    """Ones under every pair of scales, 2^-254 to 2^254 together: sums of K equal powers of two, exact where they are normal
    numbers, infinite above, and below off by what is cut off each term."""
    r = torch.arange(255, device="cuda")
    q = torch.full((255, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    x = q, r.to(torch.uint8)[:, None].expand(255, K // 32).contiguous(), None
    y = gpu_lib.linear_fp4(x, *x, out_dtype=torch.float32).double()
    e = r[:, None] + r[None, :] - 254 + K.bit_length() - 1
    want = power(e.clamp(-300, 300))
    low = e < -126
    assert torch.equal(y[~low], torch.where(e > 127, torch.inf, want)[~low])
    assert ((y - want).abs()[low] <= K * 2.0 ** -149).all()
    none = torch.zeros_like(q), x[1], None                  # nothing but zeros, whatever their scales
    assert (gpu_lib.linear_fp4(none, *x, out_dtype=torch.float32) == 0).all()
