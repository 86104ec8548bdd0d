"""The operators around the layer at the ends of their ranges, each against a
plain implementation in 64 bits: scores of very different sizes, rows of
subnormals, far scales, side streams, captured graphs, waits that run out, and
the layer with a router of its own in its other forms."""
import math

import numpy as np
import pytest
import torch

from test_gpu_operators import DT, INF, call_w4, check_norm, check_route, check_w4, gen, make_layer, make_w4, ref_experts

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
def held_back(E, k, groups, base, step, small, seed):
    """Tokens whose picks are experts of score e^small, their biases `step` apart from `base` on, and one expert of half
    the softmax's sum that its bias holds back to among them: its score has an error in 32 bits that no other has."""
    rng, T = np.random.RandomState(seed), 64
    logits, bias = np.full((T, E), -30.0), np.full(E, -1.0)
    some = rng.permutation(E // 2 if groups > 1 else E)        # within the groups that are kept
    big, other, few = some[0], some[1], some[2:k + 4]
    logits[:, big] = (np.arange(T) - T // 2) * 2e-8            # p moves by 5e-9 from token to token
    logits[:, other] = 0.0                                     # the other half of the sum, never chosen
    logits[:, few] = small + 0.1 * rng.randn(len(few))
    logits = logits.astype(np.float32)
    p = np.exp(logits[0].astype(np.float64))
    bias[few] = base + step * (1 + rng.permutation(len(few)))
    bias[big] = base + step * (1 + rng.uniform(0, len(few))) - p[big] / p.sum()
    return torch.from_numpy(logits).cuda(), torch.from_numpy(bias.astype(np.float32)).cuda()


@pytest.mark.parametrize("E,k,groups", [(32, 2, 1), (32, 4, 4), (100, 6, 1), (256, 8, 1), (256, 8, 4), (512, 16, 8)])
@pytest.mark.parametrize("base,step,small", [(0.0, 1e-8, -20.7), (1e-3, 1.5e-9, -16.1), (0.0, 4e-8, -18.0)])
def test_route_softmax_scores_with_errors_of_other_sizes(gpu_lib, E, k, groups, base, step, small):
    for seed in range(8):
        logits, bias = held_back(E, k, groups, base, step, small, seed)
        opt = dict(score="softmax", bias=bias, n_groups=groups, topk_groups=max(1, groups // 2))
        check_route(gpu_lib.route_logits(logits, k, **opt), logits, k, **opt)
    many = logits.repeat(5, 1)                                 # the choice in a launch of its own
    check_route(gpu_lib.route_logits(many, k, **opt), many, k, **opt)


@pytest.mark.parametrize("E,k", [(64, 8), (256, 8), (455, 11)])
def test_route_softmax_biases_that_level_the_scores(gpu_lib, E, k):
    """Biases of -p and a little noise: the order turns on the noise, the errors on p."""
    rng = np.random.RandomState(E)
    for noise in (1e-6, 1e-7):
        logits = rng.randn(200, E) * 1e-7
        logits += np.where(np.arange(E) == E // 3, 6.0, rng.randn(E) * 2)
        logits = logits.astype(np.float32)
        p = np.exp(logits[0].astype(np.float64) - logits[0].max())
        bias = torch.from_numpy((rng.uniform(0, noise, E) - p / p.sum()).astype(np.float32)).cuda()
        logits = torch.from_numpy(logits).cuda()
        check_route(gpu_lib.route_logits(logits, k, bias=bias), logits, k, bias=bias)


@pytest.mark.parametrize("row", [(-59.0, -75.0, -88.0, -95.0), (-1.0, -50.0, -87.9, -88.6), (-61.0, -87.5, -100.0, -130.0),
                                 (3.0, -20.0, -87.0, -88.5), (-87.4, -88.0, -88.7, -89.0)])
def test_route_sigmoid_weights_far_below_zero(gpu_lib, row):
    """The quotients of scores that are near or past the end of fp32's range, and those scores themselves."""
    logits = torch.full((3, 40), -INF, device="cuda")
    logits[:, 5:9] = torch.tensor(row, device="cuda")
    l = np.array(row, np.float64)
    log_p = np.where(l < 0, l, 0.0) - np.log1p(np.exp(-np.abs(l)))
    rel = np.exp(log_p - log_p[0])
    for renorm, scale, want in ((True, 1.0, rel / rel.sum()), (False, 2.0 ** 100, np.exp(log_p) * 2.0 ** 100)):
        r = gpu_lib.route_logits(logits, 4, score="sigmoid", renormalise=renorm, scale=scale)
        assert r["ids"].tolist() == [[5, 6, 7, 8]] * 3
        # as check_route; a subnormal score is held in steps of 2^-149, three roundings of it
        np.testing.assert_allclose(r["w"].cpu().numpy().astype(np.float64), np.tile(want, (3, 1)), rtol=170 * 2.0 ** -24,
                                   atol=2.0 ** -147 * scale)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def check_scaled(moe, x, gain, eps, group=0):
    """check_norm's E4M3 half with the scale 1 where max|y| / 448 is no normal float."""
    out, _, scales = moe.add_rmsnorm(x, None, gain, eps=eps, out_dtype=torch.float8_e4m3fn, group=group)
    T, d = x.shape
    n, rel = group or d, 64 * 2.0 ** -24                       # rel: as in check_norm
    ms = x.double().square().mean(1, keepdim=True) + eps
    y = torch.where(ms == 0, 0.0, x.double() / ms.sqrt()) * (1.0 if gain is None else gain.double())
    want = y.view(T, d // n, n).abs().amax(2) / 448
    want = torch.where(want < 2.0 ** -126, 1.0, want)
    assert ((scales.double() - want).abs() <= want * rel).all()
    v = (y.view(T, d // n, n) / want[:, :, None]).view(T, d)
    tol = (v.abs() * (2.0 ** -4 + 2 * rel)).clamp_min(2.0 ** -10 * (1 + 1e-5))
    assert ((out.float().double() - v).abs() <= tol).all()


@pytest.mark.parametrize("d", [64, 1000, 1002, 4099, 8192, 16384])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_norm_of_rows_at_the_ends_of_the_range(gpu_lib, d, dt, e4m3):
    """Rows of subnormals, single tiny elements among zeros, rows of the largest values, an eps that leaves the range when
    it is scaled."""
    g, fi = gen(d), torch.finfo(DT[dt])
    least = fi.smallest_normal * fi.eps
    x = torch.zeros(10, d, device="cuda")
    x[0] = least
    x[1, d // 3] = least
    x[2, d - 1] = fi.smallest_normal * 16
    x[3] = torch.randint(-40, 41, (d,), generator=g, device="cuda") * least
    x[4] = torch.randn(d, generator=g, device="cuda") * fi.smallest_normal * 4
    x[5] = fi.max
    x[6, 0] = fi.max
    x[7] = torch.randn(d, generator=g, device="cuda") * fi.smallest_normal * 2.0 ** 20
    x[8] = torch.randn(d, generator=g, device="cuda") * 1e-6
    x[9, 1] = 1.0
    x = x.to(DT[dt])
    gain = (1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(DT[dt])
    for eps in (0.0, 2.0 ** -140, 1e-35, 1e34):
        if e4m3:
            check_scaled(gpu_lib, x, None, eps)
            check_scaled(gpu_lib, x, gain, eps)
            if d % 64 == 0:
                check_scaled(gpu_lib, x, gain, eps, 64)
        else:
            check_norm(gpu_lib, x, None, None, eps=eps)
            check_norm(gpu_lib, x, torch.zeros_like(x), gain, eps=eps)


# ---------------------------------------------------------------------------
# 4-bit products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 3, 12])
@pytest.mark.parametrize("fmt,group", [("nvfp4", 16), ("int4", 64)])
def test_products_that_feed_each_other(gpu_lib, fmt, group, M):
    """Short products in a row, each started before the one that writes its tokens ends: eagerly and in a replayed graph
    with changing tokens, against calls with a wait between them."""
    moe, g, n = gpu_lib, gen(52), 448
    ws = [make_w4(fmt, n, n, group, True, "bf16", g)[0] for _ in range(6)]
    if fmt == "nvfp4":
        ws = [(q, s, gs / 60) for q, s, gs in ws]
    else:
        ws = [(q, (s.float() / 60).to(s.dtype), z) for q, s, z in ws]
    wide = [make_w4(fmt, 1024, 1024, group, True, "bf16", g)[0] for _ in range(2)]
    x = torch.randn(M, n, generator=g, device="cuda").to(torch.bfloat16)
    x8 = torch.randn(M, 1024, generator=g, device="cuda").to(torch.bfloat16)
    bufs = [torch.zeros(M, n, dtype=torch.bfloat16, device="cuda") for _ in ws]
    outs = [torch.zeros(M, 1024, device="cuda") for _ in wide]

    def chain(wait):
        y = x
        for w, b in zip(ws, bufs):
            y = call_w4(moe, fmt, y, w, out=b)
            if wait:
                torch.cuda.synchronize()
        u, _, sc = moe.add_rmsnorm(x8, out_dtype=torch.float8_e4m3fn, group=128)
        for w, o in zip(wide, outs):
            if wait:
                torch.cuda.synchronize()
            call_w4(moe, fmt, u, w, x_scales=sc, bias=outs[0][0] if o is not outs[0] else None, out=o)

    def got():
        torch.cuda.synchronize()
        return [b.clone() for b in bufs + outs]

    chain(True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    for i in range(30):
        x.copy_(torch.randn(M, n, generator=gen(100 + i), device="cuda"))
        x8.copy_(torch.randn(M, 1024, generator=gen(200 + i), device="cuda"))
        chain(True)
        want = got()
        assert all(torch.isfinite(v.float()).all() for v in want)
        for run in (lambda: chain(False), graph.replay):
            for b in bufs + outs:
                b.zero_()
            run()
            for a, b in zip(got(), want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("xdt", ["bf16", "e4m3"])
def test_linear_int4_scales_far_from_one(gpu_lib, group, xdt):
    """Scales of the weights and of x whose product is no normal float, while the sums are floats."""
    g = gen(51)
    M, N, K = 5, 48, 512
    for far, wide in ((-26, -112), (-40, -105), (20, 90), (-30, 120)):      # sums of about 2^(far + wide + 7)
        (q, s, z), W = make_w4("int4", N, K, group, True, "bf16", g)
        s, W = (s.float() * 2.0 ** far).to(torch.bfloat16), W * 2.0 ** far
        x, xs = torch.randn(M, K, generator=g, device="cuda"), None
        if xdt == "bf16":
            x = (x * 2.0 ** wide).to(torch.bfloat16)
            xd = x.double()
        else:
            x, xs = (x * 64).to(torch.float8_e4m3fn), torch.full((M, K // 128), 2.0 ** (wide - 8), device="cuda")
            xd = x.double() * 2.0 ** (wide - 8)
        y = gpu_lib.linear_int4(x, q, s, z, x_scales=xs, out_dtype=torch.float32).double()
        ref, size = xd @ W.t(), xd.abs() @ W.abs().t()
        # as check_w4, and half a step of the subnormals, 2^-150, for each addition: 4 per 128 columns, 2 per part of K
        tol = size * (8 * 17 + 4 * (K // 128 + 1) + 16) * 2.0 ** -23 + ref.abs() * 2.0 ** -24
        tol += (4 * (K // 128) + 2 * 8) * 2.0 ** -150
        assert ((y - ref).abs() <= tol).all(), (far, wide)


@pytest.mark.parametrize("M,N,K", [(5, 300, 1152), (3, 39000, 512), (20, 700, 4096)])
def test_a_product_whose_waits_run_out_says_so(gpu_lib, M, N, K):
    """One tile and several per CTA, K in one part and in several: NaN in every row, a status, and the next call is right."""
    moe, g = gpu_lib, gen(53)
    w, W = make_w4("nvfp4", N, K, 16, False, None, g)
    x = torch.randn(M, K, generator=g, device="cuda").to(torch.bfloat16)
    want = check_w4(moe, "nvfp4", x, w, W).clone()
    assert moe.linear_w4_status() == moe.MOE_OK
    moe.hold_linear_w4(True)
    try:
        y = moe.linear_nvfp4(x, *w)
        assert moe.linear_w4_status() == moe.MOE_ERR_TIMEOUT
    finally:
        moe.hold_linear_w4(False)
    assert torch.isnan(y).all()
    assert moe.linear_w4_status() == moe.MOE_OK          # reading it cleared it
    assert torch.equal(moe.linear_nvfp4(x, *w), want)
    assert moe.linear_w4_status() == moe.MOE_OK


# ---------------------------------------------------------------------------
# the layer with a router of its own
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("E", [1, 2, 3, 4])
def test_route_with_its_own_router_keeps_the_expert_outputs(gpu_lib, E):
    """What the last forward left is there after a route of many tokens, too."""
    g, T = gen(61), 9728
    layer, *_ = make_layer(gpu_lib, 256, 128, E, 1, T, g)
    x = torch.randn(T, 256, generator=g, device="cuda").to(torch.bfloat16)
    layer.set_router(score="sigmoid")
    layer.forward(x)
    want = layer.expert_outputs(T).clone()
    layer.route(x)
    assert torch.equal(layer.expert_outputs(T), want)


@pytest.mark.parametrize("d,sizes", [(256, (1, 16)), (320, (3, 16, 40))])
def test_forwards_with_a_router_are_profiled(gpu_lib, d, sizes):
    g = gen(62)
    layer, *_ = make_layer(gpu_lib, d, 128, 64, 4, 64, g)
    layer.set_router(score="sigmoid")
    for T in sizes:
        x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
        layer.forward(x)
        layer.profile_begin(3)
        for _ in range(5):
            layer.forward(x)
        ms = layer.profile_end()
        # routing, gate/up, down and combine; a forward in several chunks of tokens as one
        assert ms.shape == (3, 4 if T <= 16 else 1)
        assert (ms > 0).all() and (ms < 1000).all()


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------
def all_calls(moe, g):
    """(name, call(stream) -> its results), every call that allocates some."""
    T, d, E = 40, 256, 64
    layer, *_ = make_layer(moe, d, 128, E, 4, T, g)
    small = make_layer(moe, d, 128, E, 4, 8, g)[0]
    stack = moe.MoeStack([small])
    x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
    w, _ = make_w4("nvfp4", 96, d, 16, False, None, g)
    W = torch.randn(2, 64, d, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(600, E, generator=g, device="cuda")
    return [
        ("route_logits", lambda st: list(moe.route_logits(logits, 4, stream=st).values())),
        ("add_rmsnorm", lambda st: list(moe.add_rmsnorm(x, x, out_dtype=torch.float8_e4m3fn, group=64, stream=st))),
        ("linear_nvfp4", lambda st: [moe.linear_nvfp4(x, *w, stream=st)]),
        ("rmsnorm", lambda st: [moe.rmsnorm(x, stream=st)]),
        ("quantize_nvfp4", lambda st: list(moe.quantize_nvfp4(W, stream=st))),
        ("route", lambda st: list(layer.route(x, stream=st).values())),
        ("forward", lambda st: [layer.forward(x, stream=st)]),
        ("route_records", lambda st: list(layer.route_records(T, stream=st).values())),
        ("expert_outputs", lambda st: [layer.expert_outputs(T, stream=st)]),
        ("stack", lambda st: [stack.forward(x[:4].contiguous(), stream=st)]),
    ]


def test_results_belong_to_the_stream_they_are_written_on(gpu_lib):
    """Memory that was freed on the current stream, but is still to be read there, is not what a call on another stream
    writes its results to."""
    side = torch.cuda.Stream()
    for name, call in all_calls(gpu_lib, gen(71)):
        want = [t.float().clone() for t in call(None)]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        baits = [torch.full((t.numel() * t.element_size(),), 77, dtype=torch.uint8, device="cuda")
                 for _ in range(3) for t in call(None)]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)                   # some 50 ms of the current stream
        kept = [b + 0 for b in baits]                    # reads the baits after that
        del baits
        got = call(side)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b)), name
        torch.cuda.synchronize()
        assert all((k == 77).all() for k in kept), name
        segments = {s["address"]: s for s in torch.cuda.memory_snapshot()}
        for t in got:
            seg = max(a for a in segments if a <= t.data_ptr())
            assert segments[seg]["stream"] == side.cuda_stream, name
        del got


@pytest.mark.parametrize("T", [3, 40])
def test_a_router_bias_outlives_its_use(gpu_lib, T):
    """Dropped while another stream is yet to read it, and while a captured graph is replayed."""
    g, E = gen(72), 64
    layer, *_ = make_layer(gpu_lib, 256, 128, E, 4, 64, g)
    x = torch.randn(T, 256, generator=g, device="cuda").to(torch.bfloat16)
    values = torch.randn(E, generator=g, device="cuda")
    side = torch.cuda.Stream()

    def spoil():
        """Whatever memory of the bias's size is free is written over on the current stream."""
        return [torch.full((E,), -1e3 * i, device="cuda") for i in range(64)]

    layer.set_router(score="sigmoid", bias=values)
    want = layer.forward(x).clone()
    torch.cuda.synchronize()

    # another stream
    layer.set_router(score="sigmoid", bias=values.clone())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    out = layer.forward(x, stream=side)
    layer.clear_router()
    spoil()
    torch.cuda.synchronize()
    assert torch.equal(out, want)

    # a graph
    bias = values.clone()
    layer.set_router(score="sigmoid", bias=bias)
    layer.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x)
    layer.set_router(bias=torch.zeros(E, device="cuda"))
    layer.clear_router()
    del bias
    kept = spoil()
    torch.cuda.synchronize()
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    del kept


def test_a_router_bias_is_read_not_copied(gpu_lib):
    g, E = gen(73), 64
    layer, *_ = make_layer(gpu_lib, 256, 128, E, 4, 64, g)
    x = torch.randn(5, 256, generator=g, device="cuda").to(torch.bfloat16)
    a, b = (torch.randn(E, generator=g, device="cuda") for _ in range(2))
    bias = a.clone()
    layer.set_router(score="sigmoid", bias=bias)
    first = layer.route(x)["ids"].clone()
    bias.copy_(b)
    second = layer.route(x)["ids"].clone()
    layer.set_router(score="sigmoid", bias=b)
    assert torch.equal(layer.route(x)["ids"], second) and not torch.equal(first, second)


def whole_numbers(T, d, E, g):
    """Tokens and router weights whose products and sums are exact in any order, so that the layer's logits are the
    reference's to the bit: ties and all, the choice has to be the same."""
    x = torch.randint(-2, 3, (T, d), generator=g, device="cuda").float()
    wr = torch.randint(-1, 2, (E, d), generator=g, device="cuda").float() / 16
    return x.to(torch.bfloat16), wr.to(torch.bfloat16)


@pytest.mark.parametrize("form", ["plain", "normed", "interleaved", "nvfp4"])
@pytest.mark.parametrize("opt", [dict(score="sigmoid", n_groups=8, topk_groups=3, group_rule="top2", scale=2.5),
                                 dict(score="softmax", renormalise=False), dict(score="softmax", n_groups=4, topk_groups=2)])
def test_forms_of_the_layer_with_their_own_router(gpu_lib, form, opt):
    """Normed experts, interleaved rows, 4-bit experts, a bias of the router logits; from host memory too."""
    moe, g, d, I, E, k = gpu_lib, gen(81), 512, 256, 64, 6
    _, wr = whole_numbers(1, d, E, g)
    gate, up = ((0.05 * torch.randn(E, I, d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
    down = (0.05 * torch.randn(E, d, I, generator=g, device="cuda")).to(torch.bfloat16)
    lbias = torch.randint(-8, 9, (E,), generator=g, device="cuda").float() / 8
    kw = dict(top_k=k, max_tokens=300, router_bias=lbias)
    if form == "interleaved":
        layer = moe.MoeLayer(wr, w_gate_up=torch.stack((gate, up), 2).contiguous(), w_down=down, **kw)
    elif form == "nvfp4":
        layer, _, gate, up, down = make_layer(moe, d, I, E, k, 300, g, "nvfp4")
        layer = moe.MoeLayer(wr, nvfp4=dict(zip(("q_gate", "s_gate", "g_gate", "q_up", "s_up", "g_up", "q_down", "s_down", "g_down"),
                                                layer._keep[2:])), **kw)
    else:
        layer = moe.MoeLayer(wr, w_gate=gate, w_up=up, w_down=down, expert_out_norm=form == "normed", **kw)
    bias = 0.2 * torch.randn(E, generator=g, device="cuda")
    layer.set_router(bias=bias, **opt)
    for T in (1, 8, 16, 17, 32, 33, 300):
        x, _ = whole_numbers(T, d, E, g)
        logits = (x.double() @ wr.double().t() + lbias.double()).float()
        r = layer.route(x)
        check_route(r, logits, k, bias=bias, **opt)
        y = layer.forward(x)
        left = layer.route_records(T) if T <= 16 or d % 256 == 0 else r
        for n in r:
            assert torch.equal(left[n], r[n]), n
        host = torch.empty(T, d, dtype=torch.bfloat16).pin_memory()
        layer.forward_host(x.cpu().pin_memory(), host)
        assert torch.equal(host, y.cpu())
        assert layer.device_status() == moe.MOE_OK
        ids, w = r["ids"].long(), r["w"]
        if form == "normed":
            ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
            one = torch.ones(T, 1, device="cuda")
            for j in range(k):
                e = ref_experts(x, ids[:, j:j + 1], one, gate, up, down)
                ref += w[:, j:j + 1].double() * e / (e.square().mean(1, keepdim=True) + 1e-6).sqrt()
        else:
            ref = ref_experts(x, ids, w, gate, up, down)
        err = (y.double() - ref).abs().amax(1) / ref.abs().amax(1)
        assert err.max() <= (5e-2 if form == "nvfp4" else 2e-2), (T, err.max())    # the layer's own bars


@pytest.mark.parametrize("fmt", ["bf16", "nvfp4"])
def test_a_router_that_leaves_no_expert_is_reported(gpu_lib, fmt):
    moe, g = gpu_lib, gen(82)
    layer, *_ = make_layer(moe, 256, 256, 64, 4, 300, g, fmt)
    none = torch.full((64,), -INF, device="cuda")
    for T in (1, 16, 300):
        x = torch.randn(T, 256, generator=g, device="cuda").to(torch.bfloat16)
        want = layer.forward(x).clone()
        layer.set_router(score="softmax", bias=none)
        r = layer.route(x)
        assert (r["ids"] == -1).all() and (r["counts"] == 0).all() and (r["offsets"] == 0).all()
        layer.forward(x)
        assert layer.device_status() == moe.MOE_ERR_DEVICE
        layer.clear_router()
        assert torch.equal(layer.forward(x), want) and layer.device_status() == moe.MOE_OK


FIRST_USE = """
import torch
import top_moe_expert_router_gb300 as moe
g = torch.Generator(device="cuda").manual_seed(5)
def t(*s): return torch.randn(*s, generator=g, device="cuda")
def u8(*s): return torch.randint(0, 120, s, generator=g, device="cuda", dtype=torch.uint8)
few, many = t(40, 64), t(700, 300)
x, res, bias = t(5, 1024).to(torch.bfloat16), t(5, 1024).to(torch.bfloat16), t(64)
w4 = u8(300, 512), u8(300, 64), torch.full((1,), 1e-4, device="cuda")
i4 = u8(600, 512), (t(600, 16) / 100).to(torch.float16), u8(600, 16) % 16
layer = moe.MoeLayer(t(64, 256).to(torch.bfloat16), w_gate=t(64, 128, 256).to(torch.bfloat16) / 16,
                     w_up=t(64, 128, 256).to(torch.bfloat16) / 16, w_down=t(64, 256, 128).to(torch.bfloat16) / 16, top_k=4, max_tokens=64)
xl = [t(n, 256).to(torch.bfloat16) for n in (3, 40)]
layer.set_router(score="sigmoid", bias=bias, n_groups=8, topk_groups=4, group_rule="top2")
def calls():
    n8, s, sc = moe.add_rmsnorm(x, res, out_dtype=torch.float8_e4m3fn, group=128)
    out = [n8.float(), s, sc, moe.linear_nvfp4(n8, *w4, x_scales=sc), moe.linear_int4(x, *i4)]
    for l in (few, many):
        out += moe.route_logits(l, 6, score="sigmoid").values()
    return out + [layer.forward(v) for v in xl]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = calls()
for _ in range(2):
    for h in held:
        h.zero_()
    graph.replay()
torch.cuda.synchronize()
got = [h.clone() for h in held]
for a, b in zip(got, calls(), strict=True):
    assert torch.equal(a, b)
assert layer.device_status() == moe.MOE_OK
print("same")
"""


def test_first_use_of_every_operator_inside_a_capture():
    """A process whose first call of each operator, and of a layer with a router, is a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_USE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
