"""The operators around the layer without a GPU: every argument error is found
on the host before any device work."""
import ctypes

import pytest
import torch

import top_moe_expert_router_gb300 as moe

P = 1 << 20                                    # an aligned, non-null pointer value that no call below may use
BAD, UNS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def _route_desc(**kw):
    d = moe.MoeRouteDesc(256, 8, moe.MOE_SCORE_SIGMOID, None, 8, 4, moe.MOE_GROUP_TOP2, 1, 1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD_DESCS = [
    (dict(E=0), BAD), (dict(top_k=0), BAD), (dict(top_k=257), BAD), (dict(n_groups=0), BAD), (dict(n_groups=7), BAD),
    (dict(topk_groups=0), BAD), (dict(topk_groups=9), BAD), (dict(score=2), BAD), (dict(group_rule=-1), BAD),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(bias=P + 2), BAD),
    (dict(n_groups=256, topk_groups=4), BAD),                          # four groups of one expert for top 8
    (dict(E=1024), UNS), (dict(top_k=17), UNS), (dict(n_groups=64, topk_groups=64), UNS),
]


@pytest.mark.parametrize("kw,want", BAD_DESCS)
def test_route_descriptions_rejected(lib, kw, want):
    d = _route_desc(**kw)
    size = ctypes.c_size_t()
    assert lib.moe_route_logits_workspace_size(ctypes.byref(d), 4, ctypes.byref(size)) == want
    assert lib.moe_route_logits(ctypes.byref(d), P, moe.MOE_T_F32, 1024, 4, P, P, P, P, P, P, P, 1 << 30, None) == want


def test_route_arguments_rejected(lib):
    d = _route_desc()
    size = ctypes.c_size_t()

    def call(desc=d, logits=P, t=moe.MOE_T_F32, stride=256, T=4096, ids=P, w=P, counts=P, offsets=P, perm=P, pos=P, ws=P,
             n=1 << 30):
        return lib.moe_route_logits(ctypes.byref(desc) if desc else None, logits, t, stride, T, ids, w, counts,
                                    offsets, perm, pos, ws, n, None)

    assert lib.moe_route_logits_workspace_size(None, 4, ctypes.byref(size)) == BAD
    assert lib.moe_route_logits_workspace_size(ctypes.byref(d), 4, None) == BAD
    assert lib.moe_route_logits_workspace_size(ctypes.byref(d), -1, ctypes.byref(size)) == BAD
    assert lib.moe_route_logits_workspace_size(ctypes.byref(d), 262145, ctypes.byref(size)) == UNS
    assert lib.moe_route_logits_workspace_size(ctypes.byref(d), 0, ctypes.byref(size)) == OK
    assert lib.moe_route_logits_workspace_size(ctypes.byref(d), 4096, ctypes.byref(size)) == OK and size.value >= 1024
    assert call(desc=None) == BAD
    assert call(logits=None) == BAD and call(ids=None) == BAD and call(w=None) == BAD
    assert call(t=moe.MOE_T_E4M3) == UNS and call(t=9) == UNS
    assert call(stride=255) == BAD and call(T=-1) == BAD and call(T=262145) == UNS
    assert call(logits=P + 2) == BAD and call(ids=P + 1) == BAD and call(w=P + 2) == BAD and call(perm=P + 2) == BAD
    assert call(ws=None) == BAD and call(n=16) == BAD and call(ws=P + 2) == BAD


def test_packed_arguments_match_the_structures():
    """The bytes that the bindings pass are those of the ctypes structures, field by field."""
    for cls, pack in moe._PACK.items():
        assert pack.size == ctypes.sizeof(cls)
        vals = []
        for i, (_, ctype) in enumerate(cls._fields_):
            vals.append(i + 0.5 if ctype is ctypes.c_float else (1 << 40) + i if ctypes.sizeof(ctype) == 8 else i + 1)
        got = cls.from_buffer_copy(pack.pack(*vals))
        for (name, _), v in zip(cls._fields_, vals):
            assert getattr(got, name) == v, (cls, name)


@pytest.mark.parametrize("args", [(1 << 40, 8, "softmax", None, 1, 1, "max", True, 1.0),
                                  (64, 8.5, "softmax", None, 1, 1, "max", True, 1.0)])
def test_arguments_that_do_not_fit(args):
    with pytest.raises(ValueError):
        moe._route_desc(*args)


def test_set_router_rejects(lib):
    assert lib.moe_layer_set_router(None, ctypes.byref(_route_desc())) == BAD
    assert lib.moe_layer_set_router(None, None) == BAD


def _norm(**kw):
    a = moe.MoeNormArgs(P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 4096, 4096, 4096, 4096, 32, 4, 4096, 128, moe.MOE_T_BF16, moe.MOE_T_E4M3,
                        1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), BAD), (dict(out=None), BAD), (dict(scales=None), BAD), (dict(T=-1), BAD), (dict(d=0), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(group=96), BAD), (dict(group=-1), BAD), (dict(out_type=moe.MOE_T_BF16), BAD),     # a group without scales
    (dict(out_type=moe.MOE_T_F16, group=0), UNS), (dict(type=moe.MOE_T_E4M3), UNS), (dict(type=7), UNS),
    (dict(d=16400, group=0), UNS), (dict(d=8192, group=1), BAD), (dict(x_stride=4095), BAD), (dict(out_stride=1), BAD),
    (dict(res_stride=0), BAD), (dict(sum_stride=7), BAD), (dict(scales_stride=31), BAD),
    (dict(x=P + 1), BAD), (dict(res=P + 1), BAD), (dict(gain=P + 1), BAD), (dict(sum=P + 1), BAD),
    (dict(scales=P + 2), BAD),
    (dict(sum=5 * P), BAD), (dict(out=P), BAD), (dict(out=2 * P), BAD),                     # sum is out; codes in place
    (dict(sum=2 * P, sum_stride=4100), BAD), (dict(sum=P, x_stride=4100), BAD),             # in place, other rows
    (dict(out_type=moe.MOE_T_BF16, group=0, out=P, out_stride=4100), BAD),
])
def test_norm_arguments_rejected(lib, kw, want):
    if kw == dict(d=8192, group=1):            # 8192 groups: more than the kernel keeps
        a = _norm(d=8192, group=1, x_stride=8192, res_stride=8192, sum_stride=8192, out_stride=8192,
                  scales_stride=8192)
        want = UNS
    else:
        a = _norm(**kw)
    assert lib.moe_add_rmsnorm(ctypes.byref(a), None) == want


def test_norm_of_nothing(lib):
    assert lib.moe_add_rmsnorm(None, None) == BAD
    assert lib.moe_add_rmsnorm(ctypes.byref(_norm(T=0, x=None, out=None)), None) == OK


def _w4(**kw):
    a = moe.MoeW4Args(moe.MOE_W4_INT4, 4, 256, 1024, 128, P, P, moe.MOE_T_BF16, P, P, P, moe.MOE_T_E4M3, 1024, P, 8,
                      128, P, P, moe.MOE_T_BF16, 256)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), BAD), (dict(M=65), UNS), (dict(N=0), BAD), (dict(K=0), BAD), (dict(K=1000), UNS),
    (dict(K=65536), UNS), (dict(N=(1 << 30) + 1, y_stride=1 << 31), UNS), (dict(fmt=2), UNS), (dict(group=16), UNS), (dict(group=256), UNS), (dict(K=1056), BAD),
    (dict(fmt=moe.MOE_W4_NVFP4), UNS), (dict(fmt=moe.MOE_W4_NVFP4, group=16, g=None), BAD),
    (dict(s_type=moe.MOE_T_F32), UNS), (dict(x_type=moe.MOE_T_F32), UNS), (dict(y_type=moe.MOE_T_E4M3), UNS),
    (dict(x_group=64), UNS), (dict(x_group=384), BAD), (dict(x_group=-128), BAD), (dict(x_scales=None), BAD),
    (dict(x_scales_stride=7), BAD), (dict(x_stride=1023), BAD), (dict(y_stride=255), BAD),
    (dict(q=None), BAD), (dict(s=None), BAD), (dict(x=None), BAD), (dict(y=None), BAD),
    (dict(q=P + 8), BAD), (dict(s=P + 1), BAD), (dict(y=P + 1), BAD), (dict(x_scales=P + 2), BAD), (dict(bias=P + 2), BAD),
    (dict(x_type=moe.MOE_T_BF16, x=P + 1), BAD),
])
def test_linear_w4_arguments_rejected(lib, kw, want):
    assert lib.moe_linear_w4(ctypes.byref(_w4(**kw)), None) == want


def test_linear_w4_of_nothing(lib):
    assert lib.moe_linear_w4(None, None) == BAD
    assert lib.moe_linear_w4(ctypes.byref(_w4(M=0, x=None, y=None)), None) == OK


def test_bindings_refuse_cpu_tensors():
    with pytest.raises(ValueError):
        moe.route_logits(torch.zeros(2, 16), 2)
    with pytest.raises(ValueError):
        moe.add_rmsnorm(torch.zeros(2, 16))
    with pytest.raises(ValueError):
        moe.linear_nvfp4(torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.uint8),
                         torch.zeros(4, 2, dtype=torch.uint8), torch.ones(1))
