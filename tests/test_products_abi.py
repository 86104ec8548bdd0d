"""4-bit floats and the products by expert without a GPU: every argument error
is found on the host before any device work."""
import ctypes

import pytest
import torch

import top_moe_expert_router_gb300 as moe

P = 1 << 20                                    # an aligned, non-null pointer value that no call below may use
BAD, UNS, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_OK
BF16, F16, F32, E4M3 = moe.MOE_T_BF16, moe.MOE_T_F16, moe.MOE_T_F32, moe.MOE_T_E4M3


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def _with(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def _quant(**kw):
    return _with(moe.MoeQuantizeFp4Args(moe.MOE_FP4_NVFP4, BF16, P, P, 4096, 4096, P, 8, 64, 4096, P, P, P), kw)


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=2), UNS), (dict(type=F32), UNS), (dict(type=E4M3), UNS), (dict(K=4095), UNS), (dict(K=32), UNS),
    (dict(K=32832, x_stride=1 << 20, up_stride=1 << 20), UNS), (dict(K=0), BAD), (dict(T=-1), BAD), (dict(R=-1), BAD),
    (dict(rows=None), BAD),                                            # R differs from T
    (dict(x=None), BAD), (dict(q=None), BAD), (dict(s=None), BAD), (dict(g=None), BAD),
    (dict(x=P + 1), BAD), (dict(up=P + 1), BAD), (dict(rows=P + 2), BAD), (dict(q=P + 8), BAD), (dict(s=P + 2), BAD),
    (dict(g=P + 2), BAD), (dict(x_stride=4095), BAD), (dict(up_stride=4095), BAD),
])
def test_quantize_arguments_rejected(lib, kw, want):
    assert lib.moe_quantize_fp4(_quant(**kw), None) == want


def test_quantize_workspace(lib):
    """Asked for by rows that are many times the tokens alone; codes, scales in whole 16 bytes, and g of every token."""
    need = ctypes.c_size_t(7)
    size = lambda **kw: (lib.moe_quantize_fp4_workspace_size(_quant(**kw), ctypes.byref(need)), need.value)
    assert size() == (OK, 0) and size(R=1 << 20, rows=None) == (OK, 0) and size(T=1 << 19, R=1 << 20) == (OK, 0)
    assert size(R=1 << 20, T=3, K=64) == (OK, 3 * 32 + 16 + 12)
    assert size(R=1 << 20, T=3, K=64, fmt=moe.MOE_FP4_MXFP4) == (OK, 3 * 32 + 16 + 12)
    assert size(R=1 << 14, T=1 << 12, up=None) == (OK, (1 << 12) * (2048 + 256 + 4))
    assert size(T=-1)[0] == BAD and size(R=-1)[0] == BAD and size(K=0)[0] == BAD and size(K=65)[0] == UNS and size(fmt=3)[0] == UNS
    assert lib.moe_quantize_fp4_workspace_size(None, ctypes.byref(need)) == BAD
    assert lib.moe_quantize_fp4_workspace_size(_quant(), None) == BAD
    many = dict(R=1 << 20, T=3, K=64, workspace=P)
    assert lib.moe_quantize_fp4(_quant(**many, ws_bytes=123), None) == BAD
    assert lib.moe_quantize_fp4(_quant(**{**many, "workspace": P + 8}, ws_bytes=124), None) == BAD


def _dequant(**kw):
    return _with(moe.MoeDequantizeFp4Args(moe.MOE_FP4_NVFP4, BF16, P, P, P, 1, 64, 4096, P, 4096), kw)


@pytest.mark.parametrize("kw,want", [
    (dict(fmt=-1), UNS), (dict(type=E4M3), UNS), (dict(type=9), UNS), (dict(K=96), UNS), (dict(K=-64), BAD),
    (dict(R=-1), BAD), (dict(q=None), BAD), (dict(s=None), BAD), (dict(out=None), BAD), (dict(q=P + 4), BAD),
    (dict(s=P + 1), BAD), (dict(g=P + 2), BAD), (dict(out=P + 1), BAD), (dict(out_stride=4032), BAD),
])
def test_dequantize_arguments_rejected(lib, kw, want):
    assert lib.moe_dequantize_fp4(_dequant(**kw), None) == want


def _grouped(**kw):
    return _with(moe.MoeGroupedLinearArgs(BF16, 8, 64, 256, 512, P, P, 512, P, P, P, BF16, 256), kw)


def _fp4(**kw):
    return _with(moe.MoeLinearFp4Args(moe.MOE_FP4_NVFP4, 8, 64, 256, 512, P, None, 512, BF16, P, P, P, P, P, P, 0, P, P, BF16, 256), kw)


BOTH = [
    (dict(groups=0), BAD), (dict(groups=513), UNS), (dict(M=-1), BAD), (dict(M=(1 << 24) + 1), UNS), (dict(N=0), BAD),
    (dict(N=(1 << 24) + 1, groups=1, y_stride=1 << 25), UNS), (dict(groups=512, N=1 << 22, y_stride=1 << 22), UNS),
    (dict(K=0), BAD), (dict(K=500), UNS), (dict(offsets=None), BAD), (dict(offsets=P + 2), BAD), (dict(y=None), BAD),
    (dict(y=P + 1), BAD), (dict(y_type=E4M3), UNS), (dict(y_type=F32, y=P + 2), BAD), (dict(y_stride=255), BAD),
    (dict(bias=P + 2), BAD),
    (dict(groups=1, M=1 << 24, N=1 << 24, y_stride=1 << 24), UNS),      # more tiles than 31 bits count
]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(type=F32), UNS), (dict(x=None), BAD), (dict(w=None), BAD), (dict(x=P + 8), BAD), (dict(w=P + 8), BAD),
    (dict(x_stride=504), BAD), (dict(x_stride=516), BAD), (dict(K=(1 << 24) + 8, x_stride=1 << 25), UNS),
])
def test_grouped_linear_arguments_rejected(lib, kw, want):
    assert lib.moe_grouped_linear(_grouped(**kw), None) == want


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(fmt=2), UNS), (dict(K=520), UNS), (dict(K=32832), UNS), (dict(xq=None), BAD), (dict(xs=None), BAD),
    (dict(wq=None), BAD), (dict(ws=None), BAD), (dict(xq=P + 8), BAD), (dict(wq=P + 8), BAD), (dict(xs=P + 2), BAD),
    (dict(ws=P + 1), BAD), (dict(xg=P + 2), BAD), (dict(wg=P + 2), BAD),
    (dict(fmt=moe.MOE_FP4_MXFP4), BAD),                                # second scales belong to NVFP4
    (dict(x=P, x_type=F32), UNS), (dict(x=P + 1), BAD), (dict(x=P, x_stride=511), BAD), (dict(x=P, xg=None), BAD),
])
def test_linear_fp4_arguments_rejected(lib, kw, want):
    assert lib.moe_linear_fp4(_fp4(**kw), None) == want


def test_nothing_to_do(lib):
    for fn in (lib.moe_quantize_fp4, lib.moe_dequantize_fp4, lib.moe_grouped_linear, lib.moe_linear_fp4):
        assert fn(None, None) == BAD
    assert lib.moe_quantize_fp4(_quant(R=0, x=None, q=None), None) == OK
    assert lib.moe_dequantize_fp4(_dequant(R=0, q=None), None) == OK
    assert lib.moe_grouped_linear(_grouped(M=0, x=None, y=None), None) == OK
    assert lib.moe_linear_fp4(_fp4(M=0, xq=None, y=None), None) == OK


def test_bindings_refuse():
    z = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 4, dtype=torch.uint8)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: moe.quantize_fp4(z), lambda: moe.dequantize_fp4(q, s), lambda: moe.linear_fp4(z, q, s),
                 lambda: moe.grouped_linear(z, z[None], off), lambda: moe.grouped_linear_fp4(z, q[None], s[None], None, off),
                 lambda: moe.linear_fp4(z, q, s[:, :3]), lambda: moe.grouped_linear_fp4(z, q, s, None, off),
                 lambda: moe.grouped_linear_fp4(z, q[None], s[None], None, None), lambda: moe.linear_fp4(z, q[None], s[None])):
        with pytest.raises(ValueError):
            call()
