"""Python binding of libmoe.so: one top-k Mixture-of-Experts layer on one
GB300 (sm_103a).

Argument marshalling only. Every step of the layer runs in the CUDA kernels
behind the C ABI declared in ``include/moe.h``; PyTorch supplies device
memory and streams. There is no fallback: if ``libmoe.so`` is missing or no
GPU is present, the calls raise.

Every call runs on ``stream``, by default the current one. What it allocates for
its results belongs to that stream, as if the call stood in a
``torch.cuda.stream(stream)`` block. Its inputs, and buffers handed to it, have to
be ready there, and to be kept until that work is done.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

import torch

from . import _build

_lib = None
_lock = threading.Lock()
HEADER = os.path.join(_build.ROOT, "include", "moe.h")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_DEVICE, MOE_ERR_TIMEOUT = range(6)
MOE_W_BF16, MOE_W_NVFP4 = 0, 1
MOE_T_BF16, MOE_T_F16, MOE_T_F32, MOE_T_E4M3 = range(4)
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1
MOE_W4_NVFP4, MOE_W4_INT4 = 0, 1
MOE_FP4_NVFP4, MOE_FP4_MXFP4 = 0, 1
MOE_DECODE_AUTO, MOE_DECODE_CUDA_CORES, MOE_DECODE_TENSOR_CORES = 0, 1, 2


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class MoeLayerDesc(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int), ("E", ctypes.c_int), ("top_k", ctypes.c_int), ("I", ctypes.c_int),
        ("max_tokens", ctypes.c_int), ("fmt", ctypes.c_int),
        ("w_router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
        ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p),
        ("q_gate", ctypes.c_void_p), ("q_up", ctypes.c_void_p), ("q_down", ctypes.c_void_p),
        ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p), ("s_down", ctypes.c_void_p),
        ("g_gate", ctypes.c_void_p), ("g_up", ctypes.c_void_p), ("g_down", ctypes.c_void_p),
        ("expert_out_norm", ctypes.c_int),
        ("gate_up_interleaved", ctypes.c_int),
    ]


class MoeRouteDesc(ctypes.Structure):
    _fields_ = [
        ("E", ctypes.c_int), ("top_k", ctypes.c_int), ("score", ctypes.c_int), ("bias", ctypes.c_void_p),
        ("n_groups", ctypes.c_int), ("topk_groups", ctypes.c_int), ("group_rule", ctypes.c_int),
        ("renormalise", ctypes.c_int), ("scale", ctypes.c_float),
    ]


class MoeNormArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("res", ctypes.c_void_p), ("gain", ctypes.c_void_p), ("sum", ctypes.c_void_p),
        ("out", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64), ("res_stride", ctypes.c_int64), ("sum_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64), ("scales_stride", ctypes.c_int64),
        ("T", ctypes.c_int), ("d", ctypes.c_int), ("group", ctypes.c_int),
        ("type", ctypes.c_int), ("out_type", ctypes.c_int), ("eps", ctypes.c_float),
    ]


class MoeW4Args(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int), ("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int), ("group", ctypes.c_int),
        ("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("s_type", ctypes.c_int), ("g", ctypes.c_void_p),
        ("z", ctypes.c_void_p), ("x", ctypes.c_void_p), ("x_type", ctypes.c_int), ("x_stride", ctypes.c_int64),
        ("x_scales", ctypes.c_void_p), ("x_scales_stride", ctypes.c_int64), ("x_group", ctypes.c_int),
        ("bias", ctypes.c_void_p), ("y", ctypes.c_void_p), ("y_type", ctypes.c_int), ("y_stride", ctypes.c_int64),
    ]


class MoeQuantizeFp4Args(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int), ("type", ctypes.c_int), ("x", ctypes.c_void_p), ("up", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64), ("up_stride", ctypes.c_int64), ("rows", ctypes.c_void_p),
        ("T", ctypes.c_int), ("R", ctypes.c_int), ("K", ctypes.c_int),
        ("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("g", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
    ]


class MoeDequantizeFp4Args(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int), ("type", ctypes.c_int), ("q", ctypes.c_void_p), ("s", ctypes.c_void_p),
        ("g", ctypes.c_void_p), ("g_rows", ctypes.c_int), ("R", ctypes.c_int), ("K", ctypes.c_int),
        ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
    ]


class MoeGroupedLinearArgs(ctypes.Structure):
    _fields_ = [
        ("type", ctypes.c_int), ("groups", ctypes.c_int), ("M", ctypes.c_int), ("N", ctypes.c_int),
        ("K", ctypes.c_int), ("offsets", ctypes.c_void_p), ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
        ("w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("y", ctypes.c_void_p), ("y_type", ctypes.c_int),
        ("y_stride", ctypes.c_int64),
    ]


class MoeLinearFp4Args(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int), ("groups", ctypes.c_int), ("M", ctypes.c_int), ("N", ctypes.c_int),
        ("K", ctypes.c_int), ("offsets", ctypes.c_void_p), ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
        ("x_type", ctypes.c_int), ("xq", ctypes.c_void_p), ("xs", ctypes.c_void_p), ("xg", ctypes.c_void_p), ("wq", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("wg", ctypes.c_void_p),
        ("wg_cols", ctypes.c_int), ("bias", ctypes.c_void_p), ("y", ctypes.c_void_p), ("y_type", ctypes.c_int),
        ("y_stride", ctypes.c_int64),
    ]


def header_functions() -> list[str]:
    """Names of the functions include/moe.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:moe_status|int|const char\s*\*)\s*(moe_\w+)\s*\(", text, flags=re.M)))


def build(force: bool = False) -> str:
    return _build.build(force=force)


def load(path: str | None = None):
    """Load libmoe.so (building it when stale) and declare the C signatures."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or _build.build()
        lib = ctypes.CDLL(path)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        st = ctypes.c_int
        sig = {
            "moe_workspace_size": ([ctypes.POINTER(MoeLayerDesc), ctypes.POINTER(ctypes.c_size_t)], st),
            "moe_layer_create": ([ctypes.POINTER(MoeLayerDesc), vp, ctypes.c_size_t, ctypes.POINTER(vp)], st),
            "moe_route": ([vp, vp, i, vp, vp, vp, vp, vp, vp, vp], st),
            "moe_forward": ([vp, vp, vp, i, vp], st),
            "moe_forward_residual": ([vp, vp, vp, vp, i, vp], st),
            "moe_forward_host": ([vp, vp, vp, i, vp], st),
            "moe_debug_expert_outputs": ([vp, vp, i, vp], st),
            "moe_debug_route_records": ([vp, i, vp, vp, vp, vp, vp, vp, vp], st),
            "moe_debug_hold_grid_barrier": ([vp, i, vp], st),
            "moe_set_decode_path": ([vp, i], st),
            "moe_rmsnorm": ([vp, vp, i, i, f, vp], st),
            "moe_quantize_nvfp4": ([vp, i, i, i, vp, vp, vp, vp], st),
            "moe_get_device_status": ([vp, vp], st),
            "moe_last_launch_count": ([vp], i),
            "moe_profile_begin": ([vp, i], st),
            "moe_profile_end": ([vp, vp, i, ctypes.POINTER(i), ctypes.POINTER(i)], st),
            "moe_layer_destroy": ([vp], st),
            "moe_forward_static_scratch": ([ctypes.POINTER(MoeLayerDesc), vp, vp, i, vp], st),
            "moe_stack_create": ([ctypes.POINTER(vp), i, ctypes.POINTER(vp)], st),
            "moe_stack_forward": ([vp, vp, vp, i, f, vp, vp], st),
            "moe_stack_forward_host": ([vp, vp, vp, i, f, vp], st),
            "moe_stack_destroy": ([vp], st),
            "moe_route_logits_workspace_size": ([ctypes.POINTER(MoeRouteDesc), i, ctypes.POINTER(ctypes.c_size_t)], st),
            "moe_route_logits": ([ctypes.POINTER(MoeRouteDesc), vp, i, ctypes.c_int64, i, vp, vp, vp, vp, vp, vp, vp,
                                  ctypes.c_size_t, vp], st),
            "moe_layer_set_router": ([vp, ctypes.POINTER(MoeRouteDesc)], st),
            "moe_add_rmsnorm": ([ctypes.POINTER(MoeNormArgs), vp], st),
            "moe_linear_w4": ([ctypes.POINTER(MoeW4Args), vp], st),
            "moe_linear_w4_status": ([vp], st),
            "moe_debug_hold_linear_w4": ([i], st),
            "moe_quantize_fp4": ([ctypes.POINTER(MoeQuantizeFp4Args), vp], st),
            "moe_quantize_fp4_workspace_size": ([ctypes.POINTER(MoeQuantizeFp4Args), ctypes.POINTER(ctypes.c_size_t)], st),
            "moe_dequantize_fp4": ([ctypes.POINTER(MoeDequantizeFp4Args), vp], st),
            "moe_grouped_linear": ([ctypes.POINTER(MoeGroupedLinearArgs), vp], st),
            "moe_linear_fp4": ([ctypes.POINTER(MoeLinearFp4Args), vp], st),
            "moe_products_status": ([vp], st),
            "moe_debug_hold_products": ([i], st),
            "moe_status_string": ([st], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def status_string(s: int) -> str:
    return load().moe_status_string(s).decode()


def _check(s: int, what: str):
    if s != MOE_OK:
        raise MoeError(s, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, device, stream):
    """A tensor for a call's result, from the memory of the stream that the call writes it on: memory of another stream
    may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("device tensors must be contiguous CUDA tensors")


class MoeLayer:
    """One MoE layer over caller-owned device weights (torch CUDA tensors).

    bf16 experts: ``w_gate``/``w_up`` [E, I, d], ``w_down`` [E, d, I] (torch.bfloat16).
    NVFP4 experts: ``nvfp4`` dict with q_gate/q_up [E, I, d/2], q_down [E, d, I/2],
    s_gate/s_up [E, I, d/16], s_down [E, d, I/16] (uint8) and g_gate/g_up/g_down [E] (fp32).
    The workspace is allocated here with torch; the library allocates nothing.
    """

    def __init__(self, w_router, *, w_gate=None, w_up=None, w_down=None, nvfp4=None, w_gate_up=None,
                 router_bias=None, top_k=8, max_tokens=16, expert_out_norm=False):
        lib = load()
        E, d = w_router.shape
        self.d, self.E, self.k, self.max_tokens = d, E, top_k, max_tokens
        desc = MoeLayerDesc()
        desc.d, desc.E, desc.top_k, desc.max_tokens = d, E, top_k, max_tokens
        desc.expert_out_norm = 1 if expert_out_norm else 0
        self._keep = [w_router, router_bias]
        desc.w_router = _ptr(w_router)
        desc.router_bias = _ptr(router_bias)
        if w_gate_up is not None:
            # [E, I, 2, d]: gate row i then up row i of each expert
            _require_cuda(w_router, w_gate_up, w_down, router_bias)
            self.I = w_gate_up.shape[1]
            desc.fmt = MOE_W_BF16
            desc.gate_up_interleaved = 1
            desc.w_gate, desc.w_up, desc.w_down = _ptr(w_gate_up), None, _ptr(w_down)
            self._keep += [w_gate_up, w_down]
        elif nvfp4 is None:
            _require_cuda(w_router, w_gate, w_up, w_down, router_bias)
            self.I = w_gate.shape[1]
            desc.fmt = MOE_W_BF16
            desc.w_gate, desc.w_up, desc.w_down = _ptr(w_gate), _ptr(w_up), _ptr(w_down)
            self._keep += [w_gate, w_up, w_down]
        else:
            _require_cuda(w_router, router_bias, *nvfp4.values())
            self.I = nvfp4["q_gate"].shape[1]
            desc.fmt = MOE_W_NVFP4
            for key, v in nvfp4.items():
                setattr(desc, key, _ptr(v))
            self._keep += list(nvfp4.values())
        desc.I = self.I
        self.fmt = desc.fmt
        size = ctypes.c_size_t(0)
        _check(lib.moe_workspace_size(ctypes.byref(desc), ctypes.byref(size)), "moe_workspace_size")
        self.workspace = torch.empty(size.value, dtype=torch.uint8, device=w_router.device)
        h = ctypes.c_void_p()
        _check(lib.moe_layer_create(ctypes.byref(desc), _ptr(self.workspace), size.value, ctypes.byref(h)),
               "moe_layer_create")
        self._h = h
        self._desc = desc
        self._router_bias = None
        self._captured_biases = []    # those that captured graphs read

    # -- calls ----------------------------------------------------------------
    _RECORDS = ("ids", "w", "counts", "offsets", "perm", "pos")

    def _records(self, T, dev, stream):
        i32 = torch.int32
        return {
            "ids": _empty((T, self.k), i32, dev, stream),
            "w": _empty((T, self.k), torch.float32, dev, stream),
            "counts": _empty(self.E, i32, dev, stream),
            "offsets": _empty(self.E + 1, i32, dev, stream),
            "perm": _empty(T * self.k, i32, dev, stream),
            "pos": _empty((T, self.k), i32, dev, stream),
        }

    def route(self, x, stream=None):
        _require_cuda(x)
        T = x.shape[0]
        out = self._records(T, x.device, stream)
        self._use_router_bias(stream)
        _check(load().moe_route(self._h, _ptr(x), T, *(_ptr(out[n]) for n in self._RECORDS), _stream(stream)),
               "moe_route")
        return out

    def route_records(self, T, stream=None):
        """The routing records the last forward (or route) of T tokens left in
        the workspace, as that path's own kernels computed them."""
        out = self._records(T, self.workspace.device, stream)
        _check(load().moe_debug_route_records(self._h, T, *(_ptr(out[n]) for n in self._RECORDS),
                                              _stream(stream)), "moe_debug_route_records")
        return out

    def set_decode_path(self, path: int):
        """MOE_DECODE_AUTO, MOE_DECODE_CUDA_CORES or MOE_DECODE_TENSOR_CORES (T <= 16)."""
        _check(load().moe_set_decode_path(self._h, int(path)), "moe_set_decode_path")

    def hold_grid_barrier(self, hold: bool, stream=None):
        """Test hook: make the decode kernel's grid barriers wait for an arrival
        that never comes (its bounded wait then runs out), or restore them."""
        _check(load().moe_debug_hold_grid_barrier(self._h, 1 if hold else 0, _stream(stream)),
               "moe_debug_hold_grid_barrier")

    def set_router(self, *, score="softmax", bias=None, n_groups=1, topk_groups=1, group_rule="max",
                   renormalise=True, scale=1.0):
        """Choose the layer's experts as ``route_logits`` does, from the layer's own
        router logits; see ``clear_router``. ``bias``: [E] fp32 CUDA tensor or None; it is
        read, not copied, so that changes to its values count from the next call on. A
        bias that is replaced or cleared stays until what has read it is done, and, where
        a graph captured a call with it, as long as the layer."""
        desc = _route_desc(self.E, self.k, score, bias, n_groups, topk_groups, group_rule, renormalise, scale)
        if bias is not None and bias.device != self.workspace.device:
            raise ValueError(f"bias: on {bias.device}, the layer on {self.workspace.device}")
        _check(load().moe_layer_set_router(self._h, MoeRouteDesc.from_buffer_copy(desc)), "moe_layer_set_router")
        self._router_bias = bias

    def clear_router(self):
        """Back to the softmax top-k."""
        _check(load().moe_layer_set_router(self._h, None), "moe_layer_set_router")
        self._router_bias = None

    def _use_router_bias(self, stream):
        """Keeps the bias, should it be dropped, for the work on `stream` that reads it."""
        bias = self._router_bias
        if bias is None:
            return
        with torch.cuda.stream(stream):             # (None: the current one)
            if not torch.cuda.is_current_stream_capturing():
                bias.record_stream(torch.cuda.current_stream())
            elif not any(b is bias for b in self._captured_biases):
                self._captured_biases.append(bias)

    def forward(self, x, out=None, res=None, stream=None):
        _require_cuda(x, out, res)
        T = x.shape[0]
        if out is None:
            out = _empty((T, self.d), torch.bfloat16, x.device, stream)
        self._use_router_bias(stream)
        if res is None:
            _check(load().moe_forward(self._h, _ptr(x), _ptr(out), T, _stream(stream)), "moe_forward")
        else:
            _check(load().moe_forward_residual(self._h, _ptr(x), _ptr(res), _ptr(out), T, _stream(stream)),
                   "moe_forward_residual")
        return out

    def forward_host(self, x_host, out_host, stream=None):
        """x_host, out_host: CPU tensors [T, d] bf16 (pinned for async copies)."""
        T = x_host.shape[0]
        self._use_router_bias(stream)
        _check(load().moe_forward_host(self._h, _ptr(x_host), _ptr(out_host), T, _stream(stream)),
               "moe_forward_host")
        return out_host

    def expert_outputs(self, T, stream=None):
        Y = _empty((T * self.k, self.d), torch.float32, self.workspace.device, stream)
        _check(load().moe_debug_expert_outputs(self._h, _ptr(Y), T, _stream(stream)), "moe_debug_expert_outputs")
        return Y

    def device_status(self, stream=None) -> int:
        return load().moe_get_device_status(self._h, _stream(stream))

    def last_launch_count(self) -> int:
        return load().moe_last_launch_count(self._h)

    def profile_begin(self, max_forwards: int):
        _check(load().moe_profile_begin(self._h, max_forwards), "moe_profile_begin")
        self._prof_max = max_forwards

    def profile_end(self, max_kernels: int = 8):
        """-> float32 array [recorded forwards, kernels] of kernel durations in ms."""
        import numpy as np
        nf, nk = ctypes.c_int(), ctypes.c_int()
        buf = np.zeros((getattr(self, "_prof_max", 1), max_kernels), np.float32)
        _check(load().moe_profile_end(self._h, buf.ctypes.data, max_kernels, ctypes.byref(nf), ctypes.byref(nk)),
               "moe_profile_end")
        return buf[:nf.value, :nk.value]

    def close(self):
        if getattr(self, "_h", None):
            load().moe_layer_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MoeStack:
    """Layers of equal shape run in one launch: x <- x + MoE_l(RMSNorm(x)) for
    each layer in order (moe_stack_forward). The stack runs on the first
    layer's workspace; keep the layers alive while the stack is used."""

    def __init__(self, layers):
        self.layers = list(layers)
        handles = (ctypes.c_void_p * len(self.layers))(*[ly._h.value for ly in self.layers])
        h = ctypes.c_void_p()
        _check(load().moe_stack_create(handles, len(self.layers), ctypes.byref(h)), "moe_stack_create")
        self._h = h
        self.d = self.layers[0].d

    def forward(self, x, out=None, eps=1e-6, layer_out=None, stream=None):
        _require_cuda(x, out, layer_out)
        T = x.shape[0]
        if out is None:
            out = _empty((T, self.d), torch.bfloat16, x.device, stream)
        _check(load().moe_stack_forward(self._h, _ptr(x), _ptr(out), T, float(eps), _ptr(layer_out),
                                        _stream(stream)), "moe_stack_forward")
        return out

    def forward_host(self, x_host, out_host, eps=1e-6, stream=None):
        """x_host, out_host: CPU tensors [T, d] bf16 (pinned for async copies)."""
        T = x_host.shape[0]
        _check(load().moe_stack_forward_host(self._h, _ptr(x_host), _ptr(out_host), T, float(eps),
                                             _stream(stream)), "moe_stack_forward_host")
        return out_host

    def close(self):
        if getattr(self, "_h", None) is not None:
            load().moe_stack_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def rmsnorm(x, eps=1e-6, out=None, stream=None):
    _require_cuda(x, out)
    T, d = x.shape
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    _check(load().moe_rmsnorm(_ptr(x), _ptr(out), T, d, eps, _stream(stream)), "moe_rmsnorm")
    return out


def quantize_nvfp4(W, stream=None):
    """W [n, rows, K] bf16 on the GPU -> (q [n, rows, K/2] u8, s [n, rows, K/16] u8, g [n] fp32)."""
    _require_cuda(W)
    n, rows, K = W.shape
    q = _empty((n, rows, K // 2), torch.uint8, W.device, stream)
    s = _empty((n, rows, K // 16), torch.uint8, W.device, stream)
    g = _empty(n, torch.float32, W.device, stream)
    _check(load().moe_quantize_nvfp4(_ptr(W), n, rows, K, _ptr(q), _ptr(s), _ptr(g), _stream(stream)),
           "moe_quantize_nvfp4")
    return q, s, g


# -- operators around the layer -------------------------------------------------
_DTYPE = {torch.bfloat16: MOE_T_BF16, torch.float16: MOE_T_F16, torch.float32: MOE_T_F32,
          torch.float8_e4m3fn: MOE_T_E4M3}
_SCORE = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_GROUP_RULE = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}


# The current stream's handle without the Stream object around it: these calls take a few microseconds on the GPU, and
# the object costs about three on the host.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None) or torch.cuda.caching_allocator_delete

# The argument structures as bytes, in a quarter of the time that a ctypes structure takes to fill.
_PACK = {MoeRouteDesc: struct.Struct("@iiiPiiiif4x"), MoeNormArgs: struct.Struct("@6P5q5if"),
         MoeW4Args: struct.Struct("@5iPPiPPPiqPqiPPiq"), MoeQuantizeFp4Args: struct.Struct("@iiPPqqPiiiPPPPN"),
         MoeDequantizeFp4Args: struct.Struct("@iiPPPiiiPq"), MoeGroupedLinearArgs: struct.Struct("@5iPPqPPPiq"),
         MoeLinearFp4Args: struct.Struct("@5iPPqi6PiPPiq")}


def _packer(cls):
    pack = _PACK[cls].pack

    def packed(*fields):
        try:
            return pack(*fields)
        except struct.error as e:
            raise ValueError(f"{cls.__name__}: {e}") from None
    return packed


_pack_route, _pack_norm, _pack_w4, _pack_quant, _pack_dequant, _pack_grouped, _pack_fp4 = (_packer(s) for s in _PACK)
_ENTRIES = ("moe_route_logits", "moe_add_rmsnorm", "moe_linear_w4", "moe_quantize_fp4", "moe_dequantize_fp4",
            "moe_grouped_linear", "moe_linear_fp4")
_entries = None


def _load_entries():
    """The C entries _ENTRIES, which take their structures as bytes."""
    global _entries
    if _entries is None:
        lib = load()
        fns = [lib[name] for name in _ENTRIES]                # objects of their own
        for fn, typed in zip(fns, (getattr(lib, name) for name in _ENTRIES)):
            fn.argtypes = [ctypes.c_char_p, *typed.argtypes[1:]]
            fn.restype = typed.restype
        _entries = fns
    return _entries


def _entry(i):
    return (_entries or _load_entries())[i]


def _addr(t):
    return 0 if t is None else t.data_ptr()


def _refuse(name, t, dtype, shape, index, what=""):
    raise ValueError(f"{name}: a {what}{dtype} tensor of shape {tuple(shape)} on cuda:{index} expected, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}")


def _whole(name, t, dtype, shape, index):
    """The address of a contiguous tensor argument, its type, shape and device checked; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(name, t, dtype, shape, index, "contiguous ")
    return t.data_ptr()


def _rows(name, t, dtype, shape, index):
    """The address of a 2-D tensor argument, its type, shape and device checked, and the elements from one row to the
    next; 0, 0 for None."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index:
        _refuse(name, t, dtype, shape, index)
    return t.data_ptr(), _row_stride(name, t)


def _row_stride(name, t):
    """Elements from one row of a 2-D tensor to the next (rows contiguous, not overlapping)."""
    if t.is_contiguous():
        return t.shape[1] or 1
    s0, s1 = t.stride()
    rows, cols = t.shape
    if s1 == 1 and s0 >= cols and rows > 1:
        return s0
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if rows > 1 and s0 < cols:
        raise ValueError(f"{name}: rows overlap")
    return s0 if rows > 1 else cols or 1


def _input(name, t, types):
    """The first argument of a call: a 2-D CUDA tensor of one of `types`. -> its device's index"""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.dtype not in types:
        raise ValueError(f"{name}: type {t.dtype} is not supported")
    return t.get_device()


def _handle(index, stream):
    """The stream's handle; None: device `index`'s current stream."""
    return _raw_stream(index) if stream is None else stream.cuda_stream


def _run(fn, index, st, args, what):
    """fn(*args, stream handle) with device `index` current."""
    if index == _device():
        s = fn(*args, st)
    else:
        with torch.cuda.device(index):
            s = fn(*args, st)
    if s != MOE_OK:
        raise MoeError(s, what)


def _route_desc(E, top_k, score, bias, n_groups, topk_groups, group_rule, renormalise, scale):
    """A moe_route_desc as bytes."""
    if score not in _SCORE or group_rule not in _GROUP_RULE:
        raise ValueError(f"score is one of {sorted(_SCORE)}, group_rule one of {sorted(_GROUP_RULE)}")
    if bias is not None and (not bias.is_cuda or bias.dtype is not torch.float32 or bias.shape != (E,)
                             or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous fp32 CUDA tensor of one value per expert")
    return _pack_route(E, top_k, _SCORE[score], _addr(bias), n_groups, topk_groups, _GROUP_RULE[group_rule],
                       1 if renormalise else 0, scale)


_FLOATS = (torch.bfloat16, torch.float16, torch.float32)
_ROUTE_RECORDS = ("ids", "w", "counts", "offsets", "perm", "pos")
_ROUTE_TYPES = (torch.int32, torch.float32, torch.int32, torch.int32, torch.int32, torch.int32)


def route_logits(logits, top_k, *, score="softmax", bias=None, n_groups=1, topk_groups=1, group_rule="max",
                 renormalise=True, scale=1.0, out=None, stream=None):
    """Routing from given logits [T, E] (bf16, f16 or fp32; moe_route_logits).

    Scores are softmax or sigmoid of the logits; ``bias`` [E] fp32 is added to them for the choice only; with
    ``n_groups`` > 1 the choice is from the ``topk_groups`` groups with the best ``group_rule`` ("max", or "top2": the
    sum of the two best). -> dict of ids, w [T, top_k], counts [E], offsets [E+1], perm [T*top_k], pos [T, top_k] as
    ``MoeLayer.route``; slots without an expert left hold id -1, weight 0, pos -1. ``out``: such a dict to write to;
    counts, offsets, perm and pos may be left out of it and are then not computed.
    """
    index = _input("logits", logits, _FLOATS)
    T, E = logits.shape
    desc = _route_desc(E, top_k, score, bias, n_groups, topk_groups, group_rule, renormalise, scale)
    if bias is not None and bias.get_device() != index:
        raise ValueError(f"bias: on {bias.device}, logits on {logits.device}")
    if out is None:
        shapes = ((T, top_k), (T, top_k), E, E + 1, T * top_k, (T, top_k))
        out = {n: _empty(shape, dtype, logits.device, stream)
               for n, dtype, shape in zip(_ROUTE_RECORDS, _ROUTE_TYPES, shapes)}
        recs = [out[n] for n in _ROUTE_RECORDS]
    else:
        recs = [out.get(n) for n in _ROUTE_RECORDS]
        if recs[0] is None or recs[1] is None:
            raise ValueError("out must hold ids and w")
        pairs = (T, top_k)
        for n, t, dtype, shape in zip(_ROUTE_RECORDS, recs, _ROUTE_TYPES,
                                      (pairs, pairs, (E,), (E + 1,), (T * top_k,), pairs)):
            if t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != index
                                  or not t.is_contiguous()):
                _refuse(n, t, dtype, shape, index, "contiguous ")
    entry = _entry(0)
    size, ws = 0, None
    st = _handle(index, stream)
    row_stride = _row_stride("logits", logits)
    if T > 256 and any(t is not None for t in recs[2:]):   # fewer tokens, or the choice alone, need none
        need = ctypes.c_size_t(0)
        _check(_lib.moe_route_logits_workspace_size(MoeRouteDesc.from_buffer_copy(desc), T, ctypes.byref(need)),
               "moe_route_logits")
        # scratch from torch's allocator on the stream the kernels run on: every stream and captured graph has its own
        # (without a tensor around it, which costs as much as the two launches)
        size = need.value
        if _raw_alloc is not None and index == _device():
            ws = _raw_alloc(size, st)                          # what the next does, without its change of device
        else:
            ws = torch.cuda.caching_allocator_alloc(size, index, st)
    try:
        _run(entry, index, st, (desc, logits.data_ptr(), _DTYPE[logits.dtype], row_stride, T,
                                *[None if t is None else t.data_ptr() for t in recs], ws, size), "moe_route_logits")
    finally:
        if ws is not None:
            torch.cuda.caching_allocator_delete(ws)
    return out


def add_rmsnorm(x, res=None, gain=None, *, eps=1e-6, out_dtype=None, group=0, sum_out=None, out=None, scales=None,
                stream=None):
    """Residual addition and RMSNorm (moe_add_rmsnorm): s = x + res, y = s / sqrt(mean(s^2) + eps) * gain.

    x, res [T, d] and gain [d] share one type (bf16, f16 or fp32); rows may lie further apart than d elements.
    ``out_dtype`` torch.float8_e4m3fn (or an ``out`` of that type) gives E4M3 with one fp32 scale per ``group`` columns
    (0: per row). -> (out, s or None without res, scales or None). ``sum_out``, ``out``, ``scales``: buffers to write
    to; sum_out and out may be x or res themselves.
    """
    index = _input("x", x, _FLOATS)
    T, d = x.shape
    dtype = x.dtype
    if out is not None:
        if out_dtype is not None and out_dtype != out.dtype:
            raise ValueError("out_dtype and out differ")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = dtype
    e4m3 = out_dtype == torch.float8_e4m3fn
    if not e4m3 and out_dtype != dtype:
        raise ValueError(f"out_dtype {out_dtype} is not supported for {dtype} inputs")
    if group < 0 or (group and (not e4m3 or d % group)):
        raise ValueError("group divides d, and needs E4M3 output")
    if out is None:
        out = _empty((T, d), out_dtype, x.device, stream)
    if e4m3:
        cols = d // (group or d) if d else 0
        if scales is None:
            scales = _empty((T, cols), torch.float32, x.device, stream)
        scales_at, scales_ld = _rows("scales", scales, torch.float32, (T, cols), index)
    elif scales is not None:
        raise ValueError("scales need E4M3 output")
    else:
        scales_at = scales_ld = 0
    if sum_out is None and res is not None:
        sum_out = _empty((T, d), dtype, x.device, stream)
    shape = (T, d)
    res_at, res_ld = _rows("res", res, dtype, shape, index)
    sum_at, sum_ld = _rows("sum_out", sum_out, dtype, shape, index)
    out_at, out_ld = _rows("out", out, out_dtype, shape, index)
    args = _pack_norm(x.data_ptr(), res_at, _whole("gain", gain, dtype, (d,), index), sum_at, out_at, scales_at,
                      _row_stride("x", x), res_ld, sum_ld, out_ld, scales_ld, T, d, group, _DTYPE[dtype],
                      _DTYPE[out_dtype], eps)
    _run(_entry(1), index, _handle(index, stream), (args,), "moe_add_rmsnorm")
    return out, sum_out, scales


def _linear_w4(fmt, x, q, s, g, z, x_scales, bias, out, out_dtype, stream):
    index = _input("x", x, (torch.bfloat16, torch.float16, torch.float8_e4m3fn))
    M, K = x.shape
    if q.dim() != 2 or s.dim() != 2:
        raise ValueError("q and s must be 2-D")
    N = q.shape[0]
    if fmt == MOE_W4_NVFP4:
        group, s_type = 16, torch.uint8
    else:
        group, s_type = K // s.shape[1] if s.shape[1] else 0, s.dtype
        if s_type not in (torch.bfloat16, torch.float16):
            raise ValueError(f"s: type {s_type} is not supported")
    if group < 1 or K % group:
        raise ValueError("s: one scale per group of columns expected")
    x_group = xs_at = xs_ld = 0
    if x.dtype == torch.float8_e4m3fn:
        if x_scales is None or x_scales.dim() != 2 or not x_scales.shape[1] or K % x_scales.shape[1]:
            raise ValueError("E4M3 x needs x_scales [M, groups]")
        cols = x_scales.shape[1]
        x_group = K // cols if cols > 1 else 0
        xs_at, xs_ld = _rows("x_scales", x_scales, torch.float32, (M, cols), index)
    elif x_scales is not None:
        raise ValueError("x_scales belong to E4M3 x")
    if out is None:
        out_dtype = out_dtype or (torch.bfloat16 if x.dtype == torch.float8_e4m3fn else x.dtype)
        out = _empty((M, N), out_dtype, x.device, stream)
    elif out_dtype is not None and out_dtype != out.dtype:
        raise ValueError("out_dtype and out differ")
    if out.dtype not in _FLOATS:
        raise ValueError(f"out: type {out.dtype} is not supported")
    out_at, out_ld = _rows("out", out, out.dtype, (M, N), index)
    args = _pack_w4(fmt, M, N, K, group, _whole("q", q, torch.uint8, (N, K // 2), index),
                    _whole("s", s, s_type, (N, K // group), index), _DTYPE.get(s_type, 0),
                    _whole("g", g, torch.float32, (1,), index), _whole("zeros", z, torch.uint8, (N, K // group), index),
                    x.data_ptr(), _DTYPE[x.dtype], _row_stride("x", x), xs_at, xs_ld, x_group,
                    _whole("bias", bias, torch.float32, (N,), index), out_at, _DTYPE[out.dtype], out_ld)
    _run(_entry(2), index, _handle(index, stream), (args,), "moe_linear_w4")
    return out


def linear_nvfp4(x, q, s, g, *, x_scales=None, bias=None, out=None, out_dtype=None, stream=None):
    """x W^T + bias for NVFP4 weights as ``quantize_nvfp4`` writes one tensor: q [N, K/2] and s [N, K/16] (uint8),
    g [1] fp32 (moe_linear_w4).

    x [M, K], M <= 64: bf16, f16, or E4M3 with x_scales [M, groups] fp32 as ``add_rmsnorm`` writes them (one group per
    row, or groups of a multiple of 128 columns). The result is bf16, f16 or fp32 (default: x's type, bf16 for E4M3).
    """
    return _linear_w4(MOE_W4_NVFP4, x, q, s, g, None, x_scales, bias, out, out_dtype, stream)


def linear_int4(x, q, s, zeros=None, *, x_scales=None, bias=None, out=None, out_dtype=None, stream=None):
    """x W^T + bias for integer codes: w = (code - zero) * scale, q [N, K/2] uint8 (low nibble first), s [N, K/group]
    bf16 or f16 with groups of 32, 64 or 128 columns, zeros [N, K/group] uint8 or None for 8 everywhere
    (moe_linear_w4). x and the result as in ``linear_nvfp4``."""
    return _linear_w4(MOE_W4_INT4, x, q, s, None, zeros, x_scales, bias, out, out_dtype, stream)


def linear_w4_status(stream=None) -> int:
    """MOE_ERR_TIMEOUT if a wait of a 4-bit product ran out on the current device since the last call (its rows are then
    NaN), else MOE_OK (moe_linear_w4_status). Waits for the stream."""
    return load().moe_linear_w4_status(_stream(stream))


def hold_linear_w4(hold: bool):
    """Test hook: make the waits of the 4-bit products run out, or restore them."""
    _check(load().moe_debug_hold_linear_w4(1 if hold else 0), "moe_debug_hold_linear_w4")


# -- 4-bit floats, and products by expert ----------------------------------------
_HALFS = (torch.bfloat16, torch.float16)
_FP4 = {"nvfp4": (MOE_FP4_NVFP4, 16), "mxfp4": (MOE_FP4_MXFP4, 32)}
_U8, _F32 = torch.uint8, torch.float32


def _fp4_fmt(q, s):
    """Codes [.., K/2] and their scales: the format, by the columns of a scale, K, and the codes' shape."""
    shape = q.shape
    if len(shape) < 2 or s.dim() != len(shape):
        raise ValueError("codes [.., K/2] and scales [.., K/16] or [.., K/32] expected")
    K, cols = 2 * shape[-1], s.shape[-1]
    if cols * 16 == K:
        return MOE_FP4_NVFP4, K, shape
    if cols * 32 == K:
        return MOE_FP4_MXFP4, K, shape
    raise ValueError("one scale per 16 (NVFP4) or 32 (MXFP4) columns expected")


# These calls take a few microseconds on the GPU, and most of their time on the host is that of looking at their
# arguments: what is usual is tested in one condition, and looked at one by one, for the message, where that fails.


def quantize_fp4(x, fmt="nvfp4", *, up=None, rows=None, out=None, stream=None):
    """Rows [T, K] (bf16 or f16) to microscaled 4-bit floats (moe_quantize_fp4) -> (q, s, g): codes [R, K/2] uint8, the
    low nibble first, and scales. ``fmt`` "nvfp4": s [R, K/16] E4M3 bytes and a power of two g [R] fp32 per row;
    "mxfp4": s [R, K/32] biased exponents, g None.

    With ``up`` [T, K] silu(x) * up is quantised. ``rows`` [R] int32 gathers: row r is that of x at rows[r], and is not
    written where rows[r] is no row of x (as in the routing's perm past its end). ``out``: (q, s, g) to write to. K is a
    multiple of 64.
    """
    index = _input("x", x, _HALFS)
    if fmt not in _FP4:
        raise ValueError(f"fmt is one of {sorted(_FP4)}")
    code, block = _FP4[fmt]
    T, K = x.shape
    if K % 64:
        raise ValueError("K must be a multiple of 64")
    R, rows_at = T, 0
    if rows is not None:
        if rows.dim() != 1:
            raise ValueError("rows must be 1-D")
        R = rows.shape[0]
        rows_at = _whole("rows", rows, torch.int32, (R,), index)
    if out is None:
        q = _empty((R, K // 2), _U8, x.device, stream)
        s = _empty((R, K // block), _U8, x.device, stream)
        g = _empty(R, torch.float32, x.device, stream) if block == 16 else None
    else:
        q, s, g = out
        if (g is None) != (block == 32):
            raise ValueError("out: g belongs to nvfp4")
        if not (q.dtype is _U8 is s.dtype and q.get_device() == index == s.get_device() and q.is_contiguous()
                and s.is_contiguous() and q.shape == (R, K // 2) and s.shape == (R, K // block)):
            _whole("q", q, _U8, (R, K // 2), index)
            _whole("s", s, _U8, (R, K // block), index)
    up_at = up_ld = 0
    if up is not None:
        up_at, up_ld = _rows("up", up, x.dtype, (T, K), index)
    values = (code, _DTYPE[x.dtype], x.data_ptr(), up_at, K if x.is_contiguous() else _row_stride("x", x), up_ld,
              rows_at, T, R, K, q.data_ptr(), s.data_ptr(), 0 if g is None else _whole("g", g, _F32, (R,), index))
    args = _pack_quant(*values, 0, 0)
    if R < 2 * T or R * K < 1 << 24:                          # (these never take scratch)
        _run1(3, index, args, stream)
        return q, s, g
    need = ctypes.c_size_t(0)
    _check(load().moe_quantize_fp4_workspace_size(MoeQuantizeFp4Args.from_buffer_copy(args), ctypes.byref(need)),
           "moe_quantize_fp4")
    if not need.value:
        _run1(3, index, args, stream)
        return q, s, g
    ws = _scratch(need.value, index, stream)
    try:
        _run1(3, index, _pack_quant(*values, ws, need.value), stream)
    finally:
        _raw_free(ws)
    return q, s, g


def dequantize_fp4(q, s, g=None, *, dtype=None, out=None, stream=None):
    """What 4-bit floats stand for (moe_dequantize_fp4): q [R, K/2] and s [R, K/16] (NVFP4, with g [R] or [1] fp32) or
    [R, K/32] (MXFP4) -> [R, K] bf16 (default), f16 or fp32."""
    index = _input("q", q, (torch.uint8,))
    code, K, (R, _) = _fp4_fmt(q, s)
    if out is None:
        out = _empty((R, K), dtype or torch.bfloat16, q.device, stream)
    elif dtype is not None and dtype != out.dtype:
        raise ValueError("dtype and out differ")
    if out.dtype not in _FLOATS:
        raise ValueError(f"out: type {out.dtype} is not supported")
    if g is not None and code == MOE_FP4_MXFP4:
        raise ValueError("g belongs to NVFP4")
    scales, per_row, g_at = s.shape[1], 0, 0
    if not (s.dtype is _U8 and s.get_device() == index and q.is_contiguous() and s.is_contiguous() and s.shape[0] == R):
        _whole("q", q, _U8, (R, K // 2), index)
        _whole("s", s, _U8, (R, scales), index)
    if g is not None:
        per_row = 1 if g.numel() != 1 else 0
        g_at = _whole("g", g, _F32, (R if per_row else 1,), index)
    out_at, out_ld = _result_rows(out, R, K, index)
    args = _pack_dequant(code, _DTYPE[out.dtype], q.data_ptr(), s.data_ptr(), g_at, per_row, R, K, out_at, out_ld)
    _run1(4, index, args, stream)
    return out


def _result_rows(out, rows, cols, index):
    """The address of a result and the elements from one of its rows to the next, its shape and device checked."""
    if out.is_contiguous() and out.get_device() == index and out.shape == (rows, cols):
        return out.data_ptr(), cols
    return _rows("out", out, out.dtype, (rows, cols), index)


def _run1(i, index, args, stream):
    """C entry i with its packed arguments on `stream` (None: the current one) of device `index`."""
    fn = (_entries or _load_entries())[i]
    st = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _device():
        status = fn(args, st)
    else:
        with torch.cuda.device(index):
            status = fn(args, st)
    if status != MOE_OK:
        raise MoeError(status, _ENTRIES[i])


def _scratch(size, index, stream):
    """The address of memory of the stream that a call's kernels run on: every stream and captured graph has its own. For
    _raw_free, once they are launched."""
    st = _raw_stream(index) if stream is None else stream.cuda_stream
    if _raw_alloc is not None and index == _device():
        return _raw_alloc(size, st)                            # what the next does, without its change of device
    return torch.cuda.caching_allocator_alloc(size, index, st)


def _offsets(offsets, E, index):
    return _whole("offsets", offsets, torch.int32, (E + 1,), index)


def grouped_linear(x, w, offsets, *, bias=None, out=None, out_dtype=None, stream=None):
    """x[r] W[e]^T + bias[e] for the rows offsets[e] <= r < offsets[e+1] of every expert e (moe_grouped_linear).

    x [M, K] and w [E, N, K] share one type (bf16 or f16), offsets [E+1] int32 on the device as ``route_logits`` gives
    them, bias [E, N] fp32 or None. The result [M, N] is bf16, f16 or fp32 (default: x's type); rows of no expert are not
    written. K and x's row stride are multiples of 8, E <= 512.
    """
    index = _input("x", x, _HALFS)
    M, K = x.shape
    if w.dim() != 3:
        raise ValueError("w must be [E, N, K]")
    E, N, w_cols = w.shape
    if out is None:
        out = _empty((M, N), out_dtype or x.dtype, x.device, stream)
    elif out_dtype is not None and out_dtype != out.dtype:
        raise ValueError("out_dtype and out differ")
    if out.dtype not in _FLOATS:
        raise ValueError(f"out: type {out.dtype} is not supported")
    out_at, out_ld = _result_rows(out, M, N, index)
    if not (w.dtype is x.dtype and w_cols == K and w.get_device() == index and w.is_contiguous()):
        _whole("w", w, x.dtype, (E, N, K), index)
    if offsets is None:
        raise ValueError("offsets are needed")
    args = _pack_grouped(_DTYPE[x.dtype], E, M, N, K, _offsets(offsets, E, index), x.data_ptr(),
                         K if x.is_contiguous() else _row_stride("x", x), w.data_ptr(),
                         0 if bias is None else _whole("bias", bias, _F32, (E, N), index), out_at, _DTYPE[out.dtype],
                         out_ld)
    _run1(5, index, args, stream)
    return out


def _linear_fp4(x, q, s, g, offsets, bias, out, out_dtype, stream):
    code, K, shape = _fp4_fmt(q, s)
    mx = code == MOE_FP4_MXFP4
    scales = K // (32 if mx else 16)
    if len(shape) != (2 if offsets is None else 3):
        raise ValueError("q must be [N, K/2], or [E, N, K/2] with offsets")
    lead = shape[:-1]
    N = lead[-1]
    E = 1 if offsets is None else lead[0]
    codes = not isinstance(x, torch.Tensor)
    if codes:
        x, xs, xg = x
        index = _input("x codes", x, (_U8,))
    else:
        xg = None
        index = _input("x", x, _HALFS)
    M, x_cols = x.shape
    if x_cols != (K // 2 if codes else K):
        raise ValueError(f"x: {K} columns expected, got {2 * x_cols if codes else x_cols}")
    if mx and (g is not None or xg is not None):
        raise ValueError("g belongs to NVFP4")
    g_at = cols = 0
    if g is not None:
        cols = 1 if g.dim() == 2 or (offsets is None and g.numel() != 1) else 0
        g_at = _whole("g", g, _F32, lead if cols else (E,), index)
    if out is None:
        out = _empty((M, N), out_dtype or (torch.bfloat16 if codes else x.dtype), x.device, stream)
    elif out_dtype is not None and out_dtype != out.dtype:
        raise ValueError("out_dtype and out differ")
    y_type = _DTYPE.get(out.dtype, MOE_T_E4M3)
    if y_type == MOE_T_E4M3:
        raise ValueError(f"out: type {out.dtype} is not supported")
    out_at, out_ld = _result_rows(out, M, N, index)
    if not (q.dtype is _U8 is s.dtype and q.get_device() == index == s.get_device() and q.is_contiguous()
            and s.is_contiguous() and s.shape[:-1] == lead):
        _whole("q", q, _U8, shape, index)
        _whole("s", s, _U8, (*lead, scales), index)
    off_at = 0 if offsets is None else _offsets(offsets, E, index)
    bias_at = 0 if bias is None else _whole("bias", bias, _F32, lead, index)
    if codes:
        if not (xs.dtype is _U8 and xs.get_device() == index and x.is_contiguous() and xs.is_contiguous()
                and xs.shape == (M, scales)):
            _whole("x codes", x, _U8, (M, K // 2), index)
            _whole("x scales", xs, _U8, (M, scales), index)
        _run1(6, index, _pack_fp4(code, E, M, N, K, off_at, 0, 0, 0, x.data_ptr(), xs.data_ptr(),
                                  0 if xg is None else _whole("x g", xg, _F32, (M,), index), q.data_ptr(), s.data_ptr(),
                                  g_at, cols, bias_at, out_at, y_type, out_ld), stream)
        return out
    x_ld = K if x.is_contiguous() else _row_stride("x", x)
    n_q, n_s = (M * K // 2 + 15) // 16 * 16, (M * scales + 15) // 16 * 16
    ws = _scratch(n_q + n_s + 4 * M + 16, index, stream)
    try:
        _run1(6, index, _pack_fp4(code, E, M, N, K, off_at, x.data_ptr(), x_ld, _DTYPE[x.dtype], ws, ws + n_q,
                                  0 if mx else ws + n_q + n_s, q.data_ptr(), s.data_ptr(), g_at, cols, bias_at, out_at,
                                  y_type, out_ld), stream)
    finally:
        _raw_free(ws)
    return out


def linear_fp4(x, q, s, g=None, *, bias=None, out=None, out_dtype=None, stream=None):
    """x W^T + bias with both operands in microscaled 4-bit floats, on the tensor cores' 4-bit path (moe_linear_fp4).

    W: q [N, K/2] and s [N, K/16] with g [1] or [N] fp32 (NVFP4, as ``quantize_nvfp4`` or ``quantize_fp4`` write them),
    or s [N, K/32] (MXFP4). x: (q, s, g) as ``quantize_fp4`` returns them, in W's format, or [M, K] in bf16 or f16, which
    is then quantised so. bias [N] fp32 or None. The result [M, N] is bf16, f16 or fp32 (default: x's type, bf16 for
    codes). K is a multiple of 64. For up to about 16 tokens ``linear_nvfp4`` is faster with the same weights, and keeps the
    tokens' 16 bits.
    """
    return _linear_fp4(x, q, s, g, None, bias, out, out_dtype, stream)


def grouped_linear_fp4(x, q, s, g, offsets, *, bias=None, out=None, out_dtype=None, stream=None):
    """``grouped_linear`` with both operands in microscaled 4-bit floats (moe_linear_fp4): q [E, N, K/2] and s
    [E, N, K/16] with g [E] or [E, N] fp32 (NVFP4), or s [E, N, K/32] and g None (MXFP4); x as in ``linear_fp4``, bias
    [E, N] fp32 or None."""
    if offsets is None:
        raise ValueError("offsets are needed")
    return _linear_fp4(x, q, s, g, offsets, bias, out, out_dtype, stream)


def products_status(stream=None) -> int:
    """MOE_ERR_TIMEOUT if a wait of ``linear_fp4``, ``grouped_linear`` or ``grouped_linear_fp4`` ran out on the current
    device since the last call (the rows concerned are then NaN), else MOE_OK (moe_products_status). Waits for the
    stream."""
    return load().moe_products_status(_stream(stream))


def hold_products(hold: int):
    """Test hook: make the waits of those products run out (1: in all CTAs, 2: in every second), or restore them (0)."""
    _check(load().moe_debug_hold_products(int(hold)), "moe_debug_hold_products")
