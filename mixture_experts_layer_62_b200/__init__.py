"""B200 (sm_100a) forward pass of one sparse Mixture-of-Experts layer.

A thin ctypes binding over the C ABI of ``libmoe.so`` (declared in
``include/moe.h``; some calls go through a compiled module, ``_bound``, where
it is built for this Python and this torch). The functions here only marshal
arguments: every step of the layer runs in the library's CUDA kernels. PyTorch
provides device memory and the current stream. There is no CPU fallback: importing this package
raises if the library has not been built, and every call requires CUDA
tensors.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# MOE_LIBRARY=debug selects the build with device-side bounds checks
LIB_PATH = os.path.join(_PKG_DIR, "libmoe_debug.so" if os.environ.get("MOE_LIBRARY") == "debug" else "libmoe.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_TIMEOUT = 5
MOE_ERR_BOUNDS = 6

DTYPE_F32 = 0
DTYPE_BF16 = 1
BIAS_NONE = 0
BIAS_LOGIT = 1
BIAS_PROB = 2
GATE_SELECTED = 0
GATE_FULL = 1
DROP_TOKEN = 0
DROP_SLOT = 1
MAX_E = 512
MAX_K = 16

STATS_HEADER_BYTES = 48


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("capacity_factor", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("bias_mode", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32), ("gate_mode", ctypes.c_int32),
                ("drop_order", ctypes.c_int32), ("pad_rows", ctypes.c_int32), ("train", ctypes.c_int32)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("idx", "gate", "pos", "indptr", "row_token", "logits", "xp", "h", "o", "hs", "s", "ab", "total")]


class MoEError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} (code {code})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m mixture_experts_layer_62_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(Problem)
    vp = ctypes.c_void_p
    sz = ctypes.c_size_t
    lib.moe_stats_size.argtypes = [ctypes.c_int32]
    lib.moe_stats_size.restype = sz
    lib.moe_workspace_size.argtypes = [P]
    lib.moe_workspace_size.restype = sz
    lib.moe_workspace_layout.argtypes = [P, ctypes.POINTER(WorkspaceLayout)]
    lib.moe_workspace_layout.restype = ctypes.c_int
    lib.moe_error_string.argtypes = [ctypes.c_int]
    lib.moe_error_string.restype = ctypes.c_char_p
    lib.moe_gemm_variant.argtypes = [P]
    lib.moe_gemm_variant.restype = ctypes.c_int
    lib.moe_router_variant.argtypes = [P, ctypes.c_int]
    lib.moe_router_variant.restype = ctypes.c_int
    lib.moe_set_wait_limit.argtypes = [ctypes.c_longlong]
    lib.moe_set_wait_limit.restype = ctypes.c_longlong
    lib.moe_device_sm_count.argtypes = []
    lib.moe_device_sm_count.restype = ctypes.c_int
    lib.moe_permuted_rows.argtypes = [P]
    lib.moe_permuted_rows.restype = ctypes.c_int32
    lib.moe_backward_workspace_size.argtypes = [P]
    lib.moe_backward_workspace_size.restype = sz
    f32 = ctypes.c_float
    lib.moe_backward.argtypes = [P] + [vp] * 9 + [f32, f32] + [vp] * 9 + [vp, sz, vp, sz, vp]
    lib.moe_backward.restype = ctypes.c_int
    lib.moe_bias_update.argtypes = [P, vp, f32, vp, vp]
    lib.moe_bias_update.restype = ctypes.c_int
    lib.moe_forward.argtypes = [P] + [vp] * 11 + [vp, sz, vp]
    lib.moe_forward.restype = ctypes.c_int
    lib.moe_route.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_route.restype = ctypes.c_int
    lib.moe_route_from_logits.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_route_from_logits.restype = ctypes.c_int
    lib.moe_permute.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_permute.restype = ctypes.c_int
    lib.moe_experts.argtypes = [P] + [vp] * 12 + [vp, sz, vp]
    lib.moe_experts.restype = ctypes.c_int
    lib.moe_expert_up.argtypes = [P] + [vp] * 10 + [vp, sz, vp]
    lib.moe_expert_up.restype = ctypes.c_int
    lib.moe_expert_down.argtypes = [P] + [vp] * 8 + [vp, sz, vp]
    lib.moe_expert_down.restype = ctypes.c_int
    lib.moe_combine.argtypes = [P, vp, vp, vp, vp, vp, vp]
    lib.moe_combine.restype = ctypes.c_int
    i32 = ctypes.c_int32
    lib.moe_quantize_rows.argtypes = [i32, vp, i32, i32, vp, vp, vp, vp]
    lib.moe_quantize_rows.restype = ctypes.c_int
    lib.moe_int8_workspace_size.argtypes = [P]
    lib.moe_int8_workspace_size.restype = sz
    lib.moe_int8_variant.argtypes = [P, ctypes.c_int]
    lib.moe_int8_variant.restype = ctypes.c_int
    lib.moe_permute_int8.argtypes = [P] + [vp] * 8 + [vp, sz, vp]
    lib.moe_permute_int8.restype = ctypes.c_int
    lib.moe_expert_up_int8.argtypes = [P] + [vp] * 9 + [vp, sz, vp]
    lib.moe_expert_up_int8.restype = ctypes.c_int
    lib.moe_expert_down_int8.argtypes = [P] + [vp] * 7 + [vp, sz, vp]
    lib.moe_expert_down_int8.restype = ctypes.c_int
    lib.moe_combine_dropout.argtypes = [P] + [vp] * 5 + [f32, vp, vp, vp]
    lib.moe_combine_dropout.restype = ctypes.c_int
    lib.moe_combine_backward.argtypes = [P] + [vp] * 4 + [f32] + [vp] * 7
    lib.moe_combine_backward.restype = ctypes.c_int
    lib.moe_permute_backward.argtypes = [P] + [vp] * 4
    lib.moe_permute_backward.restype = ctypes.c_int
    global _BINDING
    _BINDING = _load_binding(lib)
    return lib


# calls that csrc/binding.cpp makes, in its order
_BOUND = ("quantize_rows", "permute_int8", "expert_up_int8", "expert_down_int8", "combine_dropout", "combine_backward",
          "permute_backward")
_BINDING = None
_LIB = None


class _Unbound:
    """In the place of a binding that is not there: takes no call, so that each
    goes through the checks in this file and ctypes, the same call for some
    microseconds more of the host."""

    def __getattr__(self, name):
        if name not in _BOUND:
            raise AttributeError(name)
        return lambda *args: None


def _load_binding(lib):
    """The compiled binding, where it is built for this Python and this torch."""
    try:
        from . import _binding
    except ImportError:
        return _Unbound()
    if getattr(_binding, "torch_version", None) != torch.__version__:
        return _Unbound()       # another torch's tensors may be laid out otherwise
    _binding.attach(tuple(ctypes.cast(getattr(lib, "moe_" + n), ctypes.c_void_p).value for n in _BOUND))
    return _binding


def _bound():
    """The binding: its functions return a call's code, or None, with nothing
    done, where an argument is not as it has to be (the checks in this file
    then say which)."""
    if _BINDING is None:
        _lib()
    return _BINDING


def _lib():
    """The loaded library; raises ImportError when it has not been built."""
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


GEMM_VARIANTS = {0: "single", 1: "pair", 2: "grid_split", 3: "split_k", 4: "simt", 5: "interleaved", 6: "gemv"}


def gemm_variant(p: Problem) -> str:
    """Name of the grouped-GEMM kernel the library uses for p (moe_gemm_variant)."""
    v = int(_lib().moe_gemm_variant(ctypes.byref(p)))
    if v < 0:
        raise MoEError(-v, "moe_gemm_variant")
    return GEMM_VARIANTS[v]


ROUTER_VARIANTS = {0: "small", 1: "fused_mma", 2: "fused_fma", 3: "tensor", 4: "simt"}


def router_variant(p: Problem, forward: bool = True) -> str:
    """Name of the router the library uses for p: moe_forward's (forward=True)
    or moe_route's (moe_router_variant)."""
    v = int(_lib().moe_router_variant(ctypes.byref(p), 1 if forward else 0))
    if v < 0:
        raise MoEError(-v, "moe_router_variant")
    return ROUTER_VARIANTS[v]


def set_wait_limit(ns: int) -> int:
    """Wall-clock limit (nanoseconds) of the device-side bounded waits of the
    tensor-core kernels, process-wide; ns <= 0 restores the 2 s default.
    Returns the previous limit (moe_set_wait_limit)."""
    return int(_lib().moe_set_wait_limit(int(ns)))


def error_string(code: int) -> str:
    return _lib().moe_error_string(int(code)).decode()


def _check(rc, where):
    if rc != MOE_OK:
        raise MoEError(rc, where)


def _dtype_code(dtype) -> int:
    if dtype in (torch.bfloat16, "bf16", DTYPE_BF16):
        return DTYPE_BF16
    if dtype in (torch.float32, "f32", "fp32", DTYPE_F32):
        return DTYPE_F32
    raise ValueError(f"unsupported dtype {dtype}")


def torch_dtype(code: int):
    return torch.bfloat16 if code == DTYPE_BF16 else torch.float32


def problem(T, d, d_ff, E, k, capacity_factor=0.0, dtype="bf16", bias_mode=BIAS_NONE, d_ff_shared=0,
            gate_mode=GATE_SELECTED, drop_order=DROP_TOKEN, pad_rows=0, train=0) -> Problem:
    return Problem(int(T), int(d), int(d_ff), int(E), int(k), float(capacity_factor),
                   _dtype_code(dtype), int(bias_mode), int(d_ff_shared), int(gate_mode), int(drop_order),
                   int(pad_rows), int(train))


def permuted_rows(p: Problem) -> int:
    """Rows the permuted buffers (xp, h, o, row_token) must hold for p."""
    n = int(_lib().moe_permuted_rows(ctypes.byref(p)))
    if n == 0 and p.T * p.k > 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_permuted_rows")
    return n


def stats_size(E: int) -> int:
    return int(_lib().moe_stats_size(int(E)))


def workspace_size(p: Problem) -> int:
    n = int(_lib().moe_workspace_size(ctypes.byref(p)))
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_workspace_size")
    return n


def workspace_layout(p: Problem) -> dict:
    lay = WorkspaceLayout()
    _check(_lib().moe_workspace_layout(ctypes.byref(p), ctypes.byref(lay)), "moe_workspace_layout")
    return {n: getattr(lay, n) for n, _ in WorkspaceLayout._fields_}


def device_sm_count() -> int:
    return int(_lib().moe_device_sm_count())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the MoE library must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def alloc_workspace(p: Problem, device=None) -> torch.Tensor:
    return torch.empty(workspace_size(p), dtype=torch.uint8, device=device or "cuda")


def alloc_stats(E: int, device=None) -> torch.Tensor:
    return torch.zeros(stats_size(E), dtype=torch.uint8, device=device or "cuda")


def forward(p: Problem, x, W_r, W1, W3, W2, out, stats, workspace, bias=None,
            Ws1=None, Ws3=None, Ws2=None, stream=None):
    """out[t] = sum_j gate[t,j] FFN_{idx[t,j]}(x[t]) (+ shared FFN); see moe_forward."""
    rc = _lib().moe_forward(ctypes.byref(p), _ptr(x), _ptr(W_r), _ptr(bias), _ptr(W1), _ptr(W3), _ptr(W2),
                         _ptr(Ws1), _ptr(Ws3), _ptr(Ws2), _ptr(out), _ptr(stats), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "moe_forward")
    return out


def backward_workspace_size(p: Problem) -> int:
    n = int(_lib().moe_backward_workspace_size(ctypes.byref(p)))
    if n == 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "moe_backward_workspace_size")
    return n


def alloc_backward_workspace(p: Problem, device=None) -> torch.Tensor:
    return torch.empty(backward_workspace_size(p), dtype=torch.uint8, device=device or "cuda")


def backward(p: Problem, x, W_r, W1, W3, W2, dy, dx, dW_r, dW1, dW3, dW2, stats, workspace, bwd_workspace,
             alpha=0.0, beta=0.0, Ws1=None, Ws3=None, Ws2=None, dWs1=None, dWs3=None, dWs2=None, stream=None):
    """Gradients of <dy, y> + alpha L_aux + beta L_z after a moe_forward with
    p.train = 1 on the same workspace; see moe_backward."""
    rc = _lib().moe_backward(ctypes.byref(p), _ptr(x), _ptr(W_r), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(Ws1),
                             _ptr(Ws3), _ptr(Ws2), _ptr(dy), float(alpha), float(beta), _ptr(dx), _ptr(dW_r),
                             _ptr(dW1), _ptr(dW3), _ptr(dW2), _ptr(dWs1), _ptr(dWs3), _ptr(dWs2), _ptr(stats),
                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _ptr(bwd_workspace), bwd_workspace.numel() * bwd_workspace.element_size(),
                             _stream(stream))
    _check(rc, "moe_backward")


def bias_update(p: Problem, stats, bias, gamma, stream=None):
    """bias[e] -= gamma above the mean load, += gamma below (in place)."""
    _check(_lib().moe_bias_update(ctypes.byref(p), _ptr(stats), float(gamma), _ptr(bias), _stream(stream)),
           "moe_bias_update")


def route(p: Problem, x, W_r, idx, gate, stats, workspace, bias=None, logits=None, stream=None):
    rc = _lib().moe_route(ctypes.byref(p), _ptr(x), _ptr(W_r), _ptr(bias), _ptr(idx), _ptr(gate), _ptr(logits),
                       _ptr(stats), _ptr(workspace), workspace.numel() * workspace.element_size(),
                       _stream(stream))
    _check(rc, "moe_route")


def route_from_logits(p: Problem, logits, idx, gate, stats, workspace, bias=None, stream=None):
    rc = _lib().moe_route_from_logits(ctypes.byref(p), _ptr(logits), _ptr(bias), _ptr(idx), _ptr(gate),
                                   _ptr(stats), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream))
    _check(rc, "moe_route_from_logits")


def permute(p: Problem, x, idx, pos, indptr, row_token, xp, stats, workspace, stream=None):
    rc = _lib().moe_permute(ctypes.byref(p), _ptr(x), _ptr(idx), _ptr(pos), _ptr(indptr), _ptr(row_token),
                         _ptr(xp), _ptr(stats), _ptr(workspace), workspace.numel() * workspace.element_size(),
                         _stream(stream))
    _check(rc, "moe_permute")


def experts(p: Problem, xp, indptr, W1, W3, W2, o, workspace, x=None, Ws1=None, Ws3=None, Ws2=None,
            s=None, stats=None, stream=None):
    rc = _lib().moe_experts(ctypes.byref(p), _ptr(xp), _ptr(indptr), _ptr(W1), _ptr(W3), _ptr(W2), _ptr(x),
                         _ptr(Ws1), _ptr(Ws3), _ptr(Ws2), _ptr(o), _ptr(s), _ptr(stats), _ptr(workspace),
                         workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "moe_experts")


def expert_up(p: Problem, xp, indptr, W1, W3, h, workspace, x=None, Ws1=None, Ws3=None, hs=None,
              stats=None, stream=None):
    rc = _lib().moe_expert_up(ctypes.byref(p), _ptr(xp), _ptr(indptr), _ptr(W1), _ptr(W3), _ptr(x), _ptr(Ws1),
                              _ptr(Ws3), _ptr(h), _ptr(hs), _ptr(stats), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "moe_expert_up")


def expert_down(p: Problem, h, indptr, W2, o, workspace, hs=None, Ws2=None, s=None, stats=None, stream=None):
    rc = _lib().moe_expert_down(ctypes.byref(p), _ptr(h), _ptr(indptr), _ptr(W2), _ptr(hs), _ptr(Ws2), _ptr(o),
                                _ptr(s), _ptr(stats), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream))
    _check(rc, "moe_expert_down")


def combine(p: Problem, o, pos, gate, out, s=None, stream=None):
    rc = _lib().moe_combine(ctypes.byref(p), _ptr(o), _ptr(pos), _ptr(gate), _ptr(s), _ptr(out), _stream(stream))
    _check(rc, "moe_combine")


def permute_noalloc(p: Problem, x, idx, pos, indptr, row_token, xp, stats, stream=None):
    """moe_permute without a workspace: for callers that cannot allocate
    device memory; the library's fixed 1 MiB scratch array is used instead
    (see moe_permute_noalloc in include/moe.h for the limit and the rules)."""
    lib = _lib()
    fn = lib.moe_permute_noalloc
    if fn.restype is not ctypes.c_int:
        fn.argtypes = [ctypes.POINTER(Problem)] + [ctypes.c_void_p] * 8
        fn.restype = ctypes.c_int
    rc = fn(ctypes.byref(p), _ptr(x), _ptr(idx), _ptr(pos), _ptr(indptr), _ptr(row_token), _ptr(xp), _ptr(stats),
            _stream(stream))
    _check(rc, "moe_permute_noalloc")


# The calls below are short next to a decode step, so their arguments are
# marshalled without objects in between: plain integers for pointers and the
# stream, and one look at each tensor.

def _device(t) -> int:
    """The current device, which the tensors of a call have to be on."""
    if t is None or not t.is_cuda:
        raise ValueError("tensors passed to the MoE library must be CUDA tensors")
    return torch._C._cuda_getDevice()


def _arg(t, dtype, numel, name, dev):
    """Address of a tensor of the current device with at least numel elements
    of dtype (another type, or fewer, would be read as something else or past
    the end)."""
    if t is None:
        raise ValueError(f"{name}: expected {dtype} with at least {numel} elements, got None")
    if t.dtype is not dtype or t.numel() < numel:
        raise ValueError(f"{name}: expected {dtype} with at least {numel} elements, got {t.dtype} with {t.numel()}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: tensors passed to the MoE library must be CUDA tensors of the current device "
                         f"(cuda:{dev}), got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


def _opt(t, dtype, numel, name, dev):
    return None if t is None else _arg(t, dtype, numel, name, dev)


def _on(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_of(stream, device):
    """Context in which memory is allocated for a call on this stream (an object, a handle, or None: the current one)."""
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device))


def _rows(p: Problem) -> int:
    """permuted_rows without the call (p is checked by the library)."""
    return p.T * p.k + (p.E * (p.pad_rows - 1) if p.pad_rows > 0 else 0)


_I8, _I32, _F32, _U8 = torch.int8, torch.int32, torch.float32, torch.uint8


# ---- experts in 8-bit integers ------------------------------------------------

def int8_workspace_size(p: Problem) -> int:
    n = int(_lib().moe_int8_workspace_size(ctypes.byref(p)))
    if n == 0:
        raise MoEError(MOE_ERR_UNSUPPORTED, "moe_int8_workspace_size")
    return n


def alloc_int8_workspace(p: Problem, device=None) -> torch.Tensor:
    return torch.empty(int8_workspace_size(p), dtype=torch.uint8, device=device or "cuda")


INT8_VARIANTS = {0: "single", 1: "pair"}


def int8_variant(p: Problem, down: bool = False) -> str:
    """Name of the kernel form that the up (or down) product of p takes in 8 bits (moe_int8_variant)."""
    v = int(_lib().moe_int8_variant(ctypes.byref(p), 1 if down else 0))
    if v < 0:
        raise MoEError(-v, "moe_int8_variant")
    return INT8_VARIANTS[v]


def quantize_rows(x, q=None, scale=None, used=None, stream=None):
    """Rows of x [..., cols] in 8 bits with a scale for each row (see
    moe_quantize_rows); used: a one-element int32 tensor, the rows to take.
    Returns (q, scale), allocated here, on the stream of the call, when not given."""
    if q is None or scale is None:
        with _stream_of(stream, x.device):
            q = torch.empty(x.shape, dtype=_I8, device=x.device) if q is None else q
            scale = torch.empty(x.shape[:-1], dtype=_F32, device=x.device) if scale is None else scale
    rc = _bound().quantize_rows(x, q, scale, used, stream)
    if rc is None:
        dev = _device(x)
        dt, n, cols = x.dtype, x.numel(), x.shape[-1]
        rows = n // cols if cols else 0
        rc = _lib().moe_quantize_rows(_dtype_code(dt), _arg(x, dt, n, "x", dev), rows, cols,
                                      _opt(used, _I32, 1, "used", dev), _arg(q, _I8, n, "q", dev),
                                      _arg(scale, _F32, rows, "scale", dev), _on(stream, dev))
    if rc:
        raise MoEError(rc, "moe_quantize_rows")
    return q, scale


def permute_int8(p: Problem, x, idx, pos, indptr, row_token, xq, xs, stats, workspace, stream=None):
    """moe_permute with the token rows in 8 bits (see moe_permute_int8)."""
    rc = _bound().permute_int8(p, x, idx, pos, indptr, row_token, xq, xs, stats, workspace, stream)
    if rc is None:
        dev, T, d, E = _device(x), p.T, p.d, p.E
        rows, pairs = _rows(p), T * p.k
        rc = _lib().moe_permute_int8(
            ctypes.byref(p), _arg(x, torch_dtype(p.dtype), T * d, "x", dev), _arg(idx, _I32, pairs, "idx", dev),
            _arg(pos, _I32, pairs, "pos", dev), _arg(indptr, _I32, E + 1, "indptr", dev),
            _arg(row_token, _I32, rows, "row_token", dev), _arg(xq, _I8, rows * d, "xq", dev),
            _arg(xs, _F32, rows, "xs", dev), _arg(stats, _U8, STATS_HEADER_BYTES + 16 * E, "stats", dev),
            _arg(workspace, _U8, 0, "workspace", dev), workspace.nbytes, _on(stream, dev))
    if rc:
        raise MoEError(rc, "moe_permute_int8")


def expert_up_int8(p: Problem, xq, xs, indptr, W1, w1s, W3, w3s, h, workspace, stats=None, stream=None):
    """h = SiLU(a) b over 8-bit rows and weights with their scales; see moe_expert_up_int8."""
    rc = _bound().expert_up_int8(p, xq, xs, indptr, W1, w1s, W3, w3s, h, stats, workspace, stream)
    if rc is None:
        dev, rows, E, d, dff = _device(xq), _rows(p), p.E, p.d, p.d_ff
        n = E * dff
        rc = _lib().moe_expert_up_int8(
            ctypes.byref(p), _arg(xq, _I8, rows * d, "xq", dev), _arg(xs, _F32, rows, "xs", dev),
            _arg(indptr, _I32, E + 1, "indptr", dev), _arg(W1, _I8, n * d, "W1", dev), _arg(w1s, _F32, n, "w1s", dev),
            _arg(W3, _I8, n * d, "W3", dev), _arg(w3s, _F32, n, "w3s", dev),
            _arg(h, torch_dtype(p.dtype), rows * dff, "h", dev),
            _opt(stats, _U8, STATS_HEADER_BYTES, "stats", dev), _arg(workspace, _U8, 0, "workspace", dev),
            workspace.nbytes, _on(stream, dev))
    if rc:
        raise MoEError(rc, "moe_expert_up_int8")


def expert_down_int8(p: Problem, hq, hs, indptr, W2, w2s, o, workspace, stats=None, stream=None):
    """o = hq W2^T over 8-bit rows and weights with their scales; see moe_expert_down_int8."""
    rc = _bound().expert_down_int8(p, hq, hs, indptr, W2, w2s, o, stats, workspace, stream)
    if rc is None:
        dev, rows, E, d, dff = _device(hq), _rows(p), p.E, p.d, p.d_ff
        n = E * d
        rc = _lib().moe_expert_down_int8(
            ctypes.byref(p), _arg(hq, _I8, rows * dff, "hq", dev), _arg(hs, _F32, rows, "hs", dev),
            _arg(indptr, _I32, E + 1, "indptr", dev), _arg(W2, _I8, n * dff, "W2", dev), _arg(w2s, _F32, n, "w2s", dev),
            _arg(o, torch_dtype(p.dtype), rows * d, "o", dev), _opt(stats, _U8, STATS_HEADER_BYTES, "stats", dev),
            _arg(workspace, _U8, 0, "workspace", dev), workspace.nbytes, _on(stream, dev))
    if rc:
        raise MoEError(rc, "moe_expert_down_int8")


# ---- the way back, with dropout, residual and gradients -------------------------

def _rng(rng, dev):
    """Address of the generator's {seed, offset}: two 64-bit integers."""
    if rng is None:
        return None
    return _arg(rng, torch.uint64 if rng.dtype is torch.uint64 else torch.int64, 2, "rng", dev)


def combine_dropout(p: Problem, o, pos, gate, out, s=None, residual=None, prob=0.0, rng=None, stream=None):
    """out_t = residual_t + dropout(sum_j gate[t,j] o[pos[t,j]] (+ s_t)); rng: a
    device tensor of two 64-bit integers (seed, offset). See moe_combine_dropout."""
    rc = _bound().combine_dropout(p, o, pos, gate, s, residual, prob, rng, out, stream)
    if rc is None:
        dev, dt, n, pairs = _device(o), torch_dtype(p.dtype), p.T * p.d, p.T * p.k
        rc = _lib().moe_combine_dropout(
            ctypes.byref(p), _arg(o, dt, _rows(p) * p.d, "o", dev), _arg(pos, _I32, pairs, "pos", dev),
            _arg(gate, _F32, pairs, "gate", dev), _opt(s, dt, n, "s", dev), _opt(residual, dt, n, "residual", dev), prob,
            _rng(rng, dev), _arg(out, dt, n, "out", dev), _on(stream, dev))
    if rc:
        raise MoEError(rc, "moe_combine_dropout")
    return out


def combine_backward(p: Problem, dy, o, pos, gate, dO, dgate, ds=None, prob=0.0, rng=None, indptr=None,
                     row_token=None, stream=None):
    """Gradients of combine_dropout with the same prob and rng values:
    dO[pos] = gate u, dgate = <u, o[pos]>, ds = u with u = dropout(dy); indptr
    and row_token are needed with p.pad_rows > 0. See moe_combine_backward."""
    rc = _bound().combine_backward(p, dy, o, pos, gate, prob, rng, indptr, row_token, dO, dgate, ds, stream)
    if rc is None:
        dev, dt, n, pairs, rows = _device(dy), torch_dtype(p.dtype), p.T * p.d, p.T * p.k, _rows(p)
        ends = tokens = None
        if p.pad_rows > 0:
            ends, tokens = _opt(indptr, _I32, p.E + 1, "indptr", dev), _opt(row_token, _I32, rows, "row_token", dev)
        rc = _lib().moe_combine_backward(
            ctypes.byref(p), _arg(dy, dt, n, "dy", dev), _arg(o, dt, rows * p.d, "o", dev),
            _arg(pos, _I32, pairs, "pos", dev), _arg(gate, _F32, pairs, "gate", dev), prob, _rng(rng, dev), ends, tokens,
            _arg(dO, dt, rows * p.d, "dO", dev), _arg(dgate, _F32, pairs, "dgate", dev), _opt(ds, dt, n, "ds", dev),
            _on(stream, dev))
    if rc:
        raise MoEError(rc, "moe_combine_backward")


def permute_backward(p: Problem, dxp, pos, dx, stream=None):
    """dx_t = sum_j dxp[pos[t,j]] over the kept pairs; see moe_permute_backward."""
    rc = _bound().permute_backward(p, dxp, pos, dx, stream)
    if rc is None:
        dev, dt = _device(dxp), torch_dtype(p.dtype)
        rc = _lib().moe_permute_backward(ctypes.byref(p), _arg(dxp, dt, _rows(p) * p.d, "dxp", dev),
                                         _arg(pos, _I32, p.T * p.k, "pos", dev), _arg(dx, dt, p.T * p.d, "dx", dev),
                                         _on(stream, dev))
    if rc:
        raise MoEError(rc, "moe_permute_backward")
    return dx


@dataclass
class Stats:
    status: int
    capacity: int
    rows: int
    dropped: int
    max_count: int
    l_aux: float
    max_over_mean: float
    z_loss: float
    entropy: float
    top_gap: float
    counts: list
    kept: list
    P: list
    f: list


def read_stats(stats: torch.Tensor, E: int) -> Stats:
    """Parse a statistics block (synchronises on the copy to the host)."""
    raw = stats.detach().to("cpu")
    hdr_i = raw[:STATS_HEADER_BYTES].view(torch.int32)
    hdr_f = raw[:STATS_HEADER_BYTES].view(torch.float32)
    body = raw[STATS_HEADER_BYTES:STATS_HEADER_BYTES + 16 * E]
    ints = body[:8 * E].view(torch.int32)
    flts = body[8 * E:].view(torch.float32)
    return Stats(status=int(hdr_i[0]), capacity=int(hdr_i[1]), rows=int(hdr_i[2]), dropped=int(hdr_i[3]),
                 max_count=int(hdr_i[4]), l_aux=float(hdr_f[5]), max_over_mean=float(hdr_f[6]),
                 z_loss=float(hdr_f[7]), entropy=float(hdr_f[8]), top_gap=float(hdr_f[9]),
                 counts=ints[:E].tolist(), kept=ints[E:].tolist(), P=flts[:E].tolist(), f=flts[E:].tolist())


def workspace_view(workspace: torch.Tensor, p: Problem, name: str) -> torch.Tensor:
    """A typed view of one intermediate that moe_forward leaves in the workspace."""
    lay = workspace_layout(p)
    T, k, E, d, dff, dfs = p.T, p.k, p.E, p.d, p.d_ff, p.d_ff_shared
    dt = torch_dtype(p.dtype)
    shapes = {"idx": ((T, k), torch.int32), "gate": ((T, k), torch.float32), "pos": ((T, k), torch.int32),
              "indptr": ((E + 1,), torch.int32), "row_token": ((T * k,), torch.int32),
              "logits": ((T, E), torch.float32), "xp": ((T * k, d), dt), "h": ((T * k, dff), dt),
              "o": ((T * k, d), dt), "hs": ((T, dfs), dt), "s": ((T, d), dt)}
    shape, dtype = shapes[name]
    n = 1
    for s_ in shape:
        n *= s_
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    off = lay[name]
    return workspace[off:off + nbytes].view(dtype).view(*shape)


class MoELayer:
    """Weights of one layer plus the buffers a forward call needs.

    Allocation is done once here (by PyTorch); each call of ``__call__``
    launches the library's kernels on the current stream and allocates
    nothing.
    """

    def __init__(self, p: Problem, W_r, W1, W3, W2, bias=None, Ws1=None, Ws3=None, Ws2=None):
        self.p = p
        self.W_r, self.W1, self.W3, self.W2 = W_r, W1, W3, W2
        self.bias, self.Ws1, self.Ws3, self.Ws2 = bias, Ws1, Ws3, Ws2
        dev = W1.device
        self.workspace = alloc_workspace(p, dev)
        self.stats = alloc_stats(p.E, dev)
        self.out = torch.empty((p.T, p.d), dtype=torch_dtype(p.dtype), device=dev)

    def __call__(self, x, out=None, stream=None):
        out = self.out if out is None else out
        forward(self.p, x, self.W_r, self.W1, self.W3, self.W2, out, self.stats, self.workspace,
                bias=self.bias, Ws1=self.Ws1, Ws3=self.Ws3, Ws2=self.Ws2, stream=stream)
        return out

    def read_stats(self) -> Stats:
        return read_stats(self.stats, self.p.E)


def _aligned_bytes(shape, dtype) -> int:
    """Bytes of a tensor, rounded up to the alignment of a workspace."""
    return -(-math.prod(shape) * dtype.itemsize // 256) * 256


def _split(memory, parts):
    """Tensors of the (shape, dtype) of parts, one behind another in memory (uint8)."""
    at = 0
    for shape, dtype in parts:
        yield memory[at:at + math.prod(shape) * dtype.itemsize].view(dtype).view(shape)
        at += _aligned_bytes(shape, dtype)


class MoELayerInt8:
    """MoELayer with the experts in 8 bits: the same arguments, the router in
    the problem's type, every expert weight quantised here with a scale for
    each row (the given weights are not kept), activations quantised for each
    token on the way. A call launches, on the current stream, moe_route,
    moe_permute_int8, moe_expert_up_int8, moe_quantize_rows,
    moe_expert_down_int8 and moe_combine_dropout without dropout (and for a
    shared expert the same products with one expert over all tokens); it
    allocates nothing. Every stage resets the status word that it is given, so
    each has one of its own: read_stats() tells the first failure of a pass.

    p.train must be 0. With ``residual`` a call returns residual + layer(x).
    """

    def __init__(self, p: Problem, W_r, W1, W3, W2, bias=None, Ws1=None, Ws3=None, Ws2=None):
        if p.train:
            raise MoEError(MOE_ERR_UNSUPPORTED, "MoELayerInt8")
        self.p = p
        self.W_r, self.bias = W_r, bias
        dev, dt, T, d = W1.device, torch_dtype(p.dtype), p.T, p.d
        self.experts = Problem.from_buffer_copy(p)
        self.experts.d_ff_shared = 0
        rows = permuted_rows(self.experts)
        self.router = Problem.from_buffer_copy(self.experts)
        self.router.d_ff = 64
        new = lambda shape, t: torch.empty(shape, dtype=t, device=dev)  # noqa: E731
        self.W1, self.w1s = quantize_rows(W1)
        self.W3, self.w3s = quantize_rows(W3)
        self.W2, self.w2s = quantize_rows(W2)
        self.idx, self.gate, self.pos = new((T, p.k), _I32), new((T, p.k), _F32), new((T, p.k), _I32)
        self.indptr, self.row_token = new((p.E + 1,), _I32), new((rows,), _I32)
        self.used = self.indptr[p.E:]
        # The router's workspace has room for buffers of a whole layer, of which it uses
        # what stands before the first of them; the rows behind the router lie over the others.
        rest = (((rows, d), _I8), ((rows,), _F32), ((rows, p.d_ff), dt), ((rows, p.d_ff), _I8), ((rows,), _F32),
                ((rows, d), dt))
        need, at = workspace_size(self.router), workspace_layout(self.router)["xp"]
        memory = new((max(need, at + sum(_aligned_bytes(*part) for part in rest)),), _U8)
        self.router_workspace = memory[:need]
        self.xq, self.xs, self.h, self.hq, self.hs, self.o = _split(memory[at:], rest)
        self.out, self.stats = new((T, d), dt), alloc_stats(p.E, dev)
        # of the stages after the router: the permutation, and up, down (and the shared expert's up, down)
        self.permutation_stats = alloc_stats(p.E, dev)
        self.product_stats = torch.zeros((4 if p.d_ff_shared else 2, STATS_HEADER_BYTES), dtype=_U8, device=dev)
        self._product_stats = self.product_stats.unbind()
        self.workspace = alloc_int8_workspace(self.experts, dev)
        self.shared = None
        if p.d_ff_shared:
            f = p.d_ff_shared
            q = problem(T, d, f, 1, 1, dtype=p.dtype)
            self.shared = dict(p=q, W1=quantize_rows(Ws1), W3=quantize_rows(Ws3), W2=quantize_rows(Ws2),
                               x=(new((T, d), _I8), new((T,), _F32)), h=new((T, f), dt),
                               hq=(new((T, f), _I8), new((T,), _F32)), s=new((T, d), dt),
                               indptr=torch.tensor([0, T], dtype=_I32, device=dev),
                               workspace=alloc_int8_workspace(q, dev))

    def __call__(self, x, out=None, residual=None, stream=None):
        out = self.out if out is None else out
        p, s = self.experts, None
        route(self.router, x, self.W_r, self.idx, self.gate, self.stats, self.router_workspace, bias=self.bias,
              stream=stream)
        permute_int8(p, x, self.idx, self.pos, self.indptr, self.row_token, self.xq, self.xs, self.permutation_stats,
                     self.workspace, stream=stream)
        expert_up_int8(p, self.xq, self.xs, self.indptr, self.W1, self.w1s, self.W3, self.w3s, self.h,
                       self.workspace, stats=self._product_stats[0], stream=stream)
        quantize_rows(self.h, self.hq, self.hs, used=self.used, stream=stream)
        expert_down_int8(p, self.hq, self.hs, self.indptr, self.W2, self.w2s, self.o, self.workspace,
                         stats=self._product_stats[1], stream=stream)
        if self.shared is not None:
            g = self.shared
            s = g["s"]
            quantize_rows(x, *g["x"], stream=stream)
            expert_up_int8(g["p"], *g["x"], g["indptr"], *g["W1"], *g["W3"], g["h"], g["workspace"],
                           stats=self._product_stats[2], stream=stream)
            quantize_rows(g["h"], *g["hq"], stream=stream)
            expert_down_int8(g["p"], *g["hq"], g["indptr"], *g["W2"], s, g["workspace"], stats=self._product_stats[3],
                             stream=stream)
        combine_dropout(p, self.o, self.pos, self.gate, out, s=s, residual=residual, stream=stream)
        return out

    def read_stats(self) -> Stats:
        """The layer's statistics; the status is that of the first stage of the
        last pass that did not end with MOE_OK."""
        st = read_stats(self.stats, self.p.E)
        later = [read_stats(self.permutation_stats, self.p.E).status,
                 *self.product_stats.cpu().view(torch.int32)[:, 0].tolist()]
        st.status = next((code for code in (st.status, *later) if code != MOE_OK), MOE_OK)
        return st
