"""Host-side refusals of the operators beside the layer (CPU only: nothing is launched)."""

import ctypes

import pytest
import torch

import mixture_experts_layer_62_b200 as moe

BIG = 1 << 40
PTR = ctypes.c_void_p(1 << 20)      # aligned, never touched
ODD = ctypes.c_void_p((1 << 20) + 4)
WS = ctypes.c_void_p(1 << 20)
NONE = None


def call(name, p, *args):
    return getattr(moe.lib, name)(ctypes.byref(p), *args)


def with_(args, i, v):
    args = list(args)
    args[i] = v
    return args


INT8 = {  # name -> (pointer arguments, of which required to be 16-byte aligned, optional)
    "moe_permute_int8": (8, {0, 5, 7}, set()),
    "moe_expert_up_int8": (9, {0, 3, 4, 5, 6, 7}, {8}),
    "moe_expert_down_int8": (7, {0, 3, 4, 5}, {6}),
}


@pytest.mark.parametrize("name", INT8)
def test_int8_refusals(name):
    n, aligned, optional = INT8[name]
    ok = moe.problem(16, 64, 64, 4, 2)
    args = [PTR] * n
    size = moe.int8_workspace_size(ok)
    assert call(name, ok, *args, WS, size - 1, NONE) == moe.MOE_ERR_WORKSPACE
    assert call(name, ok, *args, NONE, size, NONE) == moe.MOE_ERR_WORKSPACE
    assert call(name, ok, *args, ODD, size, NONE) == moe.MOE_ERR_WORKSPACE
    for i in range(n):
        want = moe.MOE_ERR_WORKSPACE if i in optional else moe.MOE_ERR_INVALID_ARG
        assert call(name, ok, *with_(args, i, NONE), NONE, 0, NONE) == want
        if i in aligned:
            assert call(name, ok, *with_(args, i, ODD), NONE, 0, NONE) == moe.MOE_ERR_INVALID_ARG
    for bad in (moe.problem(16, 72, 64, 4, 2, dtype="f32"), moe.problem(16, 64, 72, 4, 2, dtype="f32"),
                moe.problem(16, 64, 64, 4, 2, d_ff_shared=64), moe.problem(16, 131072, 64, 4, 2),
                moe.problem(16, 64, 131072, 4, 2)):
        assert call(name, bad, *args, WS, BIG, NONE) == moe.MOE_ERR_UNSUPPORTED
        assert moe.lib.moe_int8_workspace_size(ctypes.byref(bad)) == 0
        with pytest.raises(moe.MoEError):
            moe.int8_workspace_size(bad)
    assert call(name, moe.problem(16, 64, 64, 4, 5), *args, WS, BIG, NONE) == moe.MOE_ERR_INVALID_ARG


def test_quantize_rows_refusals():
    f = moe.lib.moe_quantize_rows
    assert f(7, PTR, 4, 32, NONE, PTR, PTR, NONE) == moe.MOE_ERR_INVALID_ARG
    assert f(1, PTR, -1, 32, NONE, PTR, PTR, NONE) == moe.MOE_ERR_INVALID_ARG
    assert f(1, PTR, 4, 0, NONE, PTR, PTR, NONE) == moe.MOE_ERR_INVALID_ARG
    assert f(1, PTR, 4, 24, NONE, PTR, PTR, NONE) == moe.MOE_ERR_UNSUPPORTED
    for i in (1, 5, 6):
        args = [1, PTR, 4, 32, NONE, PTR, PTR, NONE]
        assert f(*with_(args, i, NONE)) == moe.MOE_ERR_INVALID_ARG
        if i != 6:
            assert f(*with_(args, i, ODD)) == moe.MOE_ERR_INVALID_ARG
    assert f(1, NONE, 0, 32, NONE, NONE, NONE, NONE) == moe.MOE_OK      # no rows


def dropout_args(prob, rng):
    return [PTR] * 3 + [NONE, NONE, ctypes.c_float(prob), rng, PTR, NONE]


def test_combine_dropout_refusals():
    p = moe.problem(16, 64, 64, 4, 2)
    args = dropout_args(0.0, NONE)
    for i in (0, 1, 2, 7):
        assert call("moe_combine_dropout", p, *with_(args, i, NONE)) == moe.MOE_ERR_INVALID_ARG
    for i in (0, 3, 4, 7):
        assert call("moe_combine_dropout", p, *with_(args, i, ODD)) == moe.MOE_ERR_INVALID_ARG
    for prob in (-0.1, 1.0, 2.0, float("nan"), float("inf"), 1 - 2.0 ** -18):
        assert call("moe_combine_dropout", p, *dropout_args(prob, PTR)) == moe.MOE_ERR_INVALID_ARG
    assert call("moe_combine_dropout", p, *dropout_args(0.5, NONE)) == moe.MOE_ERR_INVALID_ARG
    assert call("moe_combine_dropout", p, *dropout_args(0.5, ODD)) == moe.MOE_ERR_INVALID_ARG
    assert call("moe_combine_dropout", moe.problem(0, 64, 64, 4, 2), *dropout_args(0.5, PTR)) == moe.MOE_OK


def test_gradient_refusals():
    p = moe.problem(16, 64, 64, 4, 2)
    args = [PTR] * 4 + [ctypes.c_float(0.0), NONE, NONE, NONE, PTR, PTR, NONE, NONE]
    for i in (0, 1, 2, 3, 8, 9):
        assert call("moe_combine_backward", p, *with_(args, i, NONE)) == moe.MOE_ERR_INVALID_ARG
    for i in (0, 1, 8, 10):
        assert call("moe_combine_backward", p, *with_(args, i, ODD)) == moe.MOE_ERR_INVALID_ARG
    padded = moe.problem(16, 64, 64, 4, 2, pad_rows=64)
    for i in (6, 7):
        full = with_(with_(args, 6, PTR), 7, PTR)
        assert call("moe_combine_backward", padded, *with_(full, i, NONE)) == moe.MOE_ERR_INVALID_ARG
    args = [PTR] * 3 + [NONE]
    for i in (0, 1, 2):
        assert call("moe_permute_backward", p, *with_(args, i, NONE)) == moe.MOE_ERR_INVALID_ARG
    for i in (0, 2):
        assert call("moe_permute_backward", p, *with_(args, i, ODD)) == moe.MOE_ERR_INVALID_ARG


class FakeCuda:
    """What the binding asks of a tensor, without a GPU."""

    def __init__(self, dtype, n, dev=0, contiguous=True):
        self.dtype, self.n, self.dev, self.c = dtype, n, dev, contiguous
        self.device, self.is_cuda, self.nbytes = f"cuda:{dev}", True, n

    def numel(self):
        return self.n

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.c

    def data_ptr(self):
        return 1 << 20


def test_binding_refuses_what_it_can_see(monkeypatch):
    p = moe.problem(4, 64, 64, 2, 1)
    cpu = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: moe.quantize_rows(cpu), lambda: moe.combine_dropout(p, cpu, cpu, cpu, cpu),
                 lambda: moe.permute_backward(p, cpu, cpu, cpu),
                 lambda: moe.expert_down_int8(p, cpu, cpu, cpu, cpu, cpu, cpu, cpu)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    bf, i32, f32, i8, u8 = torch.bfloat16, torch.int32, torch.float32, torch.int8, torch.uint8
    good = [FakeCuda(i8, 256), FakeCuda(f32, 4), FakeCuda(i32, 3), FakeCuda(i8, 8192), FakeCuda(f32, 128),
            FakeCuda(bf, 256), FakeCuda(u8, 1 << 30)]
    for i in range(7):
        for bad in (FakeCuda(torch.float64, 1 << 30), FakeCuda(good[i].dtype, good[i].n, dev=1),
                    FakeCuda(good[i].dtype, good[i].n, contiguous=False)) + \
                (() if i == 6 else (FakeCuda(good[i].dtype, good[i].n - 1),)):
            with pytest.raises(ValueError):
                moe.expert_down_int8(p, *with_(good, i, bad))
    with pytest.raises(ValueError, match="rng"):
        moe.combine_dropout(p, FakeCuda(bf, 256), FakeCuda(i32, 4), FakeCuda(f32, 4), FakeCuda(bf, 256), prob=0.5,
                            rng=FakeCuda(f32, 2))


def test_binding_leaves_what_it_does_not_take():
    # None: nothing was called, the checks in Python say what is wrong
    b = moe._bound()
    p = moe.problem(4, 64, 64, 2, 1)
    host = torch.zeros((4, 64), dtype=torch.bfloat16)
    ghost = torch.empty((4, 64), dtype=torch.bfloat16, device="meta")
    q, s = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    for x in (host, ghost, None, 3, "x", host.to(torch.float16), host[:, :0], torch.zeros(())):
        assert b.quantize_rows(x, q, s, None, None) is None
        assert b.permute_backward(p, x, s, x, None) is None
    for wrong in (None, 5, b"short", object()):
        assert b.permute_backward(wrong, host, s, host, None) is None
        assert b.expert_down_int8(wrong, q, s, s, q, s, host, None, s, None) is None
    assert b.combine_dropout(p, host, s, s, None, None, "a number", None, host, object()) is None
    with pytest.raises(TypeError):
        b.permute_backward(p)
    with pytest.raises(ValueError):
        b.attach((1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        moe.quantize_rows(host, q, s)
    with pytest.raises(ValueError, match="CUDA"):
        moe.permute_backward(p, host, s, host)
