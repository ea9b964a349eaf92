"""The checks of the seven bound calls stand twice: in the compiled binding and,
for what it does not take, in Python. Both refuse the same arguments. (Every
wrong tensor is a view into memory of the right size.)"""

import pytest
import torch

import mixture_experts_layer_62_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
T, D, F, E, K = 6, 64, 128, 3, 2
OPTIONAL = {"stats", "s", "residual", "ds", "used", "rng"}


def tensors(dt, pad):
    p = moe.problem(T, D, F, E, K, 0.0, dt, pad_rows=pad)
    rows, t = moe.permuted_rows(p), moe.torch_dtype(p.dtype)
    z = lambda *s, t=t: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    i32, i8, f32 = torch.int32, torch.int8, torch.float32
    pos = torch.arange(T * K, dtype=i32, device=DEV).view(T, K)
    indptr = torch.tensor([0, 4, 8, 12], dtype=i32, device=DEV)
    idx = torch.tensor([0, 1], dtype=i32, device=DEV).repeat(T, 1)
    ws, st = moe.alloc_int8_workspace(p, DEV), moe.alloc_stats(E, DEV)
    row_token = torch.arange(rows, dtype=i32, device=DEV) // K
    W, V = z(E, F, D, t=i8), z(E, D, F, t=i8)
    a, b = z(E, F, t=f32), z(E, D, t=f32)
    xq, hq, s = z(rows, D, t=i8), z(rows, F, t=i8), z(rows, t=f32)
    gate, rng = z(T, K, t=f32), torch.zeros(2, dtype=torch.int64, device=DEV)
    return p, {
        "quantize_rows": dict(x=z(T, D), q=z(T, D, t=i8), scale=z(T, t=f32), used=indptr[1:2]),
        "permute_int8": dict(x=z(T, D), idx=idx, pos=pos.clone(), indptr=indptr.clone(), row_token=row_token.clone(), xq=xq,
                             xs=s, stats=st, workspace=ws),
        "expert_up_int8": dict(xq=xq, xs=s, indptr=indptr, W1=W, w1s=a, W3=W.clone(), w3s=a.clone(), h=z(rows, F),
                               workspace=ws, stats=st),
        "expert_down_int8": dict(hq=hq, hs=s, indptr=indptr, W2=V, w2s=b, o=z(rows, D), workspace=ws, stats=st),
        "combine_dropout": dict(o=z(rows, D), pos=pos, gate=gate, out=z(T, D), s=z(T, D), residual=z(T, D), rng=rng),
        "combine_backward": dict(dy=z(T, D), o=z(rows, D), pos=pos, gate=gate, dO=z(rows, D), dgate=z(T, K, t=f32),
                                 ds=z(T, D), rng=rng, **(dict(indptr=indptr, row_token=row_token) if pad else {})),
        "permute_backward": dict(dxp=z(rows, D), pos=pos, dx=z(T, D)),
    }


def call(name, p, args):
    extra = dict(prob=0.5) if "rng" in args else {}
    return getattr(moe, name)(*(() if name == "quantize_rows" else (p,)), **args, **extra)


def wrong(name, arg, t):
    """(what, a tensor that the call has to refuse)"""
    yield "type", t.view(torch.float16) if t.element_size() == 2 else t.view(torch.uint8 if t.dtype == torch.int8 else
                                                                            torch.int8 if t.dtype == torch.uint8 else
                                                                            torch.int32 if t.dtype == torch.float32 else
                                                                            torch.float32 if t.element_size() == 4 else
                                                                            torch.float64)
    yield "host", t.cpu()
    twice = torch.zeros((2 * t.numel(),), dtype=t.dtype, device=DEV)[::2]
    if t.numel() > 1:
        yield "stride", twice
        if arg != "workspace" and not (name == "quantize_rows" and arg == "x"):
            # the statistics of a product are its header alone
            keep = moe.STATS_HEADER_BYTES if arg == "stats" and name != "permute_int8" else t.numel()
            yield "short", t.view(-1)[:keep - 1]
    if arg == "used":
        yield "short", t[:0]


@pytest.mark.parametrize("bound", [True, False], ids=["binding", "python"])
@pytest.mark.parametrize("dt,pad", [("bf16", 0), ("f32", 64)])
def test_what_is_refused(bound, dt, pad, monkeypatch):
    p, calls = tensors(dt, pad)
    if not bound:
        monkeypatch.setattr(moe, "_BINDING", moe._Unbound())
    for name, args in calls.items():
        call(name, p, args)                                     # all right
        for arg in args:
            none = {**args, arg: None}
            if arg in OPTIONAL - {"rng"} and not (name == "permute_int8" and arg == "stats"):
                call(name, p, none)
            elif name == "quantize_rows" and arg in ("q", "scale"):
                call(name, p, none)                         # allocated by the call
            else:
                with pytest.raises((ValueError, moe.MoEError)):
                    call(name, p, none)
            for what, t in wrong(name, arg, args[arg]):
                with pytest.raises((ValueError, moe.MoEError)) as e:
                    call(name, p, {**args, arg: t})
                # the checks of this side speak, not the library's
                assert isinstance(e.value, ValueError) or (name, arg) == ("quantize_rows", "x"), (name, arg, what)
        short = dict(args)
        if "workspace" in short:
            short["workspace"] = short["workspace"][:-1]
            with pytest.raises(moe.MoEError):
                call(name, p, short)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt,pad", [("bf16", 0), ("f32", 64)])
def test_the_binding_leaves_each_of_them(dt, pad, monkeypatch):
    # what the binding was given before the checks in Python spoke: each was left to them (None)
    p, calls = tensors(dt, pad)
    real, seen = moe._bound(), []

    class Spy:
        def __getattr__(self, name):
            def f(*args):
                seen.append(getattr(real, name)(*args))
                return seen[-1]
            return f

    monkeypatch.setattr(moe, "_BINDING", Spy())
    for name, args in calls.items():
        del seen[:]
        call(name, p, args)
        assert seen == [moe.MOE_OK], name
        for arg in args:
            for what, t in wrong(name, arg, args[arg]):
                del seen[:]
                with pytest.raises((ValueError, moe.MoEError)):
                    call(name, p, {**args, arg: t})
                assert seen == [None], (name, arg, what)
    torch.cuda.synchronize()
