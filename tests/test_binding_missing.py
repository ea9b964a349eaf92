"""The compiled binding saves time of the host and nothing depends on it: without
it, or with one compiled against another torch, the same calls go through
ctypes. (CPU: what is refused; GPU: the same bits.)"""

import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_layer_62_b200 as moe
from mixture_experts_layer_62_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIDE = {
    "missing": "sys.modules['mixture_experts_layer_62_b200._binding'] = None",
    "other torch": "torch.__version__ = '0.0.0'",
}
USE = """
import mixture_experts_layer_62_b200 as moe
p = moe.problem(16, 64, 64, 4, 2)
assert moe.workspace_size(p) > 0 and moe.int8_workspace_size(p) > 0 and moe.int8_variant(p) == "single"
x = torch.zeros((16, 64), dtype=torch.bfloat16)
for call in (lambda: moe.quantize_rows(x), lambda: moe.permute_backward(p, x, x, x), lambda: moe.combine_dropout(p, x, x, x, x)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e)
    else:
        raise AssertionError("not refused")
assert type(moe._bound()).__name__ == "_Unbound"
"""


@pytest.mark.parametrize("how", HIDE)
def test_the_package_works_without_its_binding(how):
    code = f"import sys\nimport torch\nsys.path.insert(0, {ROOT!r})\n{HIDE[how]}\n{USE}"
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_the_binding_is_this_torchs():
    assert moe._bound().torch_version == torch.__version__
    with pytest.raises(AttributeError):
        moe._Unbound().no_such_call


def test_the_binding_is_compiled_again_for_another_torch(tmp_path, monkeypatch):
    module, stamp = tmp_path / "binding.so", tmp_path / "binding.torch"
    monkeypatch.setattr(build, "BINDING_PATH", str(module))
    monkeypatch.setattr(build, "BINDING_STAMP", str(stamp))
    assert build._binding_stale()               # nothing there
    module.write_bytes(b"")
    assert build._binding_stale()               # compiled against nobody knows what
    stamp.write_text(build._torch_stamp())
    assert not build._binding_stale()
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build._binding_stale()


@pytest.mark.gpu
def test_the_same_bits_without_the_binding(monkeypatch):
    T, d, dff, E, k = 200, 256, 320, 8, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    n = lambda *s: (torch.randn(s, generator=g, device="cuda") / 16).to(torch.bfloat16)  # noqa: E731
    w = dict(W_r=n(d, E), W1=n(E, dff, d), W3=n(E, dff, d), W2=n(E, d, dff), Ws1=n(dff, d), Ws3=n(dff, d), Ws2=n(d, dff))
    x, dy, rng = n(T, d) * 16, n(T, d), torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    p = moe.problem(T, d, dff, E, k, 0.9, d_ff_shared=dff, pad_rows=64)

    def everything():
        layer = moe.MoELayerInt8(p, **w)
        y = layer(x, residual=x).clone()
        q = layer.experts
        out, dO = torch.zeros_like(y), torch.zeros_like(layer.o)
        dgate, ds, dx = torch.zeros_like(layer.gate), torch.zeros_like(y), torch.zeros_like(y)
        moe.combine_dropout(q, layer.o, layer.pos, layer.gate, out, residual=x, prob=0.3, rng=rng)
        moe.combine_backward(q, dy, layer.o, layer.pos, layer.gate, dO, dgate, ds=ds, prob=0.3, rng=rng,
                             indptr=layer.indptr, row_token=layer.row_token)
        moe.permute_backward(q, dO, layer.pos, dx)
        return [y, layer.W1, layer.w1s, layer.pos, out, dO, dgate, ds, dx]

    bound = everything()
    monkeypatch.setattr(moe, "_BINDING", moe._Unbound())
    for a, b in zip(bound, everything()):
        assert torch.equal(a, b)
