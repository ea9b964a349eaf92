"""Failure detection of the 8-bit products without a fault: bounded waits that
run out (moe_set_wait_limit(1): every wait not satisfied at its first probe
gives up), and the debug build's bounds checks. Afterwards the same calls give
the right bits."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mixture_experts_layer_62_b200 as moe
import ops_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"
CASES = [dict(T=40, d=512, dff=1024, E=4, form="single"), dict(T=2000, d=1024, dff=4096, E=2, form="pair")]


def inputs(c, seed=1):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    T, d, dff, E = c["T"], c["d"], c["dff"], c["E"]
    p = moe.problem(T, d, dff, E, 1)
    ends = torch.linspace(0, T, E + 1).to(torch.int32).to(DEV)
    return dict(p=p, q=i8(T, d), s=torch.rand((T,), generator=g, device=DEV) * 1e-4, W1=i8(E, dff, d), W3=i8(E, dff, d),
                ws=torch.rand((E, dff), generator=g, device=DEV), indptr=ends, work=moe.alloc_int8_workspace(p, DEV))


def up(m, offsets=None):
    st = moe.alloc_stats(m["p"].E, DEV)
    h = torch.full((m["p"].T, m["p"].d_ff), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.expert_up_int8(m["p"], m["q"], m["s"], m["indptr"] if offsets is None else offsets, m["W1"], m["ws"], m["W3"],
                       m["ws"], h, m["work"], stats=st)
    torch.cuda.synchronize()
    return h, moe.read_stats(st, m["p"].E).status


def right(m, h):
    a, b = (R.product(m["q"], m["s"], m[w], m["ws"], m["indptr"]) for w in ("W1", "W3"))
    return bool(((h.double() - R.swiglu(a, b)).abs() <= R.swiglu_bound(a, b, torch.bfloat16)).all())


@pytest.mark.parametrize("c", CASES, ids=lambda c: c["form"])
def test_wait_runs_out_then_recovers(c):
    m = inputs(c)
    assert moe.int8_variant(m["p"]) == c["form"]
    prev = moe.set_wait_limit(1)
    try:
        _, status = up(m)
    finally:
        moe.set_wait_limit(prev)
    assert status == moe.MOE_ERR_TIMEOUT
    for _ in range(2):
        h, status = up(m)
        assert status == moe.MOE_OK and right(m, h)


def debug_runs():
    out = {}
    for i, c in enumerate(CASES):
        m = inputs(c, 5 + i)
        h, status = up(m)
        out[f"h{i}"], out[f"status{i}"] = h.view(torch.int16).cpu().numpy(), np.array([status])
    return out


def debug_bad():
    m = inputs(CASES[0])
    h, status = up(m, torch.tensor([0, 10, 41, 20, 40], dtype=torch.int32, device=DEV))
    return {"bad": np.array([status]), "rows": (h == 7.0).all(1).cpu().numpy()}


SCRIPT = r"""
import sys
import numpy as np
sys.path.insert(0, sys.argv[2])
sys.path.insert(0, sys.argv[2] + "/tests")
import mixture_experts_layer_62_b200 as moe
assert moe.LIB_PATH.endswith("libmoe_debug.so"), moe.LIB_PATH
from test_gpu_int8_failure import debug_bad, debug_runs
np.savez(sys.argv[1], **debug_runs(), **debug_bad())
"""


def test_debug_build_gives_the_same_bits_and_reports_bad_offsets(tmp_path):
    path = tmp_path / "debug.npz"
    r = subprocess.run([sys.executable, "-c", SCRIPT, str(path), ROOT], env=dict(os.environ, MOE_LIBRARY="debug"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    dbg, rel = dict(np.load(path)), debug_runs()
    for i in range(len(CASES)):
        assert int(dbg[f"status{i}"][0]) == moe.MOE_OK and np.array_equal(dbg[f"h{i}"], rel[f"h{i}"])
    assert int(dbg["bad"][0]) == moe.MOE_ERR_BOUNDS
    # groups 1 (ends past the 40 rows) and 2 (runs backwards) are left out, 0 and 3 run
    rows = dbg["rows"]
    assert not rows[:10].any() and rows[10:20].all() and not rows[20:].any()
