"""A wait of the 8-bit products that gives up at any point of a launch: limits
from one probe to several microseconds stop the loads, the MMAs and the
epilogues at different places, also where one of them has come to its end
already and the two CTAs of a pair have requested different numbers of blocks.
What was started lands before a CTA leaves, without the two seconds after which
even that is given up, and the next call gives the right bits."""

import time

import pytest
import torch

import mixture_experts_layer_62_b200 as moe
import ops_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMITS = (1, 200, 700, 1500, 3000, 6000, 12000, 25000)
CASES = [
    dict(T=40, d=512, dff=1024, E=4, form="single"),       # K blocks of a tile: no more than stages
    dict(T=40, d=1024, dff=512, E=4, form="single"),
    dict(T=30, d=64, dff=4096, E=3, form="single"),        # one block
    dict(T=24, d=4096, dff=8192, E=2, form="single"),      # tails cut along K, more blocks than stages
    dict(T=2000, d=1024, dff=4096, E=2, form="pair"),
    dict(T=2000, d=4096, dff=4096, E=2, form="pair"),
    dict(T=2100, d=512, dff=8192, E=2, form="pair"),       # short last blocks, two sets a tile
]


def inputs(c, down):
    g = torch.Generator(device=DEV)
    g.manual_seed(c["T"] + c["d"])
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    T, d, dff, E = c["T"], c["d"], c["dff"], c["E"]
    # the products alike: K = d, N = dff
    p = moe.problem(T, dff, d, E, 1) if down else moe.problem(T, d, dff, E, 1)
    ends = torch.linspace(0, T, E + 1).to(torch.int32).to(DEV)
    return dict(p=p, q=i8(T, d), s=torch.rand((T,), generator=g, device=DEV) * 1e-4, W=[i8(E, dff, d) for _ in range(2)],
                ws=torch.rand((E, dff), generator=g, device=DEV), indptr=ends, work=moe.alloc_int8_workspace(p, DEV))


def product(m, down):
    st = moe.alloc_stats(m["p"].E, DEV)
    out = torch.full((m["p"].T, m["ws"].shape[1]), 7.0, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    if down:
        moe.expert_down_int8(m["p"], m["q"], m["s"], m["indptr"], m["W"][0], m["ws"], out, m["work"], stats=st)
    else:
        moe.expert_up_int8(m["p"], m["q"], m["s"], m["indptr"], m["W"][0], m["ws"], m["W"][1], m["ws"], out, m["work"],
                           stats=st)
    torch.cuda.synchronize()
    return out, moe.read_stats(st, m["p"].E).status, time.perf_counter() - t0


@pytest.mark.parametrize("down", [False, True], ids=["up", "down"])
@pytest.mark.parametrize("c", CASES, ids=lambda c: f"{c['form']}-T{c['T']}-K{c['d']}-N{c['dff']}")
def test_a_wait_gives_up_anywhere(c, down):
    m = inputs(c, down)
    assert moe.int8_variant(m["p"], down=down) == c["form"]
    a, b = (R.product(m["q"], m["s"], w, m["ws"], m["indptr"]) for w in m["W"])
    ref, bound = (a, R.plain_bound(a, torch.bfloat16)) if down else (R.swiglu(a, b), R.swiglu_bound(a, b, torch.bfloat16))
    right, status, _ = product(m, down)
    assert status == moe.MOE_OK and ((right.double() - ref).abs() <= bound).all()
    stopped = 0
    for limit in LIMITS:
        prev = moe.set_wait_limit(limit)
        try:
            for _ in range(4):
                out, status, seconds = product(m, down)
                assert status == moe.MOE_ERR_TIMEOUT or (status == moe.MOE_OK and torch.equal(out, right))
                stopped += status == moe.MOE_ERR_TIMEOUT
                assert seconds < 1.0
        finally:
            moe.set_wait_limit(prev)
        out, status, _ = product(m, down)
        assert status == moe.MOE_OK and torch.equal(out, right)
    assert stopped > 0
