"""A stage of the 8-bit layer gives up a wait: read_stats() names the first
failure of the pass, also when every stage after it ended well, and the next
pass is MOE_OK again."""

import math

import pytest
import torch

import mixture_experts_layer_62_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(T, d, dff, E, k, dfs=0, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(T + E)
    n = lambda *s: (torch.randn(s, generator=g, device=DEV) / math.sqrt(s[-1])).to(torch.bfloat16)  # noqa: E731
    w = dict(W_r=n(d, E), W1=n(E, dff, d), W3=n(E, dff, d), W2=n(E, d, dff))
    if dfs:
        w |= dict(Ws1=n(dfs, d), Ws3=n(dfs, d), Ws2=n(d, dfs))
    p = moe.problem(T, d, dff, E, k, d_ff_shared=dfs, pad_rows=pad)
    return moe.MoELayerInt8(p, **w), (8 * n(T, d)).contiguous()


def at_call(monkeypatch, name, call, then):
    """then(call, args, kw) takes the place of the call-th call (from 0) of moe.<name>."""
    real, seen = getattr(moe, name), []

    def wrapped(*args, **kw):
        seen.append(name)
        return real(*args, **kw) if len(seen) - 1 != call else then(real, args, kw)

    monkeypatch.setattr(moe, name, wrapped)
    return seen


def give_up(real, args, kw):
    """Its waits run out at their first probe (which is satisfied in time where there is little to wait for)."""
    prev = moe.set_wait_limit(1)
    try:
        return real(*args, **kw)
    finally:
        moe.set_wait_limit(prev)


def record(real, args, kw):
    """It ends with the word that a wait which gave up would have left."""
    real(*args, **kw)
    stats = kw["stats"] if "stats" in kw else args[5]      # moe.route takes it in its sixth place
    stats[:4].view(torch.int32).fill_(moe.MOE_ERR_TIMEOUT)


STAGES = {"router": ("route", 0), "up": ("expert_up_int8", 0), "down": ("expert_down_int8", 0),
          "shared up": ("expert_up_int8", 1), "shared down": ("expert_down_int8", 1)}


@pytest.mark.parametrize("stage", STAGES)
def test_the_first_failure_of_a_pass_is_kept(stage, monkeypatch):
    layer, x = make(300, 512, 1024, 64, 2, dfs=256)
    right = layer(x).clone()
    first = layer.read_stats()
    assert first.status == moe.MOE_OK
    name, call = STAGES[stage]
    with monkeypatch.context() as m:
        seen = at_call(m, name, call, record)
        layer(x)
        assert len(seen) > call
    assert layer.read_stats().status == moe.MOE_ERR_TIMEOUT
    again = layer(x)
    assert layer.read_stats() == first and torch.equal(again, right)


@pytest.mark.parametrize("T,d,dff,E,k,form", [(1, 256, 512, 8, 2, "single"), (40, 512, 1024, 8, 2, "single"),
                                              (3000, 1024, 2048, 2, 1, "pair")])
def test_an_up_projection_that_gave_up_is_not_covered_by_the_down_projection(T, d, dff, E, k, form, monkeypatch):
    layer, x = make(T, d, dff, E, k)
    assert moe.int8_variant(layer.experts) == form
    right = layer(x).clone()
    seen = set()
    for _ in range(5):
        with monkeypatch.context() as m:
            at_call(m, "expert_up_int8", 0, give_up)
            layer(x)
        seen.add(layer.read_stats().status)
        assert torch.equal(layer(x), right) and layer.read_stats().status == moe.MOE_OK
    assert moe.MOE_ERR_TIMEOUT in seen


def test_a_captured_pass_reports_it_too(monkeypatch):
    layer, x = make(24, 256, 512, 8, 2)
    right, out = layer(x).clone(), torch.zeros_like(layer.out)
    torch.cuda.synchronize()
    graphs = []
    for bad in (False, True):
        with monkeypatch.context() as m:
            if bad:
                at_call(m, "expert_up_int8", 0, record)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                layer(x, out=out)
            graphs.append(g)
    for bad in (True, False, True, True, False):
        graphs[bad].replay()
        torch.cuda.synchronize()
        assert layer.read_stats().status == (moe.MOE_ERR_TIMEOUT if bad else moe.MOE_OK)
        assert bad or torch.equal(out, right)


def test_the_statistics_are_the_routers_and_the_permutations():
    for pad in (0, 64):
        layer, x = make(200, 256, 320, 16, 4, pad=pad)
        layer(x)
        st, per = layer.read_stats(), moe.alloc_stats(16, DEV)
        p = layer.experts
        moe.permute_int8(p, x, layer.idx, layer.pos, layer.indptr, layer.row_token, layer.xq, layer.xs, per, layer.workspace)
        per = moe.read_stats(per, 16)
        assert (st.counts, st.kept, st.rows, st.dropped, st.capacity, st.max_count, st.max_over_mean) == \
            (per.counts, per.kept, per.rows, per.dropped, per.capacity, per.max_count, per.max_over_mean)
        assert st.l_aux > 0 and abs(sum(st.P) - 1) < 1e-3
