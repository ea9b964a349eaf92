"""The router on the tensor cores gives up a wait: the statistics of the call
say so, although the scan that follows writes the rest of their header."""

import math

import pytest
import torch

import mixture_experts_layer_62_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,E", [(300, 64), (1000, 256)])
def test_route_reports_a_wait_that_gave_up(T, E):
    d, k = 1024, 2
    p = moe.problem(T, d, 64, E, k)
    assert moe.router_variant(p, forward=False) == "tensor"
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    x = torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16)
    W_r = (torch.randn((d, E), generator=g, device=DEV) / math.sqrt(d)).to(torch.bfloat16)
    work, st = moe.alloc_workspace(p, DEV), moe.alloc_stats(E, DEV)

    def route():
        idx, gate = torch.zeros((T, k), dtype=torch.int32, device=DEV), torch.zeros((T, k), device=DEV)
        moe.route(p, x, W_r, idx, gate, st, work)
        return idx, gate, moe.read_stats(st, E)

    idx, gate, right = route()
    assert right.status == moe.MOE_OK
    prev = moe.set_wait_limit(1)
    try:
        assert route()[2].status == moe.MOE_ERR_TIMEOUT
    finally:
        moe.set_wait_limit(prev)
    again = route()
    assert again[2] == right and torch.equal(again[0], idx) and torch.equal(again[1], gate)
