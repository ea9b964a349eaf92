"""moe_permute when a token names an expert in more than one slot: every pair
still gets a row of its own, in slot order."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_62_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("drop", [0, 1])
def test_permute_names_an_expert_twice(drop):
    T, E, k, d = 70, 5, 3, 64
    p = moe.problem(T, d, 64, E, k, drop_order=drop)
    rng = np.random.default_rng(1)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)      # repeats within a token are common
    x = torch.randn((T, d), device=DEV).to(torch.bfloat16)
    i32 = lambda *s: torch.full(s, -5, dtype=torch.int32, device=DEV)  # noqa: E731
    pos, indptr, rt, xp = i32(T, k), i32(E + 1), i32(T * k), torch.zeros((T * k, d), dtype=torch.bfloat16, device=DEV)
    moe.permute(p, x, torch.from_numpy(idx).to(DEV), pos, indptr, rt, xp, moe.alloc_stats(E, DEV), moe.alloc_workspace(p, DEV))
    order = [(t, j) for j in range(k) for t in range(T)] if drop else [(t, j) for t in range(T) for j in range(k)]
    start = np.concatenate([[0], np.cumsum(np.bincount(idx.reshape(-1), minlength=E))])
    want, seen = np.zeros((T, k), dtype=np.int64), [0] * E
    for t, j in order:
        e = idx[t, j]
        want[t, j] = start[e] + seen[e]
        seen[e] += 1
    assert (pos.cpu().numpy() == want).all() and (indptr.cpu().numpy() == start).all()
    token = np.repeat(np.arange(T), k)
    got = rt.cpu().numpy()
    assert (got[want.reshape(-1)] == token).all()
    assert torch.equal(xp[torch.from_numpy(want.reshape(-1)).to(DEV)], x[torch.from_numpy(token).to(DEV)])
