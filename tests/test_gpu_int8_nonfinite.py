"""Rows with an infinity or a NaN in 8 bits: the scale is NaN, so that everything
computed from such a row is NaN, and no other row changes a bit."""

import pytest
import torch

import mixture_experts_layer_62_b200 as moe
import ops_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BAD = (float("nan"), float("inf"), -float("inf"))


def spoiled(x, seed):
    """x with one value (or several, or all) of every third row made not finite, and those rows."""
    g = torch.Generator().manual_seed(seed)
    x, rows, cols = x.clone(), x.shape[0], x.shape[1]
    hit = torch.zeros(rows, dtype=torch.bool)
    hit[::3] = True
    for i, r in enumerate(hit.nonzero()[:, 0].tolist()):
        at = [0, cols - 1, int(torch.randint(cols, (1,), generator=g))][i % 3]
        x[r, at] = BAD[i // 3 % 3]
        if i % 5 == 3:
            x[r, (at + 7) % cols] = BAD[(i + 1) % 3]
        if i % 5 == 4:
            x[r] = BAD[i % 3]
    return x, hit.to(DEV)


def check(x, q, s, hit):
    assert s[hit].isnan().all()
    R.check_quantized(x[~hit], q[~hit], s[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (50, 64), (40, 2064), (33, 4096), (20, 8208), (17, 16400), (300, 208)])
def test_quantize_rows(rows, cols, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(rows + cols)
    x, hit = spoiled(torch.randn((rows, cols), generator=g, device=DEV).to(DT[dtype]), rows)
    check(x, *moe.quantize_rows(x), hit)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [30, 1500])      # one launch, and three
def test_permutation_and_product(T, dtype):
    d, N, E, k = 256, 192, 4, 2
    p = moe.problem(T, N, d, E, k, 0.0, dtype, pad_rows=64)
    rows = moe.permuted_rows(p)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    x, hit = spoiled(torch.randn((T, d), generator=g, device=DEV).to(DT[dtype]), T)
    idx = R.routed(T, E, k, T).to(DEV)
    pos, indptr = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty(E + 1, dtype=torch.int32, device=DEV)
    token = torch.empty(rows, dtype=torch.int32, device=DEV)
    xq, xs = torch.empty((rows, d), dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    up = moe.problem(T, d, N, E, k, 0.0, dtype, pad_rows=64)
    work, st = moe.alloc_int8_workspace(up, DEV), moe.alloc_stats(E, DEV)
    moe.permute_int8(up, x, idx, pos, indptr, token, xq, xs, st, work)
    n = int(indptr[E])
    real = token[:n] >= 0
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[real] = hit[token[:n][real].long()]
    at = token[:n][real].long()
    check(x[at], xq[:n][real], xs[:n][real], hit[at])
    assert (xq[:n][~real] == 0).all() and (xs[:n][~real] == 0).all()
    W = [torch.randint(-128, 128, (E, N, d), generator=g, device=DEV, dtype=torch.int8) for _ in range(2)]
    ws = torch.rand((E, N), generator=g, device=DEV) * 1e-2
    # rows that nothing spoils, from the same values
    xs0 = torch.where(xs.isnan(), torch.zeros_like(xs), xs)
    outs = []
    for scale in (xs, xs0):
        h, o = (torch.full((rows, N), 7.0, dtype=DT[dtype], device=DEV) for _ in range(2))
        moe.expert_up_int8(up, xq, scale, indptr, W[0], ws, W[1], ws, h, work)
        moe.expert_down_int8(p, xq, scale, indptr, W[0], ws, o, work)
        outs.append((h, o))
    for a, b in zip(*outs):
        assert a[:n][bad].isnan().all()
        assert torch.equal(a[:n][~bad], b[:n][~bad]) and (a[n:] == 7.0).all()
