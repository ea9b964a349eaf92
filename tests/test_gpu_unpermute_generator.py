"""The generator of the dropout against the published test vector of
Philox4x32-10, and masks and gradients past 2^31 elements."""

import numpy as np
import pytest
import torch

import mixture_experts_layer_62_b200 as moe
import ops_ref as R

DEV = "cuda"
# Random123's known answers (Salmon, Moraes, Dror and Shaw 2011): counter, key, result
VECTORS = [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
]


def philox(counter, key):
    x, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(p1 >> 32) ^ x[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ x[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return tuple(x)


def halves(block, seed, offset):
    """The numbers of the elements 8 block .. 8 block + 7."""
    m = 0xFFFFFFFF
    w = philox((block & m, block >> 32, offset & m, offset >> 32), (seed & m, seed >> 32))
    return [h for v in w for h in (v & 0xFFFF, v >> 16)]


def test_published_vectors():
    for counter, key, want in VECTORS:
        assert philox(counter, key) == want
    # the generator that the other tests use: its first blocks, with words of every size in seed and offset
    for seed, offset in ((0, 0), (0x299F31D0A4093822, 0x0370734413198A2E), ((1 << 64) - 1, (1 << 64) - 1)):
        for thr in (1, 30000, 65535):
            keep = R.philox_keep(40, seed, offset, thr)
            assert keep.tolist() == [h >= thr for b in range(5) for h in halves(b, seed, offset)]


def signed(v):
    return v - (1 << 64) if v >> 63 else v


@pytest.mark.gpu
@pytest.mark.parametrize("seed,offset", [(0, 0), (0x299F31D0A4093822, 0x0370734413198A2E), ((1 << 64) - 1, (1 << 64) - 1)])
def test_the_kernels_numbers(seed, offset):
    # an element is kept up to the probability of its number, and dropped from the next one on
    if (seed, offset) == (0, 0):
        assert halves(0, 0, 0) == [h for v in VECTORS[0][2] for h in (v & 0xFFFF, v >> 16)]
    d, p = 64, moe.problem(1, 64, 64, 1, 1)
    o = torch.ones((1, d), dtype=torch.bfloat16, device=DEV)
    pos, gate = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV)
    rng = torch.tensor([signed(seed), signed(offset)], dtype=torch.int64, device=DEV)
    numbers = [h for b in range(d // 8) for h in halves(b, seed, offset)]
    for i in range(8):
        for thr in (numbers[i], numbers[i] + 1):
            if 0 < thr < 65536:
                y = moe.combine_dropout(p, o, pos, gate, torch.empty_like(o), prob=thr / 65536, rng=rng)
                assert (y[0] != 0).tolist() == [h >= thr for h in numbers]


@pytest.mark.gpu
def test_past_32_bits_of_elements():
    T, d, prob = (1 << 31) // 4096 + 3000, 4096, 0.25      # 2^31 elements and 3000 tokens more
    p = moe.problem(T, d, 64, 1, 1)
    seed, offset, thr = 0x123456789ABCDEF0, (1 << 40) + 9, 16384
    rng = torch.tensor([seed, offset], dtype=torch.int64, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    new = lambda: torch.empty((T, d), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    o, dy = (new().normal_(generator=g) for _ in range(2))
    # the rows in reverse order: the last tokens read the first rows
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device=DEV)[:, None].contiguous()
    gate = torch.rand((T, 1), generator=g, device=DEV)
    out, dO, ds, dgate, dx = new(), new(), new(), torch.empty((T, 1), device=DEV), new()
    moe.combine_dropout(p, o, pos, gate, out, prob=prob, rng=rng)
    moe.combine_backward(p, dy, o, pos, gate, dO, dgate, ds=ds, prob=prob, rng=rng)
    moe.permute_backward(p, dO, pos, dx)
    half = R.HALF[torch.bfloat16]
    for t0 in (0, (1 << 31) // d - 2, T - 4):               # first, across the border, last
        keep = np.array([[h >= thr for b in range(t * d // 8, (t + 1) * d // 8) for h in halves(b, seed, offset)]
                         for t in range(t0, t0 + 4)])
        f = torch.from_numpy(keep).to(DEV).double() * (65536 / (65536 - thr))
        rows = pos[t0:t0 + 4, 0].long()
        go, u = gate[t0:t0 + 4].double(), dy[t0:t0 + 4].double() * f
        x = o[rows].double()
        ref = go * x * f
        assert ((out[t0:t0 + 4].double() - ref).abs() <= ref.abs() * (half + 4 * R.U)).all()
        assert ((ds[t0:t0 + 4].double() - u).abs() <= u.abs() * (half + 3 * R.U)).all()
        ref = go * u
        assert ((dO[rows].double() - ref).abs() <= ref.abs() * (half + 4 * R.U)).all()
        assert torch.equal(dx[t0:t0 + 4], dO[rows])
        # a thread's chain (8 columns of every 128th vector), a warp's five halvings, four warps, u's two roundings
        chain, prod = 8 * -(-d // (8 * 128)) + 5 + 4 + 2, u * x
        assert ((dgate[t0:t0 + 4, 0].double() - prod.sum(1)).abs() <= 1.01 * chain * R.U * prod.abs().sum(1) + 1e-37).all()


@pytest.mark.gpu
def test_rows_in_8_bits_past_32_bits_of_elements():
    d, E, k = 4096, 4, 2
    T = (1 << 30) // d + 1500                                # 2^31 elements and 3000 rows more once permuted
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.empty((T, d), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    idx = torch.stack([torch.arange(T, device=DEV) % E, (torch.arange(T, device=DEV) + 1) % E], 1).to(torch.int32).contiguous()
    p = moe.problem(T, d, 64, E, k)
    N = moe.permuted_rows(p)
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    pos, indptr, token = i32(T, k), i32(E + 1), i32(N)
    xq, xs = torch.empty((N, d), dtype=torch.int8, device=DEV), torch.empty(N, device=DEV)
    moe.permute_int8(p, x, idx, pos, indptr, token, xq, xs, moe.alloc_stats(E, DEV), moe.alloc_int8_workspace(p, DEV))
    assert int(indptr[E]) == N and N * d > 1 << 31
    for lo in (0, (1 << 31) // d - 20, N - 40):
        rows = slice(lo, lo + 40)
        R.check_quantized(x[token[rows].long()], xq[rows], xs[rows])
    assert torch.equal(token[pos.long()], torch.arange(T, dtype=torch.int32, device=DEV)[:, None].expand(T, k))
    big = x.view(-1)[:(T // 2) * 2 * d].view(T // 2, 2 * d)
    big = torch.cat([big, big[:3000 + 5]])                   # 2^29 elements ..
    rows = torch.cat([big, big, big, big])                   # .. and past 2^31
    q, s = moe.quantize_rows(rows)
    assert rows.numel() > 1 << 31
    for lo in (0, (1 << 31) // (2 * d) - 20, rows.shape[0] - 40):
        R.check_quantized(rows[lo:lo + 40], q[lo:lo + 40], s[lo:lo + 40])


@pytest.mark.gpu
@pytest.mark.parametrize("E,form", [(2, "pair"), (512, "single")])
def test_products_past_32_bits_of_results(E, form):
    K, N = 64, 14336
    T = (1 << 31) // N + 700
    p = moe.problem(T, K, N, E, 1)
    assert moe.int8_variant(p) == form
    g = torch.Generator(device=DEV)
    g.manual_seed(E)
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    xq, W1, W3 = i8(T, K), i8(E, N, K), i8(E, N, K)
    xs, ws = torch.rand(T, generator=g, device=DEV) * 1e-3, 0.5 + torch.rand((E, N), generator=g, device=DEV)
    ends = torch.linspace(0, T, E + 1, dtype=torch.float64).to(torch.int32).to(DEV)
    h = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    st = moe.alloc_stats(E, DEV)
    moe.expert_up_int8(p, xq, xs, ends, W1, ws, W3, ws, h, moe.alloc_int8_workspace(p, DEV), stats=st)
    assert moe.read_stats(st, E).status == moe.MOE_OK
    host = ends.tolist()
    for lo in (0, (1 << 31) // N - 20, T - 40):
        for r in range(lo, lo + 40):
            e = max(i for i in range(E) if host[i] <= r)
            one = torch.tensor([0, 1])
            a, b = (R.product(xq[r:r + 1], xs[r:r + 1], W[e:e + 1], ws[e:e + 1], one) for W in (W1, W3))
            assert ((h[r:r + 1].double() - R.swiglu(a, b)).abs() <= R.swiglu_bound(a, b, torch.bfloat16)).all()
