"""The way back from the experts (dropout, residual, gradients) against
64-bit plain forms (tests/ops_ref.py)."""

import pytest
import torch

import mixture_experts_layer_62_b200 as moe
import ops_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

CASES = [dict(T=1, d=64, E=4, k=1), dict(T=1, d=4096, E=8, k=2, prob=0.1), dict(T=5, d=192, E=16, k=16, prob=0.5),
         dict(T=45, d=128, E=7, k=3, cf=0.7, pad=64, shared=True, prob=0.25),
         dict(T=300, d=1024, E=8, k=2, cf=0.5, residual=True, prob=0.9), dict(T=130, d=2112, E=12, k=5, residual=True),
         dict(T=700, d=320, E=64, k=8, cf=1.0, pad=128, shared=True, residual=True, prob=0.05),
         dict(T=64, d=7168, E=9, k=9, cf=0.6, prob=0.3, shared=True),
         dict(T=2500, d=64, E=40, k=3, pad=128, prob=0.1), dict(T=3, d=520 * 8, E=70, k=2, pad=64)]


def make(c, dtype, seed=0):
    T, d, E, k = c["T"], c["d"], c["E"], c["k"]
    if dtype == "f32":
        d += 8      # rows that end inside a warp's stretch
    dt, pad, cf = DT[dtype], c.get("pad", 0), c.get("cf", 0.0)
    p = moe.problem(T, d, 64, E, k, cf, dtype, pad_rows=pad)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + T + d)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    idx = R.routed(T, E, k, seed + T, 1.0)
    if T > 3:
        idx[2] = idx[2, 0]      # one expert in every slot
    pos, indptr, rt, _, _ = R.permutation(idx, E, R.capacity(cf, T, k, E), pad)
    N = moe.permuted_rows(p)
    row_token = torch.full((N,), 123456, dtype=torch.int32)    # behind the last row: anything
    row_token[:len(rt)] = torch.from_numpy(rt)
    o = rn(N, d)
    used = torch.zeros(N, dtype=torch.bool, device=DEV)
    pos_t = torch.from_numpy(pos).to(DEV)
    used[pos_t[pos_t >= 0]] = True
    o[~used] = float("nan")     # rows of no pair are never read
    m = dict(p=p, T=T, d=d, E=E, k=k, N=N, dt=dt, pos=pos_t.to(torch.int32), used=used, o=o.to(dt),
             gate=torch.softmax(rn(T, k), 1), dy=rn(T, d).to(dt), s=rn(T, d).to(dt) if c.get("shared") else None,
             residual=rn(T, d).to(dt) if c.get("residual") else None, prob=c.get("prob", 0.0),
             indptr=torch.from_numpy(indptr).to(torch.int32).to(DEV), row_token=row_token.to(DEV), n=len(rt))
    seed64, off = 0x9E3779B97F4A7C15 ^ (T * 77), (1 << 63) + 12345 + d
    m["rng"] = torch.tensor([seed64 - (1 << 64) if seed64 >> 63 else seed64, off - (1 << 64)], dtype=torch.int64, device=DEV)
    m["factor"] = R.factor_of(T, d, m["prob"], seed64, off, DEV)
    return m


def forward(m, out=None):
    out = torch.full((m["T"], m["d"]), 9.0, dtype=m["dt"], device=DEV) if out is None else out
    return moe.combine_dropout(m["p"], m["o"], m["pos"], m["gate"], out, s=m["s"], residual=m["residual"],
                               prob=m["prob"], rng=m["rng"] if m["prob"] else None)


def backward(m):
    dO = torch.full((m["N"], m["d"]), 9.0, dtype=m["dt"], device=DEV)
    dgate = torch.full((m["T"], m["k"]), 9.0, device=DEV)
    ds = torch.full((m["T"], m["d"]), 9.0, dtype=m["dt"], device=DEV)
    moe.combine_backward(m["p"], m["dy"], m["o"], m["pos"], m["gate"], dO, dgate, ds=ds, prob=m["prob"],
                         rng=m["rng"] if m["prob"] else None, indptr=m["indptr"], row_token=m["row_token"])
    return dO, dgate, ds


ids = lambda c: "-".join(f"{k}{v}" for k, v in c.items())  # noqa: E731


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES, ids=ids)
def test_combine_dropout(c, dtype):
    m = make(c, dtype)
    y = forward(m)
    ref, mag = R.mix(m["o"], m["pos"], m["gate"], m["s"], m["residual"], m["factor"])
    assert ((y.double() - ref).abs() <= R.mix_bound(ref, mag, m["k"], m["dt"])).all()
    if m["prob"] and m["residual"] is None:
        assert (y[m["factor"] == 0] == 0).all()      # dropped means exactly nothing
    assert torch.equal(forward(m), y)
    if m["prob"] == 0 and m["residual"] is None:
        # without dropout and residual it is moe_combine, bit for bit
        z = torch.empty_like(y)
        moe.combine(m["p"], m["o"], m["pos"], m["gate"], z, s=m["s"])
        assert torch.equal(y, z)
    if m["residual"] is not None:                     # in place over the residual
        m["residual"] = m["residual"].clone()
        assert torch.equal(forward(m, out=m["residual"]), y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES, ids=ids)
def test_combine_backward(c, dtype):
    m = make(c, dtype)
    dO, dgate, ds = backward(m)
    u = m["dy"].double()
    if m["factor"] is not None:
        u = torch.where(m["factor"] > 0, u * m["factor"], torch.zeros_like(u))
    half = R.HALF[m["dt"]]
    assert ((ds.double() - u).abs() <= u.abs() * (half + 2 * R.U)).all()
    want = torch.full((m["N"], m["d"]), 9.0, dtype=torch.float64, device=DEV)
    if m["p"].pad_rows:
        want[:m["n"]][m["row_token"][:m["n"]] < 0] = 0.0    # padding rows; the others of no pair stay
    gref, mag = torch.zeros((m["T"], m["k"]), dtype=torch.float64, device=DEV), torch.zeros((m["T"], m["k"]), device=DEV)
    for j in range(m["k"]):
        on = (m["pos"][:, j] >= 0).nonzero()[:, 0]
        r = m["pos"][on, j].long()
        want[r] = m["gate"][on, j, None].double() * u[on]
        prod = u[on] * m["o"][r].double()
        gref[on, j] = prod.sum(1)
        mag[on, j] = prod.abs().sum(1).float()
    assert ((dO.double() - want).abs() <= want.abs() * (half + 4 * R.U)).all()
    assert (dgate[m["pos"] < 0] == 0).all()
    # a thread's chain of fused multiply-adds (8 columns of every 128th vector), five
    # halvings in a warp, the warps' sums, and u's own two roundings
    chain = 8 * -(-m["d"] // (8 * 128)) + 5 + 4 + 2
    assert ((dgate.double() - gref).abs() <= 1.01 * chain * R.U * mag.double() + 1e-37).all()
    again = backward(m)
    assert all(torch.equal(a, b) for a, b in zip(again, (dO, dgate, ds)))


@pytest.mark.parametrize("c", [CASES[3], CASES[4], CASES[6]], ids=ids)
def test_gradients_are_differences(c):
    # y is linear in o, s and the residual and, at fixed o, in the gates: a
    # central difference with a step of 1 is exact but for the rounding of y,
    # which mix_bound states
    m = make(c, "f32")
    m["o"] = torch.where(m["used"][:, None], m["o"], torch.zeros_like(m["o"]))
    dO, dgate, ds = backward(m)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    rn = lambda t: torch.randn(t.shape, generator=g, device=DEV)  # noqa: E731
    dy = m["dy"].double()

    def loss():
        y, mag = R.mix(m["o"], m["pos"], m["gate"], m["s"], m["residual"], m["factor"])
        return (dy * forward(m).double()).sum(), (dy.abs() * R.mix_bound(y, mag, m["k"], m["dt"])).sum()

    def difference(name, v):
        keep, out, slack = m[name], [], 0.0
        for sign in (1.0, -1.0):
            m[name] = keep + sign * v
            val, off = loss()
            out.append(val)
            # the shifted input itself is rounded: one U of its magnitude
            y, mag = R.mix(*(m[n] if n != name else m[n].abs() for n in ("o", "pos", "gate", "s", "residual")), m["factor"])
            slack += off + (dy.abs() * mag).sum() * R.U * 2
        m[name] = keep
        return (out[0] - out[1]) / 2, slack / 2

    w = dO.double().clone()
    w[~m["used"]] = 0
    for name, grad in (("o", w), ("gate", dgate.double())) + ((("s", ds.double()),) if m["s"] is not None else ()):
        v = rn(m[name])
        diff, slack = difference(name, v)
        got = (grad * v.double()).sum()
        # the gradient's own bound: dO and ds one rounding each and the scale, dgate its chain
        chain = 8 * -(-m["d"] // (8 * 128)) + 12
        off = (grad.abs() * v.double().abs()).sum() * 6 * R.U
        if name == "gate":
            u = dy if m["factor"] is None else dy * m["factor"]
            for j in range(m["k"]):
                on = (m["pos"][:, j] >= 0).nonzero()[:, 0]
                r = m["pos"][on, j].long()
                off = off + chain * R.U * ((u[on] * m["o"][r].double()).abs().sum(1) * v[on, j].abs()).sum()
        assert (got - diff).abs() <= 1.01 * (slack + off), (name, got.item(), diff.item(), (slack + off).item())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", CASES, ids=ids)
def test_permute_backward(c, dtype):
    m = make(c, dtype)
    dx = torch.full((m["T"], m["d"]), 9.0, dtype=m["dt"], device=DEV)
    moe.permute_backward(m["p"], m["o"], m["pos"], dx)
    ref, mag = R.mix(m["o"], m["pos"], torch.ones_like(m["gate"]))
    assert ((dx.double() - ref).abs() <= R.mix_bound(ref, mag, m["k"], m["dt"])).all()
    gone = (m["pos"] < 0).all(1)
    assert (dx[gone] == 0).all()


def test_positions_outside_the_rows_count_as_dropped():
    m = make(dict(T=20, d=64, E=4, k=2), "bf16")
    for bad in (m["N"], m["N"] + 7, 2 ** 31 - 1, -1, -2 ** 31):
        wild, tame = dict(m), dict(m)
        wild["pos"], tame["pos"] = m["pos"].clone(), m["pos"].clone()
        wild["pos"][3, 1], tame["pos"][3, 1] = bad, -1
        assert torch.equal(forward(wild), forward(tame))
        assert all(torch.equal(a, b) for a, b in zip(backward(wild), backward(tame)))


def test_no_tokens():
    p = moe.problem(0, 64, 64, 4, 2)
    z = torch.zeros((1, 64), dtype=torch.bfloat16, device=DEV)
    i, f = torch.zeros((1, 2), dtype=torch.int32, device=DEV), torch.zeros((1, 2), device=DEV)
    z.fill_(3)
    moe.combine_dropout(p, z, i, f, z)
    moe.combine_backward(p, z, z, i, f, z, f)
    moe.permute_backward(p, z, i, z)
    assert (z == 3).all()


def test_dropout_keeps_its_share_and_follows_the_generator():
    T, d = 500, 1024
    p = moe.problem(T, d, 64, 1, 1)
    o = torch.ones((T, d), dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)[:, None].contiguous()
    gate = torch.ones((T, 1), device=DEV)
    rng = torch.tensor([42, 7], dtype=torch.int64, device=DEV)
    masks = []
    for prob in (0.1, 0.5, 0.99998):
        y = moe.combine_dropout(p, o, pos, gate, torch.empty_like(o), prob=prob, rng=rng)
        kept = (y != 0).float().mean().item()
        # n independent elements: five standard deviations
        assert abs(kept - (1 - prob)) <= 5 * (prob * (1 - prob) / (T * d)) ** 0.5 + 2.0 ** -16
        masks.append(y != 0)
    assert (masks[1] & ~masks[0]).sum() == 0      # one generator: a larger probability drops more of the same
    rng[1] = 8
    other = moe.combine_dropout(p, o, pos, gate, torch.empty_like(o), prob=0.5, rng=rng) != 0
    same = (other == masks[1]).float().mean().item()
    assert abs(same - 0.5) <= 5 * (0.25 / (T * d)) ** 0.5
    # below half a step of 2^-16 nothing is dropped, and no generator is needed
    y = moe.combine_dropout(p, o, pos, gate, torch.empty_like(o), prob=2.0 ** -18)
    assert torch.equal(y, o)


def test_graph_replay_draws_anew_and_streams():
    m = make(dict(T=200, d=512, E=8, k=2, prob=0.3, residual=True), "bf16")
    outs = dict(y=torch.zeros((200, 512), dtype=m["dt"], device=DEV), dO=torch.zeros_like(m["o"]),
                dgate=torch.zeros((200, 2), device=DEV), dx=torch.zeros((200, 512), dtype=m["dt"], device=DEV))

    def step():
        forward(m, out=outs["y"])
        moe.combine_backward(m["p"], m["dy"], m["o"], m["pos"], m["gate"], outs["dO"], outs["dgate"], prob=m["prob"],
                             rng=m["rng"])
        moe.permute_backward(m["p"], outs["dO"], m["pos"], outs["dx"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    first = {n: v.clone() for n, v in outs.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in outs.values():
        v.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first[n], outs[n]) for n in outs)
    m["rng"][1] += 1
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first["y"], outs["y"])
    step_again = {n: v.clone() for n, v in outs.items()}
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(step_again[n], outs[n]) for n in outs)
