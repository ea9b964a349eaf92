"""Calls of the 8-bit experts and of the way back that the documentation allows
and the other tests do not make: rows longer than the registers of their
threads, unsigned generators, every mode of the layer, two host threads."""

import math
import threading

import pytest
import torch

import mixture_experts_layer_62_b200 as moe
import ops_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("T,k", [(5, 2), (1100, 2)])       # one launch, and three
@pytest.mark.parametrize("d,dtype", [(16448, "bf16"), (40960, "bf16"), (16400, "f32"), (33008, "f32")])
def test_permutation_of_long_rows(T, k, d, dtype):
    E, g = 6, gen(T + d)
    p = moe.problem(T, d, 64, E, k, 0.9, dtype, pad_rows=64)
    x = torch.randn((T, d), generator=g, device=DEV).to(DT[dtype])
    idx = R.routed(T, E, k, T, 0.5).to(DEV)
    rows = moe.permuted_rows(p)
    new = lambda n, t: torch.full(n, 99, dtype=t, device=DEV)  # noqa: E731
    pos, indptr, token = new((T, k), torch.int32), new((E + 1,), torch.int32), new((rows,), torch.int32)
    xq, xs = new((rows, d), torch.int8), new((rows,), torch.float32)
    moe.permute_int8(p, x, idx, pos, indptr, token, xq, xs, moe.alloc_stats(E, DEV), moe.alloc_int8_workspace(p, DEV))
    pos_r, ind_r, rt_r, _, _ = R.permutation(idx, E, R.capacity(0.9, T, k, E), 64)
    n = int(ind_r[-1])
    assert (pos.cpu().numpy() == pos_r).all() and (token[:n].cpu().numpy() == rt_r).all()
    real = torch.from_numpy(rt_r).to(DEV)
    on = real >= 0
    R.check_quantized(x[real[on]], xq[:n][on], xs[:n][on])
    assert (xq[:n][~on] == 0).all() and (xs[:n][~on] == 0).all() and (xq[n:] == 99).all() and (xs[n:] == 99).all()


def test_an_unsigned_generator():
    T, d = 30, 128
    p, g = moe.problem(T, d, 64, 1, 1), gen(1)
    o, dy = (torch.randn((T, d), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    pos, gate = torch.arange(T, dtype=torch.int32, device=DEV)[:, None].contiguous(), torch.rand((T, 1), generator=g, device=DEV)
    signed = torch.tensor([-5, 1 << 40], dtype=torch.int64, device=DEV)
    outs = []
    for rng in (signed, signed.view(torch.uint64)):
        y, dO, dg = torch.empty_like(o), torch.empty_like(o), torch.empty_like(gate)
        moe.combine_dropout(p, o, pos, gate, y, prob=0.4, rng=rng)
        moe.combine_backward(p, dy, o, pos, gate, dO, dg, prob=0.4, rng=rng)
        outs.append((y, dO, dg))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def layer_of(c, seed):
    g, dt = gen(seed), DT[c.get("dtype", "bf16")]
    T, d, dff, E, k, dfs = c["T"], c["d"], c["dff"], c["E"], c["k"], c.get("dfs", 0)
    n = lambda *s: (torch.randn(s, generator=g, device=DEV) / math.sqrt(s[-1])).to(dt)  # noqa: E731
    w = dict(W_r=n(d, E), W1=n(E, dff, d), W3=n(E, dff, d), W2=n(E, d, dff))
    if dfs:
        w |= dict(Ws1=n(dfs, d), Ws3=n(dfs, d), Ws2=n(d, dfs))
    bias = torch.rand(E, generator=g, device=DEV) * 0.2 if c.get("bias") else None
    p = moe.problem(T, d, dff, E, k, c.get("cf", 0.0), c.get("dtype", "bf16"), c.get("bias", 0), dfs, c.get("gate", 0),
                    c.get("drop", 0), pad_rows=c.get("pad", 0))
    return moe.MoELayerInt8(p, bias=bias, **w), w, bias, (n(T, d) * math.sqrt(d)).contiguous()


MODES = [dict(T=200, d=256, dff=320, E=24, k=16, cf=0.8, drop=1, pad=128, bias=moe.BIAS_PROB),
         dict(T=3, d=128, dff=64, E=5, k=1, gate=moe.GATE_FULL, dfs=64),
         dict(T=700, d=208, dff=144, E=12, k=4, cf=1.0, dtype="f32", drop=1, dfs=96, bias=moe.BIAS_LOGIT),
         dict(T=64, d=16, dff=16, E=3, k=2, dtype="f32", pad=64, gate=moe.GATE_FULL),
         dict(T=2600, d=512, dff=1024, E=2, k=2, cf=0.7)]


@pytest.mark.parametrize("c", MODES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_the_layer_is_its_stages(c):
    layer, w, bias, x = layer_of(c, c["T"])
    p, T, d, E, k, dt = layer.p, c["T"], c["d"], c["E"], c["k"], DT[c.get("dtype", "bf16")]
    residual = x.flip(0).contiguous()
    out = torch.full((T, d), 3.0, dtype=dt, device=DEV)
    assert layer(x, out=out, residual=residual) is out
    assert layer.read_stats().status == moe.MOE_OK
    q, rows = layer.experts, moe.permuted_rows(layer.experts)
    new = lambda shape, t: torch.full(shape, 77, dtype=t, device=DEV)  # noqa: E731
    idx, gate, pos = new((T, k), torch.int32), new((T, k), torch.float32), new((T, k), torch.int32)
    indptr, token, st = new((E + 1,), torch.int32), new((rows,), torch.int32), moe.alloc_stats(E, DEV)
    moe.route(p, x, w["W_r"], idx, gate, st, moe.alloc_workspace(p, DEV), bias=bias)
    xq, xs, work = new((rows, d), torch.int8), new((rows,), torch.float32), moe.alloc_int8_workspace(q, DEV)
    moe.permute_int8(q, x, idx, pos, indptr, token, xq, xs, st, work)
    W1, W3, W2 = (moe.quantize_rows(w[n]) for n in ("W1", "W3", "W2"))
    h, o = new((rows, c["dff"]), dt), new((rows, d), dt)
    moe.expert_up_int8(q, xq, xs, indptr, *W1, *W3, h, work)
    hq, hs = moe.quantize_rows(h, used=indptr[E:])
    moe.expert_down_int8(q, hq, hs, indptr, *W2, o, work)
    s = None
    if c.get("dfs"):
        f = c["dfs"]
        one, ends = moe.problem(T, d, f, 1, 1, dtype=c.get("dtype", "bf16")), torch.tensor([0, T], dtype=torch.int32, device=DEV)
        sw, sh, s = moe.alloc_int8_workspace(one, DEV), new((T, f), dt), new((T, d), dt)
        moe.expert_up_int8(one, *moe.quantize_rows(x), ends, *moe.quantize_rows(w["Ws1"]), *moe.quantize_rows(w["Ws3"]), sh, sw)
        moe.expert_down_int8(one, *moe.quantize_rows(sh), ends, *moe.quantize_rows(w["Ws2"]), s, sw)
    y = new((T, d), dt)
    moe.combine_dropout(q, o, pos, gate, y, s=s, residual=residual)
    assert torch.equal(y, out)
    # in place over the residual
    layer(x, out=residual, residual=residual)
    assert torch.equal(residual, out)


def test_two_host_threads():
    cases = (MODES[0], MODES[4])
    layers = [layer_of(c, 7 + i) for i, c in enumerate(cases)]
    want = [layer(x).clone() for layer, _, _, x in layers]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        layer, _, _, x = layers[i]
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(60):
                y = layer(x)
                stream.synchronize()
                if not torch.equal(y, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and all(layer.read_stats().status == moe.MOE_OK for layer, _, _, _ in layers)


def test_no_tokens():
    # (the tensors have a row each: pointers are checked before anything else)
    E, d, dff = 4, 64, 128
    p = moe.problem(0, d, dff, E, 2)
    one = lambda *s, t=torch.int32: torch.full(s, 3, dtype=t, device=DEV)  # noqa: E731
    x, h, o = (one(1, n, t=torch.bfloat16) for n in (d, dff, d))
    indptr, st, work = one(E + 1), moe.alloc_stats(E, DEV), moe.alloc_int8_workspace(p, DEV)
    st.fill_(255)
    q, s = one(1, d, t=torch.int8), one(1, t=torch.float32)
    moe.permute_int8(p, x, one(1, 2), one(1, 2), indptr, one(2), q, s, st, work)
    W, V, a, b = one(E, dff, d, t=torch.int8), one(E, d, dff, t=torch.int8), torch.ones((E, dff), device=DEV), torch.ones((E, d), device=DEV)
    moe.expert_up_int8(p, q, s, indptr, W, a, W, a, h, work)
    moe.expert_down_int8(p, one(1, dff, t=torch.int8), s, indptr, V, b, o, work)
    moe.quantize_rows(h[:0], one(1, dff, t=torch.int8), s)
    assert (indptr == 0).all() and (h == 3).all() and (o == 3).all() and (q == 3).all() and (s == 3).all()
    got = moe.read_stats(st, E)
    assert got.status == moe.MOE_OK and got.rows == got.dropped == got.max_count == 0 and not any(got.counts)
