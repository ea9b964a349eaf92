"""8-bit experts on the GPU: quantisation, permutation and products against
64-bit plain forms (tests/ops_ref.py)."""

import math

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


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def ints(g, *shape):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)


# ---- quantisation -------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 2048), (5, 2064), (7, 4096), (130, 8192), (9, 8208), (4, 14336),
                                       (3, 16400), (2, 131072), (2000, 208)])
def test_quantize_rows(rows, cols, dtype):
    g = gen(rows * 7 + cols)
    x = randn(g, rows, cols) * torch.exp(4 * randn(g, rows, 1))
    x = x.to(DT[dtype])
    q, s = moe.quantize_rows(x)
    R.check_quantized(x, q, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_rows_at_the_borders(dtype):
    # whole rows of exact ties and of values one step of the type beside them:
    # a = 127 2^e makes the steps whole, so x = m + 1/2 are ties
    rows = []
    for scale in (1.0, 2.0 ** -30, 2.0 ** 20):
        ties = torch.tensor([127.0] + [m + 0.5 for m in range(-63, 63)] + [-127.0])
        rows += [ties * scale]
    # a = 1: 127 x is a tie at x = (m + 1/2) / 127, not representable; its two neighbours in the type
    near = torch.tensor([(m + 0.5) / 127 for m in range(-63, 63)], dtype=torch.float64).to(DT[dtype]).float()
    one = torch.ones(1)
    rows += [torch.cat([one, near, -one])]
    up = torch.nextafter(near, torch.full_like(near, 9.0)) if dtype == "f32" else near
    rows += [torch.cat([one, up, -one])]
    # maxima that are no powers of two
    g = torch.Generator().manual_seed(3)
    for _ in range(40):
        a = torch.rand(1, generator=g) + 0.5
        m = torch.randint(-127, 127, (126,), generator=g).double() + 0.5
        rows += [torch.cat([a, (m * a.double() / 127).float().clamp(-a.item(), a.item()), -a])]
    x = torch.stack([r.to(DT[dtype]) for r in rows]).to(DEV)
    q, s = moe.quantize_rows(x)
    R.check_quantized(x, q, s)


def test_quantize_rows_tiny_zero_and_unused_rows():
    x = torch.zeros((6, 48), device=DEV)
    x[1, 3] = 2.0 ** -101          # below the floor: a row of zeros
    x[2, 5] = 2.0 ** -100          # on it
    x[3] = 3.0e38                  # the largest values
    x[4:] = float("nan")           # rows that nobody uses may hold anything
    q = torch.full((6, 48), 77, dtype=torch.int8, device=DEV)
    s = torch.full((6,), 5.0, device=DEV)
    moe.quantize_rows(x, q, s, used=torch.tensor([4], dtype=torch.int32, device=DEV))
    R.check_quantized(x[:4], q[:4], s[:4])
    assert q[1].abs().max() == 0 and s[1] == 0 and q[2, 5] == 127 and (q[3] == 127).all()
    assert (q[4:] == 77).all() and (s[4:] == 5.0).all()
    # used past the rows, and none used
    moe.quantize_rows(x[:4], q, s, used=torch.tensor([900], dtype=torch.int32, device=DEV))
    R.check_quantized(x[:4], q[:4], s[:4])
    q.fill_(9)
    moe.quantize_rows(x, q, s, used=torch.tensor([0], dtype=torch.int32, device=DEV))
    assert (q == 9).all()


# ---- permutation --------------------------------------------------------------

PERM = [dict(T=1, E=8, k=2), dict(T=1, E=1, k=1), dict(T=3, E=5, k=5), dict(T=31, E=7, k=3, cf=0.8),
        dict(T=200, E=8, k=2, cf=1.0, drop=1), dict(T=257, E=16, k=4, pad=64, skew=1.5),
        dict(T=64, E=512, k=16, pad=128, cf=1.0), dict(T=900, E=9, k=8, pad=128, drop=1, cf=0.7),
        dict(T=3000, E=64, k=8, cf=1.2, skew=1.0), dict(T=5000, E=3, k=1), dict(T=1025, E=4, k=2, drop=1, cf=0.5, pad=64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", PERM, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_permute_int8(c, dtype):
    T, E, k = c["T"], c["E"], c["k"]
    d = 192 if dtype == "bf16" else 208
    p = moe.problem(T, d, 64, E, k, c.get("cf", 0.0), dtype, drop_order=c.get("drop", 0), pad_rows=c.get("pad", 0))
    g = gen(T + E)
    x = (randn(g, T, d) * torch.exp(randn(g, T, 1))).to(DT[dtype])
    idx = R.routed(T, E, k, T * 31 + E, c.get("skew", 0.0))
    if T > 2:
        idx[1] = idx[1, 0]          # the same expert in every slot of a token
        idx[2, 0] = -1              # not an expert: the pair takes no row
    idx = idx.to(DEV)
    N = moe.permuted_rows(p)
    pos = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    indptr = torch.full((E + 1,), -7, dtype=torch.int32, device=DEV)
    rt = torch.full((N,), -7, dtype=torch.int32, device=DEV)
    xq = torch.full((N, d), 99, dtype=torch.int8, device=DEV)
    xs = torch.full((N,), -3.0, device=DEV)
    st, ws = moe.alloc_stats(E, DEV), moe.alloc_int8_workspace(p, DEV)
    st.fill_(255)
    ws.fill_(255)
    moe.permute_int8(p, x, idx, pos, indptr, rt, xq, xs, st, ws)
    cap = R.capacity(c.get("cf", 0.0), T, k, E)
    pos_r, ind_r, rt_r, kept, count = R.permutation(idx, E, cap, c.get("pad", 0), bool(c.get("drop", 0)))
    assert (pos.cpu().numpy() == pos_r).all()
    assert (indptr.cpu().numpy() == ind_r).all()
    n = int(ind_r[-1])
    assert (rt[:n].cpu().numpy() == rt_r).all()
    assert (rt[n:] == -7).all() and (xq[n:] == 99).all() and (xs[n:] == -3.0).all()
    real = torch.from_numpy(rt_r).to(DEV)
    on = real >= 0
    R.check_quantized(x[real[on]], xq[:n][on], xs[:n][on])
    assert (xq[:n][~on] == 0).all() and (xs[:n][~on] == 0).all()
    s = moe.read_stats(st, E)
    assert s.status == 0 and s.kept == kept.tolist() and s.counts == count.tolist()
    assert s.rows == int(kept.sum()) and s.dropped == int((count - kept).sum()) and s.max_count == int(count.max())
    assert s.capacity == (-1 if cap is None else cap)


# ---- products -----------------------------------------------------------------

def split(total, E, g):
    """Random group ends with empty groups among them."""
    cut = torch.randint(0, total + 1, (E - 1,), generator=torch.Generator().manual_seed(g)).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.long), cut, torch.tensor([total])]).to(torch.int32)


def run_products(T, d, dff, E, k, dtype, indptr, g, ws_fill=255, stats=True, scale_a=None):
    """Both products over given groups; results against the plain form."""
    p = moe.problem(T, d, dff, E, k, 0.0, dtype)
    N, dt = moe.permuted_rows(p), DT[dtype]
    indptr = indptr.to(DEV)
    n = int(indptr[-1])
    ws = moe.alloc_int8_workspace(p, DEV)
    ws.fill_(ws_fill)
    st = moe.alloc_stats(E, DEV)
    st.fill_(255)
    xq, hq = ints(g, N, d), ints(g, N, dff)
    # scales that give pre-activations around 1, and some far out
    xs = torch.rand((N,), generator=g, device=DEV) * (4.0 / (74 * 74 * math.sqrt(d)))
    xs[::5] *= 30
    hs = torch.rand((N,), generator=g, device=DEV) / (74 * 74 * math.sqrt(dff))
    W1, W3, W2 = ints(g, E, dff, d), ints(g, E, dff, d), ints(g, E, d, dff)
    w1s, w3s, w2s = (0.5 + torch.rand((E, m), generator=g, device=DEV) for m in (dff, dff, d))
    xs[n:] = float("nan")    # rows of no group: whatever they hold is not looked at
    hs[n:] = float("nan")
    h = torch.full((N, dff), 7.0, dtype=dt, device=DEV)
    o = torch.full((N, d), 7.0, dtype=dt, device=DEV)
    moe.expert_up_int8(p, xq, xs, indptr, W1, w1s, W3, w3s, h, ws, stats=st if stats else None)
    if stats:
        assert moe.read_stats(st, E).status == moe.MOE_OK
        st.fill_(255)
    moe.expert_down_int8(p, hq, hs, indptr, W2, w2s, o, ws, stats=st if stats else None)
    if stats:
        assert moe.read_stats(st, E).status == moe.MOE_OK
    a, b = R.product(xq[:n], xs[:n], W1, w1s, indptr), R.product(xq[:n], xs[:n], W3, w3s, indptr)
    ref = R.swiglu(a, b)
    assert ((h[:n].double() - ref).abs() <= R.swiglu_bound(a, b, dt)).all()
    ref = R.product(hq[:n], hs[:n], W2, w2s, indptr)
    assert ((o[:n].double() - ref).abs() <= R.plain_bound(ref, dt)).all()
    assert (h[n:] == 7.0).all() and (o[n:] == 7.0).all()
    return h, o


SMALL = [(1, 64, 64, 1, 1), (1, 128, 192, 8, 2), (4, 256, 448, 8, 2), (5, 1088, 320, 4, 2), (9, 64, 2048, 3, 3),
         (16, 512, 512, 8, 2), (33, 192, 128, 2, 2), (40, 4096, 1024, 8, 2), (100, 256, 256, 16, 4),
         (250, 320, 576, 8, 2), (300, 64, 64, 64, 8)]
LARGE = [(1024, 512, 256, 4, 2), (2000, 192, 448, 8, 2), (700, 1024, 640, 1, 1), (3000, 256, 320, 5, 1),
         (513, 2048, 1408, 2, 2)]


@pytest.mark.parametrize("T,d,dff,E,k", SMALL + LARGE)
def test_products_bf16(T, d, dff, E, k):
    g = gen(T * 3 + d)
    for s in range(2):
        run_products(T, d, dff, E, k, "bf16", split(T * k, E, s + T), g, stats=s == 0)
    if k == 1 or E > 1:
        one = torch.zeros(E + 1, dtype=torch.int32)
        one[E // 2 + 1:] = T * k    # every row in one group
        run_products(T, d, dff, E, k, "bf16", one, g, ws_fill=0)


@pytest.mark.parametrize("T,d,dff,E,k", [(1, 16, 16, 1, 1), (3, 48, 80, 2, 2), (77, 208, 336, 5, 3), (8, 1040, 272, 4, 1),
                                         (600, 144, 176, 3, 2), (1500, 400, 240, 2, 2)])
def test_products_f32(T, d, dff, E, k):
    g = gen(T + dff)
    run_products(T, d, dff, E, k, "f32", split(T * k, E, T), g)
    if k == 1 or E > 1:
        short = split(T * k, E, T + 1).clamp(max=T * k // 2)   # half of the rows in no group
        run_products(T, d, dff, E, k, "f32", short, g)


def test_products_without_rows():
    g = gen(1)
    for T in (1, 9, 600):
        run_products(T, 128, 64, 4, 2, "bf16", torch.zeros(5, dtype=torch.int32), g)


@pytest.mark.parametrize("rows", [1, 3, 12, 140, 400])
def test_products_at_the_largest_sums(rows):
    # every product (-128)^2 over the longest K that is taken: the sums reach 2^31 - 2^14 or so
    K, N = 131056, 16
    p = moe.problem(rows, N, K, 1, 1, 0.0, "f32")
    ws = moe.alloc_int8_workspace(p, DEV)
    hq = torch.full((rows, K), -128, dtype=torch.int8, device=DEV)
    W2 = torch.full((1, N, K), -128, dtype=torch.int8, device=DEV)
    W2[0, 1] = 127
    hs = torch.ones(rows, device=DEV)
    o = torch.zeros((rows, N), device=DEV)
    moe.expert_down_int8(p, hq, hs, torch.tensor([0, rows], dtype=torch.int32, device=DEV), W2,
                         torch.ones((1, N), device=DEV), o, ws)
    want = torch.full((rows, N), float(K) * 128 * 128, device=DEV)
    want[:, 1] = -float(K) * 128 * 127
    assert torch.equal(o, want.to(torch.float64).float())


@pytest.mark.parametrize("T", [2, 60, 900])
def test_products_are_the_same_bits_again(T):
    a = run_products(T, 256, 320, 4, 2, "bf16", split(T * 2, 4, 5), gen(11))
    b = run_products(T, 256, 320, 4, 2, "bf16", split(T * 2, 4, 5), gen(11), ws_fill=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_products_past_32_bit_offsets():
    # W1 / W3 beyond 2^31 bytes, rows of the last expert among them; plain form on that expert alone
    E, dff, d, T = 40, 8192, 8192, 3
    p = moe.problem(T, d, dff, E, 1, 0.0, "bf16")
    g = gen(2)
    W = torch.zeros((E, dff, d), dtype=torch.int8, device=DEV)
    W[E - 1] = ints(g, dff, d)
    ws_ = torch.ones((E, dff), device=DEV)
    xq, xs = ints(g, T, d), torch.full((T,), 1.0 / (74 * 74 * 90), device=DEV)
    indptr = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    indptr[E] = T
    h = torch.zeros((T, dff), dtype=torch.bfloat16, device=DEV)
    moe.expert_up_int8(p, xq, xs, indptr, W, ws_, W, ws_, h, moe.alloc_int8_workspace(p, DEV))
    a = R.product(xq, xs, W[E - 1:], ws_[:1], torch.tensor([0, T]))
    assert ((h.double() - R.swiglu(a, a)).abs() <= R.swiglu_bound(a, a, torch.bfloat16)).all()


# ---- the chain, streams and graphs ------------------------------------------------

def layer_inputs(T, d, dff, E, k, seed, dfs=0):
    g = gen(seed)
    n = lambda *s: (randn(g, *s) / math.sqrt(s[-1])).to(torch.bfloat16)  # noqa: E731
    w = dict(W_r=(randn(g, d, E) / math.sqrt(d)).to(torch.bfloat16), W1=n(E, dff, d), W3=n(E, dff, d), W2=n(E, d, dff))
    if dfs:
        w |= dict(Ws1=n(dfs, d), Ws3=n(dfs, d), Ws2=n(d, dfs))
    return randn(g, T, d).to(torch.bfloat16), w


LAYERS = [dict(T=1, d=256, dff=512, E=8, k=2), dict(T=40, d=512, dff=320, E=16, k=4, cf=0.9, pad=64),
          dict(T=700, d=256, dff=448, E=4, k=2, dfs=192, bias=True), dict(T=1500, d=1024, dff=1536, E=2, k=1, cf=1.1)]


@pytest.mark.parametrize("c", LAYERS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_layer_stage_by_stage(c):
    T, d, dff, E, k, dfs = c["T"], c["d"], c["dff"], c["E"], c["k"], c.get("dfs", 0)
    x, w = layer_inputs(T, d, dff, E, k, 3, dfs)
    bias = torch.linspace(0.4, -0.4, E, device=DEV) if c.get("bias") else None
    p = moe.problem(T, d, dff, E, k, c.get("cf", 0.0), "bf16", bias_mode=moe.BIAS_LOGIT if c.get("bias") else 0,
                    d_ff_shared=dfs, pad_rows=c.get("pad", 0))
    layer = moe.MoELayerInt8(p, bias=bias, **w)
    residual = torch.randn((T, d), device=DEV).to(torch.bfloat16)
    y = layer(x, residual=residual)
    st = layer.read_stats()
    assert st.status == moe.MOE_OK
    # the routing is moe_route's, and the statistics are whole
    idx, gate, stats = torch.empty_like(layer.idx), torch.empty_like(layer.gate), moe.alloc_stats(E, DEV)
    moe.route(p, x, w["W_r"], idx, gate, stats, moe.alloc_workspace(p, DEV), bias=bias)
    assert torch.equal(idx, layer.idx) and torch.equal(gate, layer.gate)
    ref = moe.read_stats(stats, E)
    assert (st.counts, st.kept, st.l_aux, st.P, st.dropped) == (ref.counts, ref.kept, ref.l_aux, ref.P, ref.dropped)
    for q, s, W in ((layer.W1, layer.w1s, w["W1"]), (layer.W2, layer.w2s, w["W2"])):
        R.check_quantized(W.reshape(-1, W.shape[-1]), q.reshape(-1, W.shape[-1]), s.reshape(-1))
    pos, indptr, rt, _, _ = R.permutation(idx, E, R.capacity(c.get("cf", 0.0), T, k, E), c.get("pad", 0))
    n = int(indptr[-1])
    rt = torch.from_numpy(rt).to(DEV)
    assert (layer.pos.cpu().numpy() == pos).all()
    R.check_quantized(x[rt[rt >= 0]], layer.xq[:n][rt >= 0], layer.xs[:n][rt >= 0])
    a = R.product(layer.xq[:n], layer.xs[:n], layer.W1, layer.w1s, indptr)
    b = R.product(layer.xq[:n], layer.xs[:n], layer.W3, layer.w3s, indptr)
    assert ((layer.h[:n].double() - R.swiglu(a, b)).abs() <= R.swiglu_bound(a, b, torch.bfloat16)).all()
    R.check_quantized(layer.h[:n], layer.hq[:n], layer.hs[:n])
    o = R.product(layer.hq[:n], layer.hs[:n], layer.W2, layer.w2s, indptr)
    assert ((layer.o[:n].double() - o).abs() <= R.plain_bound(o, torch.bfloat16)).all()
    s = None
    if dfs:
        g, one = layer.shared, torch.tensor([0, T])
        R.check_quantized(x, *g["x"])
        a, b = (R.product(*g["x"], g[m][0][None], g[m][1][None], one) for m in ("W1", "W3"))
        assert ((g["h"].double() - R.swiglu(a, b)).abs() <= R.swiglu_bound(a, b, torch.bfloat16)).all()
        R.check_quantized(g["h"], *g["hq"])
        s = R.product(*g["hq"], g["W2"][0][None], g["W2"][1][None], one)
        assert ((g["s"].double() - s).abs() <= R.plain_bound(s, torch.bfloat16)).all()
        s = g["s"]
    ref, mag = R.mix(layer.o, layer.pos, layer.gate, s, residual)
    assert ((y.double() - ref).abs() <= R.mix_bound(ref, mag, k, torch.bfloat16)).all()


def test_layer_is_near_the_layer_in_bf16():
    # each of the three products has two factors in 8 bits; a factor's error is
    # at most half a step, uniform in a step of amax / 127: for normal data of
    # these lengths amax is at most 4.5 sigma, so the relative error of one
    # factor is at most 4.5 / (127 sqrt(12)) = 1.03 % rms. Two factors a
    # product, and the down projection sees the up projections' through SiLU(a)
    # b, at most 2.1 x one product's: sqrt(2 + (2.1^2) 2) x 1.03 % = 3.4 %, plus
    # bf16's roundings. The bar is 6 %; a wrong scale or row is off by tens of
    # percent or more.
    T, d, dff, E, k = 300, 512, 1024, 8, 2
    x, w = layer_inputs(T, d, dff, E, k, 9)
    p = moe.problem(T, d, dff, E, k)
    a, b = moe.MoELayer(p, **w)(x).double(), moe.MoELayerInt8(p, **w)(x).double()
    assert (a - b).norm() / a.norm() < 0.06


def test_layer_in_graphs_that_share_buffers():
    T, d, dff, E, k = 24, 256, 512, 8, 2
    x, w = layer_inputs(T, d, dff, E, k, 4)
    layer = moe.MoELayerInt8(moe.problem(T, d, dff, E, k), **w)
    outs = [torch.zeros((T, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    xs = [x.clone(), x.flip(0).contiguous()]
    want = []
    for i in range(2):
        want.append(layer(xs[i]).clone())
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer(xs[i], out=outs[i])
        graphs.append(g)
    layer.workspace.fill_(0x5A)      # the workspace's contents are nobody's
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            assert torch.equal(outs[i], want[i])
    xs[0].copy_(xs[1])               # a replay reads what the inputs hold then
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])


def test_two_streams_at_once():
    T, d, dff, E, k = 400, 512, 1024, 8, 2
    x, w = layer_inputs(T, d, dff, E, k, 5)
    layers = [moe.MoELayerInt8(moe.problem(T, d, dff, E, k), **w) for _ in range(2)]
    xs = [x, (x.float() * 0.5).flip(1).to(torch.bfloat16).contiguous()]
    want = [layers[i](xs[i]).clone() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            layers[i].out.zero_()
            streams[i].wait_stream(torch.cuda.current_stream())
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                layers[i](xs[i])
        torch.cuda.synchronize()
        assert all(torch.equal(layers[i].out, want[i]) for i in range(2))
    # and given as an argument, from another current stream
    layers[0].out.zero_()
    streams[1].wait_stream(torch.cuda.current_stream())
    layers[0](xs[0], stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(layers[0].out, want[0])


def test_variants_by_size():
    v = lambda T, d, dff, E, k: (moe.int8_variant(moe.problem(T, d, dff, E, k)),  # noqa: E731
                                 moe.int8_variant(moe.problem(T, d, dff, E, k), down=True))
    assert v(1, 4096, 14336, 8, 2) == ("single", "single")
    assert v(4096, 4096, 14336, 8, 2) == ("pair", "pair")
    assert v(1024, 4096, 14336, 8, 2) == ("pair", "pair")
    assert v(448, 4096, 14336, 8, 2) == ("single", "single")     # 112 rows an expert
    assert v(1500, 1024, 2048, 8, 2) == ("single", "single")     # 375 rows, short K
    assert v(4000, 640, 2048, 24, 3) == ("single", "single")     # 500 rows; 640 channels fill 5/8 of their tiles
    assert v(2048, 7168, 2048, 256, 8) == ("single", "single")


@pytest.mark.parametrize("T,d,dff,E,k", [(2000, 512, 4096, 2, 1), (4000, 512, 8192, 4, 1), (3000, 4096, 1088, 2, 2)])
def test_products_in_pairs(T, d, dff, E, k):
    # sizes whose products run on CTA pairs: whole tiles, ragged ends of every kind, empty groups
    p = moe.problem(T, d, dff, E, k)
    assert "pair" in (moe.int8_variant(p), moe.int8_variant(p, down=True))
    R_ = T * k
    for cut in ([R_], [1], [R_ - 31], [256], [R_ // 2 + 7], [0]):
        ends = torch.tensor([0] + [min(cut[0], R_)] * (E - 1) + [R_], dtype=torch.int32)
        run_products(T, d, dff, E, k, "bf16", ends, gen(cut[0] + 1))


@pytest.mark.parametrize("n", [192, 193, 223, 224, 225, 255, 256, 257, 449, 511])
def test_products_in_pairs_by_last_block(n):
    # groups whose last block is the largest short one, a whole one with a ragged stretch of 32 rows, a full one
    T, d, dff, E = 1600, 512, 8192, 2
    p = moe.problem(T, d, dff, E, 1)
    assert moe.int8_variant(p) == "pair"
    run_products(T, d, dff, E, 1, "bf16", torch.tensor([0, n, n + 512 + n % 32], dtype=torch.int32), gen(n))


@pytest.mark.parametrize("T,d,dff,E,k", [
    (40, 256, 8192, 1, 1),       # one or two tiles, K in 16 shares
    (40, 192, 8192, 3, 1),       # the same, the last 64 channels of 256 alone in their half
    (65, 320, 4096, 2, 1),       # more than 64 rows
    (60, 8192, 4096, 4, 1),      # 128 tiles of a 148th each: not cut
    (260, 1024, 1408, 2, 1),     # tall tiles, short K: not cut
    (300, 2432, 2560, 2, 1),     # whole tiles and a tail
])
def test_products_by_their_tail(T, d, dff, E, k):
    for s in (0, 1):
        run_products(T, d, dff, E, k, "bf16", split(T * k, E, s), gen(T + s), ws_fill=255 * s)


def test_products_in_pairs_f32():
    T, d, dff, E = 1700, 1040, 4112, 2
    p = moe.problem(T, d, dff, E, 1, 0.0, "f32")
    assert moe.int8_variant(p) == "pair"
    for cut in (1, 850, 1699):
        run_products(T, d, dff, E, 1, "f32", torch.tensor([0, cut, T], dtype=torch.int32), gen(cut))


def test_bad_offsets_are_left_out():
    # offsets that do not fit the rows: those groups are skipped, the others run
    T, d, E, dff = 64, 128, 4, 192
    p = moe.problem(T, d, dff, E, 1)
    g = gen(8)
    q, s, W, ws_ = ints(g, T, dff), torch.rand((T,), generator=g, device=DEV), ints(g, E, d, dff), torch.ones((E, d), device=DEV)
    o = torch.full((T, d), 7.0, dtype=torch.bfloat16, device=DEV)
    indptr = torch.tensor([0, 20, 70, 30, 64], dtype=torch.int32, device=DEV)   # 1 ends past the rows, 2 runs backwards
    moe.expert_down_int8(p, q, s, indptr, W, ws_, o, moe.alloc_int8_workspace(p, DEV))
    for e, lo, hi in ((0, 0, 20), (3, 30, 64)):
        r = (q[lo:hi].double() @ W[e].double().T) * s[lo:hi, None].double()
        assert ((o[lo:hi].double() - r).abs() <= R.plain_bound(r, torch.bfloat16)).all()
    assert (o[20:30] == 7.0).all()


def test_calls_wait_for_what_comes_before_them():
    # the kernels start early beside the work before them; what they read has
    # to be there all the same: behind a slow producer on their own stream, on
    # another one (an event between them), and in a graph with a fork and a join
    g = gen(3)
    rows, cols, N = 300, 2048, 512
    src = randn(g, rows, cols).to(torch.bfloat16)
    x, q, s = torch.zeros_like(src), torch.zeros((rows, cols), dtype=torch.int8, device=DEV), torch.zeros(rows, device=DEV)
    W, ws_ = ints(g, 1, N, cols), torch.ones((1, N), device=DEV)
    p = moe.problem(rows, N, cols, 1, 1)
    work, o = moe.alloc_int8_workspace(p, DEV), torch.zeros((rows, N), dtype=torch.bfloat16, device=DEV)
    indptr = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    moe.quantize_rows(src, q, s)
    moe.expert_down_int8(p, q, s, indptr, W, ws_, o, work)
    torch.cuda.synchronize()
    want = [t.clone() for t in (q, s, o)]

    def consume():
        moe.quantize_rows(x, q, s)
        moe.expert_down_int8(p, q, s, indptr, W, ws_, o, work)

    def produce():
        torch.cuda._sleep(2_000_000)    # about a millisecond
        x.copy_(src)

    def check():
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((q, s, o), want))
        for t in (x, q, s, o):
            t.zero_()
        torch.cuda.synchronize()

    other = torch.cuda.Stream()
    check()
    for _ in range(3):
        produce()
        consume()
        check()
        moe.quantize_rows(src, q, s)    # a kernel of the library's own before the wait for the event
        with torch.cuda.stream(other):
            produce()
            done = other.record_event()
        torch.cuda.current_stream().wait_event(done)
        consume()
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        fork = main.record_event()
        other.wait_event(fork)
        with torch.cuda.stream(other):
            produce()
            done = other.record_event()
        moe.quantize_rows(src, q, s)
        main.wait_event(done)
        consume()
    for _ in range(3):
        graph.replay()
        check()


@pytest.mark.parametrize("T", [500, 3000])
def test_permutation_waits_for_what_comes_before_it(T):
    # its rows are read early: behind a slow producer, and right behind a kernel of the library that writes them
    g = gen(T)
    d, E, k = 256, 8, 2
    p = moe.problem(T, d, 64, E, k)
    src, idx = randn(g, T, d).to(torch.bfloat16), R.routed(T, E, k, T, 0.5).to(torch.int32).to(DEV)
    rows = moe.permuted_rows(p)
    x, dead = torch.zeros_like(src), torch.zeros((T, d), dtype=torch.int8, device=DEV)
    pos, indptr = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty(E + 1, dtype=torch.int32, device=DEV)
    row_token = torch.empty(rows, dtype=torch.int32, device=DEV)
    xq, xs = torch.zeros((rows, d), dtype=torch.int8, device=DEV), torch.zeros(rows, device=DEV)
    work, st = moe.alloc_int8_workspace(p, DEV), moe.alloc_stats(E, DEV)
    # as one expert of one slot and gate 1, the way back copies its rows
    one = moe.problem(T, d, 64, 1, 1)
    at, gate = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1), torch.ones((T, 1), device=DEV)

    def permute():
        moe.permute_int8(p, x, idx, pos, indptr, row_token, xq, xs, st, work)

    x.copy_(src)
    permute()
    torch.cuda.synchronize()
    want = xq.clone(), xs.clone()
    for slow in (False, True, True):
        for t in (x, xq, xs):
            t.zero_()
        torch.cuda.synchronize()
        if slow:
            torch.cuda._sleep(2_000_000)
            moe.quantize_rows(src, dead, torch.empty(T, device=DEV))
        moe.combine_dropout(one, src, at, gate, x)
        permute()
        torch.cuda.synchronize()
        assert torch.equal(x, src) and torch.equal(xq, want[0]) and torch.equal(xs, want[1])


def test_binding_takes_what_is_right_and_nothing_else():
    b, g = moe._bound(), gen(4)
    x = randn(g, 8, 64).to(torch.bfloat16)
    q, s = torch.zeros((8, 64), dtype=torch.int8, device=DEV), torch.zeros(8, device=DEV)
    want = moe.quantize_rows(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream, 0):
        q.zero_(), s.zero_()
        torch.cuda.synchronize()
        assert b.quantize_rows(x, q, s, None, stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(q, want[0]) and torch.equal(s, want[1])
    q.zero_()
    for bad in ((x.cpu(), q, s), (x, q.cpu(), s), (x, q[:7], s), (x, q, s[:7]), (x, q, s.double()), (x.t(), q, s),
                (x, q.t(), s), (x, q.view(torch.uint8), s), (x.half(), q, s)):
        assert b.quantize_rows(*bad, None, None) is None
    assert b.quantize_rows(x, q, s, torch.zeros(1, device=DEV), None) is None
    # the library's own refusals come through as its codes
    assert b.quantize_rows(x.view(-1)[:504].view(8, 63), q, s, None, None) == moe.MOE_ERR_UNSUPPORTED
    assert b.quantize_rows(x.view(-1)[4:68].view(1, 64), q, s, None, None) == moe.MOE_ERR_INVALID_ARG   # 8 bytes off
    torch.cuda.synchronize()
    assert not q.any()
