"""Memory of the 8-bit layer: its weights, its rows and small change. The router's
workspace, which has room for buffers of a whole layer, takes none of its own."""

import gc
import math

import pytest
import torch

import mixture_experts_layer_62_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,d,dff,E,k,dtype,pad", [(2048, 2048, 1024, 64, 8, "bf16", 0), (4096, 1024, 512, 8, 2, "f32", 0),
                                                   (1000, 1024, 1024, 16, 4, "bf16", 128)])
def test_memory_of_the_layer(T, d, dff, E, k, dtype, pad):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    n = lambda *s: (torch.randn(s, generator=g, device=DEV) / math.sqrt(s[-1])).to(dt)  # noqa: E731
    w, x = dict(W_r=n(d, E), W1=n(E, dff, d), W3=n(E, dff, d), W2=n(E, d, dff)), 8 * n(T, d)
    p = moe.problem(T, d, dff, E, k, dtype=dtype, pad_rows=pad)
    rows = moe.permuted_rows(p)
    gc.collect()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    layer = moe.MoELayerInt8(p, **w)
    taken = torch.cuda.memory_allocated() - before
    weights = 3 * E * dff * d + 4 * E * (2 * dff + d)
    behind_router = rows * (d + 4 + dff * dt.itemsize + dff + 4 + d * dt.itemsize)
    tokens = T * (d * dt.itemsize + 12 * k) + 4 * rows
    router = moe.workspace_layout(layer.router)["xp"]       # what it uses
    need = weights + max(router + behind_router, layer.router_workspace.nbytes) + tokens + layer.workspace.nbytes
    assert taken <= need + (1 << 20)
    y = layer(x).clone()

    # stage by stage, in buffers that share nothing
    new = lambda shape, t: torch.zeros(shape, dtype=t, device=DEV)  # noqa: E731
    idx, gate, pos = new((T, k), torch.int32), new((T, k), torch.float32), new((T, k), torch.int32)
    indptr, token, st = new((E + 1,), torch.int32), new((rows,), torch.int32), moe.alloc_stats(E, DEV)
    moe.route(p, x, w["W_r"], idx, gate, st, moe.alloc_workspace(p, DEV))
    xq, xs, work = new((rows, d), torch.int8), new((rows,), torch.float32), moe.alloc_int8_workspace(p, DEV)
    moe.permute_int8(p, x, idx, pos, indptr, token, xq, xs, st, work)
    h, o, out = new((rows, dff), dt), new((rows, d), dt), new((T, d), dt)
    moe.expert_up_int8(p, xq, xs, indptr, layer.W1, layer.w1s, layer.W3, layer.w3s, h, work)
    hq, hs = moe.quantize_rows(h)
    moe.expert_down_int8(p, hq, hs, indptr, layer.W2, layer.w2s, o, work)
    moe.combine_dropout(p, o, pos, gate, out)
    m = int(indptr[E])
    for a, b in ((layer.idx, idx), (layer.gate, gate), (layer.pos, pos), (layer.xq[:m], xq[:m]), (layer.xs[:m], xs[:m]),
                 (layer.h[:m], h[:m]), (layer.hq[:m], hq[:m]), (layer.hs[:m], hs[:m]), (layer.o[:m], o[:m]), (y, out)):
        assert torch.equal(a, b)
    for _ in range(3):
        assert torch.equal(layer(x), y)
    # what the router left in its workspace is still there behind the pass
    logits = torch.zeros((T, E), device=DEV)
    moe.route(p, x, w["W_r"], idx, gate, st, moe.alloc_workspace(p, DEV), logits=logits)
    assert torch.equal(moe.workspace_view(layer.router_workspace, layer.router, "logits"), logits)
