"""Plain 64-bit forms of the operators beside the layer, and the bounds their
results are held to. Everything is torch in float64 / int64 on the inputs'
device; nothing of the library is used."""

import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step of the type, relative
U = 2.0 ** -24                                                  # one fp32 rounding


def permutation(idx, E, cap, pad=0, slot=False):
    """pos [T, k], indptr [E + 1], row_token [rows], kept [E] by counting, pair after pair."""
    T, k = idx.shape
    ids = idx.cpu().numpy()
    order = [(t, j) for j in range(k) for t in range(T)] if slot else [(t, j) for t in range(T) for j in range(k)]
    count = [0] * E
    rank = {}
    for t, j in order:
        e = int(ids[t, j])
        if 0 <= e < E:
            rank[t, j] = count[e]
            count[e] += 1
    kept = [c if cap is None else min(c, cap) for c in count]
    held = [-(-c // pad) * pad if pad else c for c in kept]
    indptr = np.concatenate([[0], np.cumsum(held)]).astype(np.int64)
    pos = np.full((T, k), -1, dtype=np.int64)
    row_token = np.full(int(indptr[-1]), -1, dtype=np.int64)
    # rows keep token order inside an expert under both drop orders' ranks
    for (t, j), r in rank.items():
        e = int(ids[t, j])
        if r < kept[e]:
            pos[t, j] = indptr[e] + r
            row_token[indptr[e] + r] = t
    return pos, indptr, row_token, np.array(kept), np.array(count)


def check_quantized(x, q, scale):
    """q and scale are the definition's for x, decided exactly: 254 x and
    2 q a are exact in float64 (at most 24 + 8 bits), so is their comparison
    with a; ties must have gone to the even whole number."""
    X = x.double()
    a = X.abs().amax(1)
    live = a >= 2.0 ** -100
    af = a.float()
    assert torch.equal(scale, torch.where(live, af / torch.full_like(af, 127.0), torch.zeros_like(af)))
    Q = q.double()
    assert (Q[~live] == 0).all()
    off = (254.0 * X - 2.0 * Q * a[:, None])[live]
    al = a[live][:, None].expand_as(off)
    assert (off.abs() <= al).all(), "not the nearest whole number"
    tie = off.abs() == al
    assert (q.long()[live][tie] % 2 == 0).all(), "a tie went to the odd number"


def product(q, s, W, ws, indptr):
    """Exact integer sums times the scales, per group, in float64 [rows, N]."""
    E, N, K = W.shape
    out = torch.zeros((q.shape[0], N), dtype=torch.float64, device=q.device)
    for e in range(E):
        lo, hi = int(indptr[e]), int(indptr[e + 1])
        if hi > lo:
            # float64 products of whole numbers: exact below 2^53
            out[lo:hi] = (q[lo:hi].double() @ W[e].double().T) * s[lo:hi, None].double() * ws[e][None, :].double()
    return out


def swiglu(a, b):
    return a * torch.sigmoid(a) * b


def plain_bound(ref, dtype):
    """float(sum) sa sb: one rounding of the sum and two of the products, then the type's."""
    return ref.abs() * (HALF[dtype] + 4 * U) + 1e-30


def swiglu_bound(a, b, dtype):
    """a and b carry 3 roundings each (plain_bound). SiLU(a) = a / (1 + exp(-a))
    passes a relative error of a on with a factor of at most 1 + |a|. The
    exponential is off by at most 2 + 1.173 |a| steps (the bound CUDA states
    for its fast form), a step being 2 U relative; the sum, the quotient (at
    most 2 steps) and the product with b add 1 + 4 + 1 roundings."""
    ref = swiglu(a, b)
    rel = 3 * (1 + a.abs()) + 3 + 2 * (2 + 1.173 * a.abs()) + 6
    # below exp(-80) the fp32 quotient is subnormal or 0
    return ref.abs() * (HALF[dtype] + 1.01 * rel * U) + 1e-30 * (1 + b.abs())


def philox_keep(n, seed, offset, thr):
    """Truth values of n elements (Philox4x32-10, eight 16-bit numbers a block)."""
    m, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    nb = -(-n // 8)
    b = np.arange(nb, dtype=np.uint64)
    x = [b & m, b >> s32, np.full(nb, offset & 0xFFFFFFFF, np.uint64), np.full(nb, (offset >> 32) & 0xFFFFFFFF, np.uint64)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p0, p1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(p1 >> s32) ^ x[1] ^ np.uint64(k[0]), p1 & m, (p0 >> s32) ^ x[3] ^ np.uint64(k[1]), p0 & m]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    halves = np.stack([v for w in x for v in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1).reshape(-1)[:n]
    return torch.from_numpy(halves.astype(np.int64) >= thr)


def mix(o, pos, gate, s=None, residual=None, factor=None):
    """residual + factor * (sum_j gate o[pos] + s), and the sum of magnitudes that bounds its rounding."""
    T, k = pos.shape
    d = o.shape[1]
    y = torch.zeros((T, d), dtype=torch.float64, device=o.device)
    mag = torch.zeros_like(y)
    for j in range(k):
        on = (pos[:, j] >= 0).nonzero()[:, 0]
        v = gate[on, j, None].double() * o[pos[on, j].long()].double()
        y[on] += v
        mag[on] += v.abs()
    if s is not None:
        y += s.double()
        mag += s.double().abs()
    if factor is not None:
        # a dropped element is 0 whatever its value
        y = torch.where(factor > 0, y * factor, torch.zeros_like(y))
        mag = torch.where(factor > 0, mag * factor, torch.zeros_like(mag))
    if residual is not None:
        y += residual.double()
        mag += residual.double().abs()
    return y, mag


def mix_bound(y, mag, k, dtype):
    """k fused multiply-adds, the shared row, the scale (its own rounding and the product's) and the residual."""
    return y.abs() * HALF[dtype] + (k + 5) * 1.01 * U * mag + 1e-37


def factor_of(T, d, prob, seed, offset, device):
    thr = int(math.floor(prob * 65536 + 0.5))
    if thr == 0:
        return None
    keep = philox_keep(T * d, seed, offset, thr).reshape(T, d).to(device)
    return keep.double() * (65536.0 / (65536 - thr))


def routed(T, E, k, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((T, E), generator=g) + skew * torch.randn((1, E), generator=g)
    return z.topk(k, dim=1).indices.to(torch.int32)


def capacity(cf, T, k, E):
    return math.ceil(float(np.float32(cf)) * T * k / E) if cf > 0 else None
