"""Plain binary64 forms of the rows and drafted-tree operators, with the error each kernel may make.

A bound counts roundings: half a step of the storage type (torch.finfo(t).eps / 2, relative) for
each rounding to it, and 2^-24 for each binary32 operation on the way to a value.
"""
import math

import torch

U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def rows(qkv, positions, q_heads, kv_heads, d, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False):
    """(q, k, v, bound_q, bound_k) of rows [n][(Hq + 2 Hkv) d] in binary64.

    The bound before the store: the norm's sum of squares runs 8 products per lane and 5 levels of
    lanes (13 roundings, halved by the root), then the mean, eps, root, quotient and two products
    (6); the angle's rest is rounded to 2^-27 half turns (half a unit) and its sine and cosine to
    two units; a product, a fused product and sum. 20 units of |y_a| + |y_b| covers them."""
    x = qkv.double().unflatten(-1, (q_heads + 2 * kv_heads, d))
    outs = []
    for part, w in ((x[:, :q_heads], q_weight), (x[:, q_heads:q_heads + kv_heads], k_weight)):
        y = part if w is None else part / torch.sqrt(part.square().mean(-1, keepdim=True) + eps) * w.double()
        bound = y.abs() * 20 * U32 if w is not None else torch.zeros_like(y)
        out = y.clone()
        half = 0 if inv_freq is None else inv_freq.numel()
        if half:
            ang = positions.double()[:, None] * inv_freq.double()
            c, s = ang.cos()[:, None], ang.sin()[:, None]
            ia = torch.arange(half, device=x.device)
            ib = ia + half
            if interleaved:
                ia, ib = 2 * ia, 2 * ia + 1
            a, b = y[..., ia], y[..., ib]
            out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
            # the binary64 product rounds the angle itself at far positions
            size = (20 * U32 + ang.abs()[:, None] * 2.0 ** -52) * (a.abs() + b.abs())
            bound[..., ia], bound[..., ib] = size, size
        outs.append((out, bound + half_step(qkv.dtype) * out.abs()))
    return outs[0][0], outs[1][0], x[:, q_heads + kv_heads:], outs[0][1], outs[1][1]


def attend(pool, slot_block, lengths, counts, q, k, v, mask):
    """(out, bound) of the drafted tokens' attention, [R][T][Hq][d] in binary64; rows past a request's
    count are NaN in out. pool [R][Hkv][Kb][2][bs][d].

    Bound of a row: scores are sums of d products, each operation within 2^-24 (2^-23 for the tensor
    cores' accumulation) of the sum of absolute products, so a weight is off by twice that
    (relative, the maximum's part included) and the exponential's 2^-22; the sums of n weights and
    of n products add n roundings each; bf16 weights round to half a step; and the result rounds
    once."""
    R, T, Hq, d = q.shape
    H, kb, bs = pool.shape[1], pool.shape[2], pool.shape[4]
    g = Hq // H
    unit = 2.0 ** -23 if q.dtype == torch.bfloat16 else U32
    weight = half_step(q.dtype) if q.dtype == torch.bfloat16 else 0.0
    out = torch.full((R, T, Hq, d), float("nan"), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    lens = lengths.tolist()
    cnts = [T] * R if counts is None else [min(max(int(c), 0), T) for c in counts.tolist()]
    bits = mask.tolist()
    for r in range(R):
        n = cnts[r]
        if n == 0:
            continue
        sees = torch.tensor([[bits[r][i] >> j & 1 for j in range(n)] for i in range(n)], dtype=torch.bool, device=q.device)
        for h in range(H):
            b = slot_block[r, h].long()[:, None]
            pos = (b * bs + torch.arange(bs, device=q.device))
            ok = ((b >= 0) & (pos < lens[r])).reshape(-1)
            kk = pool[r, h, :, 0].reshape(-1, d)[ok].double()
            vv = pool[r, h, :, 1].reshape(-1, d)[ok].double()
            kd, vd = k[r, :n, h].double(), v[r, :n, h].double()
            for i in range(n):
                ki = torch.cat((kk, kd[sees[i]]))
                vi = torch.cat((vv, vd[sees[i]]))
                heads = slice(h * g, (h + 1) * g)
                if not len(ki):
                    out[r, i, heads] = 0.0
                    continue
                qi = q[r, i, heads].double()
                sc = qi @ ki.T / math.sqrt(d)
                p = torch.softmax(sc, -1)
                o = p @ vi
                err = (d + 8) * unit * ((qi.abs() @ ki.abs().T / math.sqrt(d)).amax(-1, keepdim=True))
                rel = torch.expm1(2 * err) + 2.0 ** -21 + 2 * (len(ki) + 16) * unit + weight
                out[r, i, heads] = o
                bound[r, i, heads] = rel * (p @ vi.abs()) * 1.01 + half_step(q.dtype) * o.abs()
    return out, bound


def random_trees(R, T, gen, device):
    """[R][T] ancestor masks of random trees (every token sees itself)."""
    mask = [[0] * T for _ in range(R)]
    pick = torch.rand(R, T, generator=gen).tolist()
    for r in range(R):
        for t in range(T):
            up = mask[r][int(pick[r][t] * t)] if t else 0
            mask[r][t] = up | 1 << t
    signed = [[m - (1 << 64) if m >> 63 else m for m in row] for row in mask]
    return torch.tensor(signed, dtype=torch.int64, device=device)
