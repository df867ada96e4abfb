"""Plain binary64 forms of the operators of a bounded cache, with the error each kernel may make: half a step of the
storage type for each rounding to it, 2^-24 (2^-23 in the tensor cores' sums) for each binary32 operation."""
import math

import torch

from tree_ref import U32, half_step


def new_tokens(lengths, counts, T):
    """New tokens of each request as the calls take them."""
    lens = lengths.tolist()
    cnts = [T] * len(lens) if counts is None else [min(max(int(c), 0), T) for c in counts.tolist()]
    return lens, [0 if n < 0 or n + T > 2 ** 31 - 1 else c for n, c in zip(lens, cnts)]


def attend(pool, slot_block, lengths, counts, q, window=0, sinks=0, weight=None):
    """((out, lse, weight_out), their bounds): out [R][T][Hq][d] and lse [R][T][Hq] (NaN on rows from a request's count
    on), weight_out [R][Hkv][Kb].

    Bounds. A score: d products and the scale, each within `unit` of the sum of absolute products. A weight: its score's and the
    maximum's error and the exponential's 2^-22, and a rounding to bf16 where the product takes it so. Sums of n
    terms: n + 16 roundings. lse: the score's and the sum's errors, and six roundings of numbers of its own and the largest
    score's size. What a slot draws: each weight by its score, lse and the rounding of both in the exponent; sums of at most
    128 rows, of those, of the slot's tokens; and the last addition."""
    R, T, Hq, d = q.shape
    H, kb, bs = pool.shape[1], pool.shape[2], pool.shape[4]
    g, dev = Hq // H, q.device
    bf16 = q.dtype == torch.bfloat16
    unit, rounded = (2.0 ** -23, half_step(q.dtype)) if bf16 else (U32, 0.0)
    nan = dict(fill_value=float("nan"), dtype=torch.float64, device=dev)
    out, lse = torch.full((R, T, Hq, d), **nan), torch.full((R, T, Hq), **nan)
    out_b, lse_b = torch.zeros_like(out), torch.zeros_like(lse)
    drawn = torch.zeros(R, H, kb, dtype=torch.float64, device=dev) if weight is None else weight.double()
    drawn_b = torch.zeros_like(drawn)
    lens, cnts = new_tokens(lengths, counts, T)
    for r in range(R):
        n = cnts[r]
        p = lens[r] + torch.arange(n, device=dev)[:, None]
        for h in range(H if n else 0):
            b = slot_block[r, h].long()[:, None]
            pos = b * bs + torch.arange(bs, device=dev)
            keep = ((b >= 0) & (pos < lens[r] + n)).reshape(-1).nonzero()[:, 0]
            pos = pos.reshape(-1)[keep]
            sees = pos <= p
            if window:
                sees &= (p - pos < window) | (pos < sinks)
            k, v = (pool[r, h, :, i].reshape(-1, d)[keep].double() for i in (0, 1))
            total = torch.zeros(kb * bs, dtype=torch.float64, device=dev)
            total_b = torch.zeros_like(total)
            for j in range(h * g, h * g + g):
                qi = q[r, :n, j].double()
                z = (qi @ k.T / math.sqrt(d)).masked_fill(~sees, -math.inf)
                top = z.amax(-1, keepdim=True) if len(keep) else torch.full((n, 1), -math.inf, dtype=torch.float64, device=dev)
                e = torch.where(sees, torch.exp(z - torch.where(top == -math.inf, 0.0, top)), 0.0)
                l = e.sum(-1, keepdim=True)
                w = torch.where(sees, e / torch.where(l == 0, 1.0, l), 0.0)
                # a value that a row does not see is no part of it, whatever it is
                odd = ~torch.isfinite(v).all(-1)
                o = w @ torch.where(odd[:, None], 0.0, v)
                oa = w @ torch.where(odd[:, None], 0.0, v).abs()
                for t in odd.nonzero()[:, 0].tolist():
                    o = torch.where((sees[:, t] & (l[:, 0] != 0))[:, None], o + w[:, t:t + 1] * v[t], o)
                size = (qi.abs() @ k.abs().T / math.sqrt(d)).masked_fill(~sees, 0.0).nan_to_num(0.0, 0.0, 0.0)
                size = size.amax(-1, keepdim=True) if len(keep) else torch.zeros(n, 1, dtype=torch.float64, device=dev)
                err = (d + 8) * unit * size
                out[r, :n, j] = o
                out_b[r, :n, j] = (torch.expm1(2 * err) + 2.0 ** -21 + 2 * (len(keep) + 16) * unit + rounded) * oa * 1.01 + half_step(q.dtype) * o.abs()
                s = torch.where(l == 0, -math.inf, torch.where(top == -math.inf, 0.0, top) + l.log())
                lse[r, :n, j] = s[:, 0]
                sb = err + 2.0 ** -21 + (len(keep) + 16) * unit + 6 * U32 * (s.abs() + size)
                lse_b[r, :n, j] = sb[:, 0]
                total.index_add_(0, keep, w.sum(0))
                rel = torch.where(l == 0, 0.0, torch.expm1(err + sb + 2.0 ** -21 + 4 * U32 * (s.abs() + size)))
                total_b.index_add_(0, keep, (w * rel.nan_to_num(0.0)).sum(0))
            drawn[r, h] += total.view(kb, bs).sum(-1)
            drawn_b[r, h] = total_b.view(kb, bs).sum(-1) + (128 + n * g / 32 + bs + 8) * U32 * total.view(kb, bs).sum(-1) + U32 * drawn[r, h].abs()
    return (out, lse, drawn), (out_b, lse_b, drawn_b)


def evict(slot_block, weight, lengths, counts, n_new, block_size, sinks=0, recent=0):
    """(slot_block, weight) after room was made, as lists of lists, slot by slot as the definition says it."""
    bs = block_size
    lens, cnts = new_tokens(lengths, counts, n_new)
    table, drawn = slot_block.tolist(), weight.tolist()
    for r, (n, c) in enumerate(zip(lens, cnts)):
        if c == 0:
            continue
        for sb, w in zip(table[r], drawn[r]):
            held, stop = set(sb), -(-(n + c) // bs)
            begin = -(-n // bs)
            empty, old = [], []
            for i, b in enumerate(sb):
                if b < 0 or (b * bs >= n and b >= stop):
                    empty.append(i)
                elif b * bs < n and b * bs >= sinks and (b + 1) * bs <= n - recent:
                    old.append((math.inf if math.isnan(w[i]) else w[i], math.isnan(w[i]), i))
            order = empty + [i for _, _, i in sorted(old)]
            wanted = []
            b = stop - 1
            while b >= begin and len(wanted) < len(order):
                if b not in held:
                    wanted.append(b)
                b -= 1
            for i, b in zip(sorted(order[:len(wanted)]), sorted(wanted)):
                sb[i], w[i] = b, 0.0
    return table, drawn
