"""Workloads of the operators around a decode step: the rows a projection gives (per-head norms and
the position rotation), appending them to a paged pool, and attention of a tree of drafted tokens
over a request's resident set.

``listed()`` gives the fixed cases, ``draw()`` more of the same ranges; ``prepare()`` makes a
case's inputs on the GPU, ``run()`` makes one pass: through the library's entry points where
``own`` is set, in elementary torch operations where it is not. ``exact()`` computes the same
outputs in binary64 from the definitions.

Shapes (R requests, T new tokens each, Hq / Hkv heads, d head_dim, Kb slots of bs tokens):
  rows    qkv [n][(Hq + 2 Hkv) d] -> q [n][Hq][d], k [n][Hkv][d], v [n][Hkv][d]
  append  qkv [R][T][...] -> q [R][T][Hq][d], and the pool [R][Hkv][Kb][2][bs][d]
  tree    q [R][T][Hq][d], k, v [R][T][Hkv][d], mask [R][T] over the pool -> out [R][T][Hq][d]
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    qwen = dict(q_heads=32, kv_heads=8, head_dim=128, dtype="bf16")     # Qwen3-8B attention
    gqa32 = dict(q_heads=64, kv_heads=8, head_dim=128, dtype="bf16")    # the 32B-class GQA shapes
    tiny = dict(q_heads=8, kv_heads=2, head_dim=64, dtype="f32")        # the tiny single-layer step
    full = dict(rotary_dim=128, interleaved=False, norm=True)
    pool = dict(block_size=16, slots=128)                               # budget 2048
    return [
        # one request's next token: latency
        dict(name="rows_b1", op="rows", n=1, start=16384, stride_pad=0, skip=0, **qwen, **full),
        # 128 requests' trees of 16 drafted tokens
        dict(name="rows_b128x16", op="rows", n=2048, start=16384, stride_pad=0, skip=0, **qwen, **full),
        # a prefill chunk of 16K tokens
        dict(name="rows_prefill16k", op="rows", n=16384, start=0, stride_pad=0, skip=0, **gqa32, **full),
        # binary32, a rotation of half the head in adjacent pairs, no norms, a row stride past the
        # row and some padded rows
        dict(name="rows_f32_partial", op="rows", n=1003, start=100000, stride_pad=20, skip=9, **tiny,
             rotary_dim=32, interleaved=True, norm=False),
        # a decode step's token of 128 requests at 16K
        dict(name="append_b128", op="append", R=128, T=1, context=16384, ragged=False, **qwen, **pool, **full),
        # ragged chunks of up to 1024 tokens of 16 requests
        dict(name="append_chunk_ragged", op="append", R=16, T=1024, context=4099, ragged=True, **gqa32, **pool, **full),
        # binary32, a few tokens of two requests
        dict(name="append_f32", op="append", R=2, T=5, context=4093, ragged=True, **tiny, block_size=16, slots=32,
             rotary_dim=64, interleaved=False, norm=True),
        # one request, a small tree: latency
        dict(name="tree_b1x8", op="tree", R=1, T=8, context=16384, ragged=False, **qwen, **pool),
        # the decode batch at 16K, 16 drafted tokens each
        dict(name="tree_b128x16", op="tree", R=128, T=16, context=16384, ragged=False, **qwen, **pool),
        # wide trees on the widest group: 512 query rows for every key head
        dict(name="tree_b32x64_gqa8", op="tree", R=32, T=64, context=32768, ragged=False, **gqa32, **pool),
        # binary32
        dict(name="tree_f32", op="tree", R=16, T=12, context=4096, ragged=False, **tiny, block_size=16, slots=32),
        # ragged trees, contexts from nothing to past the budget, a group of three, other sizes
        dict(name="tree_odd_ragged", op="tree", R=37, T=13, context=1500, ragged=True, q_heads=24, kv_heads=8,
             head_dim=64, dtype="bf16", block_size=32, slots=33),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "append", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([64, 128, 128, 32, 96, 256] if op != "tree" else [64, 128, 128, 128, 96])
    hkv = rng.choice([1, 2, 4, 8, 8])
    g = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    c = dict(op=op, q_heads=hkv * g, kv_heads=hkv, head_dim=d, dtype=dtype)
    if op != "tree":
        c.update(rotary_dim=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.8)
    elem = 4 if dtype == "f32" else 2
    if op == "rows":
        row = (c["q_heads"] + 2 * hkv) * d * elem
        c.update(n=_log(rng, 1, min(16384, 335_000_000 // row)), start=_log(rng, 1, 1_000_000),
                 stride_pad=rng.choice([0, 0, 24]), skip=rng.choice([0, 0, 5]))
        return c
    bs = rng.choice([8, 16, 16, 32, 64])
    c.update(block_size=bs, slots=max(1, _log(rng, 64, 4096) // bs), context=_log(rng, 1, 60000),
             ragged=rng.random() < 0.5)
    unit = hkv * c["slots"] * 2 * bs * d * elem
    c["R"] = _log(rng, 1, max(1, min(128, 1_000_000_000 // unit)))
    if op == "append":
        row = (c["q_heads"] + 2 * hkv) * d * elem
        c["T"] = _log(rng, 1, max(1, min(1024, 300_000_000 // (row * c["R"]))))
    else:
        rows = (6 if dtype == "f32" else 100) * 1_000_000 // (c["R"] * c["q_heads"] * c["slots"] * bs)
        c["T"] = _log(rng, 1, max(1, min(64, rows)))
    return c


def _lengths(case):
    """Tokens of each request before the new ones, and its new tokens: of the case alone."""
    R, T, n = case["R"], case["T"], case["context"]
    if not case["ragged"]:
        return [n] * R, [T] * R
    lengths = [(n * (r * 37 % 101)) // 100 for r in range(R)]  # 0 .. n, request 0 has nothing
    counts = [T - (r * 5 % (T + 1)) for r in range(R)]         # T .. 0
    return lengths, counts


def _resident(case, length):
    """(occupied slots, valid tokens in them) of a unit of a tree case: the last block is among them."""
    bs = case["block_size"]
    blocks = -(-length // bs)
    n = min(case["slots"], blocks)
    return n, (n - 1) * bs + (length - (blocks - 1) * bs) if n else 0


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    d, hq, hkv = case["head_dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "rows":
        n = case["n"] - (case["n"] // case["skip"] if case["skip"] else 0)
        return {"bytes": n * (2 * (hq + 2 * hkv) * d * e + 4), "flops": n * (hq + hkv) * d * 7}
    lengths, counts = _lengths(case)
    new = sum(counts)
    if case["op"] == "append":
        return {"bytes": new * 2 * (hq + 2 * hkv) * d * e + case["R"] * (hkv * case["slots"] * 4 + 8),
                "flops": new * (hq + hkv) * d * 7}
    kept = [_resident(case, n)[1] if t else 0 for n, t in zip(lengths, counts)]
    moved = 2 * hkv * d * e * (sum(kept) + new) + 2 * new * hq * d * e + new * 8 + case["R"] * (hkv * case["slots"] * 4 + 8)
    return {"bytes": moved, "flops": sum(4 * d * hq * t * (n + 1) for n, t in zip(kept, counts))}


# ---- inputs --------------------------------------------------------------------------------------

def _rope(case, gen, dev, dtype):
    rot, d = case["rotary_dim"], case["head_dim"]
    inv = 1e6 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    w = (1 + 0.2 * torch.randn(2, d, generator=gen, device=dev)).to(dtype)
    return {"inv_freq": inv.float(), "q_weight": w[0].contiguous() if case["norm"] else None,
            "k_weight": w[1].contiguous() if case["norm"] else None, "eps": 1e-6, "interleaved": case["interleaved"]}


def _slots(case, gen, dev):
    """Slot tables: [R][Hkv][Kb] block ids or -1. In a tree case a random set of a request's blocks
    with the last one among them, in any order; in an append case the latest blocks, of which one
    in eight is not resident."""
    R, H, kb, bs = case["R"], case["kv_heads"], case["slots"], case["block_size"]
    lengths, counts = _lengths(case)
    end = torch.tensor([n + (t if case["op"] == "append" else 0) for n, t in zip(lengths, counts)], device=dev)
    nb = (end + bs - 1) // bs
    place = torch.rand(R, H, kb, generator=gen, device=dev).argsort(-1)
    if case["op"] == "append":
        ids = (nb - 1)[:, None, None] - torch.arange(kb, device=dev)
        ids = torch.where((ids >= 0) & (ids % 8 != 5), ids, -1).expand(R, H, kb)
    else:
        most = int(nb.max()) if R else 0
        key = torch.rand(R, H, max(most, kb), generator=gen, device=dev)
        b = torch.arange(key.shape[-1], device=dev)
        key = torch.where(b == (nb - 1)[:, None, None], 2.0, key)
        key = torch.where(b < nb[:, None, None], key, -1.0)
        top = key.topk(kb, dim=-1)
        ids = torch.where(top.values >= 0, top.indices, -1)
        # a short context fills the first slots, as the staging does
        return ids.to(torch.int32).contiguous() if int(nb.min()) < kb else ids.gather(-1, place).to(torch.int32).contiguous()
    return ids.gather(-1, place).to(torch.int32).contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dtype = _DTYPES[case["dtype"]]
    d, hq, hkv = case["head_dim"], case["q_heads"], case["kv_heads"]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    s = {"case": dict(case), "dtype": dtype}
    if case["op"] == "rows":
        n, width = case["n"], (hq + 2 * hkv) * d
        s["qkv"] = rand(n, width + case["stride_pad"])[:, :width]
        pos = case["start"] + torch.randint(0, 1 + case["n"], (n,), generator=gen, device=dev)
        if case["skip"]:  # padded rows: a negative position
            pos[case["skip"] - 1::case["skip"]] = -1
        s["positions"] = pos.to(torch.int32)
        s["rope"] = _rope(case, gen, dev, dtype)
        s["q"] = torch.zeros(n, hq, d, device=dev, dtype=dtype)
        s["k"] = torch.zeros(n, hkv, d, device=dev, dtype=dtype)
        s["v"] = torch.zeros(n, hkv, d, device=dev, dtype=dtype)
        return s
    R, T, kb, bs = case["R"], case["T"], case["slots"], case["block_size"]
    lengths, counts = _lengths(case)
    s["lengths"] = torch.tensor(lengths, device=dev, dtype=torch.int32)
    s["counts"] = torch.tensor(counts, device=dev, dtype=torch.int32)
    s["slot_block"] = _slots(case, gen, dev)
    s["pool"] = torch.empty(R, hkv, kb, 2, bs, d, device=dev, dtype=dtype).normal_(generator=gen)
    if case["op"] == "append":
        s["qkv"] = rand(R, T, (hq + 2 * hkv) * d)
        s["rope"] = _rope(case, gen, dev, dtype)
        s["q"] = torch.zeros(R, T, hq, d, device=dev, dtype=dtype)
        return s
    s["q"] = (2 * torch.randn(R, T, hq, d, generator=gen, device=dev)).to(dtype)  # scores of spread 2
    s["k"], s["v"] = rand(R, T, hkv, d), rand(R, T, hkv, d)
    # a random tree: every token sees itself and what its parent sees; in a ragged case some rows
    # see no drafted token at all
    parent = (torch.rand(R, T, generator=gen, device=dev) * torch.arange(T, device=dev)).long()
    mask = torch.zeros(R, T, device=dev, dtype=torch.int64)
    for t in range(T):
        up = mask.gather(1, parent[:, t:t + 1])[:, 0] if t else 0
        mask[:, t] = up | (-(1 << 63) if t == 63 else 1 << t)
    if case["ragged"]:
        mask[:, T // 2::5] = 0
    s["mask"] = mask
    s["out"] = torch.zeros(R, T, hq, d, device=dev, dtype=dtype)
    return s


# ---- one pass ------------------------------------------------------------------------------------

def _rotary(rope):
    from sparse_kv_cache_draft_gb300 import Rotary
    return Rotary(rope["inv_freq"], q_weight=rope["q_weight"], k_weight=rope["k_weight"], eps=rope["eps"],
                  interleaved=rope["interleaved"])


def _norm(x, weight, eps):
    return x if weight is None else x * (x.square().mean(-1, keepdim=True) + eps).rsqrt() * weight.float()


def _turn(x, positions, rope):
    """Rotates the first 2 len(inv_freq) dims of x [..., heads, d] by positions [...] * inv_freq."""
    half = rope["inv_freq"].numel()
    angle = positions.double()[..., None] * rope["inv_freq"].double()
    cos, sin = angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]
    y, rest = x[..., :2 * half], x[..., 2 * half:]
    if rope["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _plain_rows(qkv, positions, case, rope):
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    x = qkv.unflatten(-1, (hq + 2 * hkv, d))
    q = _turn(_norm(x[..., :hq, :].float(), rope["q_weight"], rope["eps"]), positions, rope)
    k = _turn(_norm(x[..., hq:hq + hkv, :].float(), rope["k_weight"], rope["eps"]), positions, rope)
    return q.to(qkv.dtype), k.to(qkv.dtype), x[..., hq + hkv:, :]


def _run_rows(s):
    c = s["case"]
    if own:
        from sparse_kv_cache_draft_gb300 import norm_rope
        norm_rope(s["qkv"], s["positions"], s["q"], s["k"], s["v"], q_heads=c["q_heads"], kv_heads=c["kv_heads"],
                  head_dim=c["head_dim"], rotary=_rotary(s["rope"]))
        return s["q"], s["k"], s["v"]
    rows = _plain_rows(s["qkv"], s["positions"], c, s["rope"])
    keep = (s["positions"] >= 0)[:, None, None]
    return tuple(torch.where(keep, x, s[name]) for x, name in zip(rows, "qkv"))


def _run_append(s):
    c = s["case"]
    if own:
        from sparse_kv_cache_draft_gb300 import append_qkv_static
        append_qkv_static(s["qkv"], s["lengths"], s["counts"], s["pool"], s["slot_block"], s["q"],
                          q_heads=c["q_heads"], kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                          block_size=c["block_size"], slots=c["slots"], rotary=_rotary(s["rope"]))
        return s["q"], s["pool"]
    bs = c["block_size"]
    t = torch.arange(c["T"], device=s["qkv"].device)
    positions = s["lengths"][:, None] + t
    fresh = t < s["counts"][:, None]
    q, k, v = _plain_rows(s["qkv"], positions, c, s["rope"])
    q = torch.where(fresh[..., None, None], q, s["q"])
    # [R][T][Hkv][Kb]: the slot that holds the token's block, if any
    hit = s["slot_block"][:, None] == (positions // bs)[:, :, None, None]
    r, t, h = (hit.any(-1) & fresh[..., None]).nonzero(as_tuple=True)
    slot, at = hit.int().argmax(-1)[r, t, h], (positions % bs)[r, t]
    s["pool"][r, h, slot, 0, at] = k[r, t, h]
    s["pool"][r, h, slot, 1, at] = v[r, t, h]
    return q, s["pool"]


def _run_tree(s):
    c = s["case"]
    if own:
        from sparse_kv_cache_draft_gb300 import attend_tree_static
        attend_tree_static(s["pool"], s["slot_block"], s["lengths"], s["counts"], s["q"], s["k"], s["v"], s["mask"],
                           s["out"], q_heads=c["q_heads"], kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                           block_size=c["block_size"], slots=c["slots"])
        return s["out"]
    R, T, H, kb, bs, d = c["R"], c["T"], c["kv_heads"], c["slots"], c["block_size"], c["head_dim"]
    g = c["q_heads"] // H
    dev = s["q"].device
    t = torch.arange(T, device=dev)
    fresh = t < s["counts"][:, None]
    # keys and values of the resident set and of the drafted tokens, and who sees them
    block = s["slot_block"].long()[..., None]
    token = block * bs + torch.arange(bs, device=dev)
    valid = ((block >= 0) & (token < s["lengths"][:, None, None, None])).flatten(2)      # [R][H][Kb bs]
    k = torch.cat((s["pool"][:, :, :, 0].flatten(2, 3), s["k"].transpose(1, 2)), 2).float()
    v = torch.cat((s["pool"][:, :, :, 1].flatten(2, 3), s["v"].transpose(1, 2)), 2).float()
    held = torch.cat((valid, fresh[:, None].expand(R, H, T)), 2)[..., None]
    k, v = torch.where(held, k, 0.0), torch.where(held, v, 0.0)
    drafted = ((s["mask"][..., None] >> t) & 1).bool() & fresh[:, None]                  # [R][T][T]
    sees = torch.cat((valid[:, :, None].expand(R, H, T, kb * bs), drafted[:, None].expand(R, H, T, T)), 3)
    q = s["q"].float().unflatten(2, (H, g)).permute(0, 2, 1, 3, 4)                       # [R][H][T][g][d]
    score = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (T, g)) / math.sqrt(d)
    score = score.masked_fill_(~sees[:, :, :, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = (score - torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (T, g)) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3).to(s["q"].dtype)
    return torch.where(fresh[..., None, None], o, s["out"])


def run(state):
    return {"rows": _run_rows, "append": _run_append, "tree": _run_tree}[state["case"]["op"]](state)


# ---- the definitions in binary64 -----------------------------------------------------------------

def _exact_head(x, weight, eps, positions, inv_freq, interleaved):
    """x [n][heads][d] -> normed and turned, pair by pair as complex numbers."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + eps) * weight.double()
    half = inv_freq.numel()
    unit = torch.polar(torch.ones((), device=x.device, dtype=torch.float64),
                       torch.outer(positions.double(), inv_freq.double()))[:, None, :]
    out = x.clone()
    if interleaved:
        z = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2]) * unit
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :half], x[..., half:2 * half]) * unit
        out[..., :half], out[..., half:2 * half] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "rows":
        rope, keep = s["rope"], s["positions"] >= 0
        x, pos = s["qkv"][keep].unflatten(-1, (hq + 2 * hkv, d)), s["positions"][keep]
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        q[keep] = _exact_head(x[:, :hq], rope["q_weight"], rope["eps"], pos, rope["inv_freq"], rope["interleaved"])
        k[keep] = _exact_head(x[:, hq:hq + hkv], rope["k_weight"], rope["eps"], pos, rope["inv_freq"], rope["interleaved"])
        v[keep] = x[:, hq + hkv:].double()
        return q, k, v
    bs, kb = case["block_size"], case["slots"]
    lengths, counts = _lengths(case)
    if case["op"] == "append":
        rope, q, pool = s["rope"], s["q"].double(), s["pool"].double()
        for r in range(case["R"]):
            n = counts[r]
            if not n:
                continue
            pos = lengths[r] + torch.arange(n, device=q.device)
            x = s["qkv"][r, :n].unflatten(-1, (hq + 2 * hkv, d))
            q[r, :n] = _exact_head(x[:, :hq], rope["q_weight"], rope["eps"], pos, rope["inv_freq"], rope["interleaved"])
            k = _exact_head(x[:, hq:hq + hkv], rope["k_weight"], rope["eps"], pos, rope["inv_freq"], rope["interleaved"])
            # from the slots' side: the new token each place of the pool holds, if any
            first = s["slot_block"][r].long()[..., None] * bs
            idx = first + torch.arange(bs, device=q.device) - lengths[r]
            new = (first >= 0) & (idx >= 0) & (idx < n)
            h, slot, at = torch.nonzero(new, as_tuple=True)
            pool[r, h, slot, 0, at] = k[idx[new], h]
            pool[r, h, slot, 1, at] = x[idx[new], hq + hkv + h].double()
        return q, pool
    out = s["out"].double()
    g = hq // hkv
    for r in range(case["R"]):
        n = counts[r]
        if not n:
            continue
        bits = s["mask"][r, :n].tolist()
        sees = torch.tensor([[m >> j & 1 for j in range(n)] for m in bits], device=out.device, dtype=torch.bool)
        blocks = s["slot_block"][r].long()
        for h in range(hkv):
            pos = (blocks[h][:, None] * bs + torch.arange(bs, device=out.device)).reshape(-1)
            ok = (pos >= 0) & (pos < lengths[r])
            k = torch.cat((s["pool"][r, h, :, 0].reshape(-1, d)[ok], s["k"][r, :n, h])).double()
            v = torch.cat((s["pool"][r, h, :, 1].reshape(-1, d)[ok], s["v"][r, :n, h])).double()
            who = torch.cat((torch.ones(n, int(ok.sum()), device=out.device, dtype=torch.bool), sees), 1)
            q = s["q"][r, :n, h * g:(h + 1) * g].double()
            z = torch.einsum("tgd,jd->tgj", q, k) * d ** -0.5
            z = torch.where(who[:, None], z, -math.inf)
            p = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)  # a row that sees nothing is zero
            out[r, :n, h * g:(h + 1) * g] = torch.einsum("tgj,jd->tgd", p, v)
    return out
