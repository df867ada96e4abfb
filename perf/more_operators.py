"""Workloads of the operators that keep a bounded cache without a context: attention of a chunk of new
tokens over a paged pool (causal, with a sliding window and first tokens that stay visible), the
attention weight that each slot of the pool has drawn, and eviction by that weight.

``listed()`` gives the fixed cases, ``draw()`` more of the same ranges; ``prepare()`` makes a
case's inputs on the GPU, ``run()`` makes one pass: through the library's entry points where
``own`` is set, in elementary torch operations where it is not. ``exact()`` computes the same
outputs in binary64 from the definitions.

Shapes (R requests, T new tokens each, Hq / Hkv heads, d head_dim, Kb slots of bs tokens):
  chunk   q [R][T][Hq][d] over the pool [R][Hkv][Kb][2][bs][d], whose slots hold the new tokens' keys and
          values already -> out [R][T][Hq][d], lse [R][T][Hq] and, where weigh is set, weight [R][Hkv][Kb]
  evict   slot_block, weight [R][Hkv][Kb] -> the same with slots for the blocks of T new tokens
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
    pool = dict(block_size=16, slots=128)                               # budget 2048
    plain = dict(window=0, sinks=0, weigh=False, ragged=False)
    return [
        # one chunk of a prompt, everything before it in the pool: 16K tokens
        dict(name="chunk_16k", op="chunk", R=1, T=2048, context=14336, **qwen, block_size=16, slots=1024, **plain),
        # chunks of four prompts of 32K on the widest group: the largest
        dict(name="chunk_gqa8_32k", op="chunk", R=4, T=1024, context=31744, **gqa32, block_size=64, slots=512, **plain),
        # short chunks of 16 requests over a budget of 2048 tokens each
        dict(name="chunk_budget_b16", op="chunk", R=16, T=256, context=16384, **qwen, **pool, **plain),
        # prompts in chunks under a window, with first tokens that stay visible
        dict(name="window_chunk_b8", op="chunk", R=8, T=1024, context=8192, **qwen, block_size=16, slots=256,
             window=1024, sinks=64, weigh=False, ragged=False),
        # a decode step of 128 requests under the same window
        dict(name="window_decode_b128", op="chunk", R=128, T=1, context=16384, **qwen, **pool, window=1024, sinks=64,
             weigh=False, ragged=False),
        # one request's next token: latency
        dict(name="decode_b1", op="chunk", R=1, T=1, context=16384, **qwen, **pool, **plain),
        # binary32
        dict(name="chunk_f32", op="chunk", R=4, T=100, context=700, **tiny, block_size=16, slots=64, **plain),
        # ragged chunks and contexts, a group of three, other sizes, a window that cuts blocks
        dict(name="chunk_odd_ragged", op="chunk", R=37, T=61, context=1500, q_heads=24, kv_heads=8, head_dim=64,
             dtype="bf16", block_size=32, slots=33, window=300, sinks=5, weigh=False, ragged=True),
        # a decode step of 128 requests that counts what each block draws
        dict(name="weigh_decode_b128", op="chunk", R=128, T=1, context=16384, **qwen, **pool, window=0, sinks=0,
             weigh=True, ragged=False),
        # chunks of eight prompts, counted
        dict(name="weigh_chunk_b8", op="chunk", R=8, T=512, context=6000, **qwen, block_size=16, slots=256, window=0,
             sinks=0, weigh=True, ragged=True),
        # room for the next token of 128 requests: a sixteenth of them begins a block
        dict(name="evict_b128", op="evict", R=128, T=1, context=16384, kv_heads=8, **pool, sinks=64, recent=256,
             ragged=True),
        # room for chunks of 16 requests in large tables
        dict(name="evict_chunk_b16", op="evict", R=16, T=1000, context=40000, kv_heads=8, block_size=16, slots=1024,
             sinks=64, recent=1024, ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "evict"])
    bs = rng.choice([8, 16, 16, 32, 64, 24])
    hkv = rng.choice([1, 2, 4, 8, 8])
    if op == "evict":
        return dict(op=op, R=_log(rng, 1, 128), T=_log(rng, 1, 1024), context=_log(rng, 1, 60000), kv_heads=hkv,
                    block_size=bs, slots=_log(rng, 1, 1024), sinks=rng.choice([0, 4, 64]), recent=_log(rng, 1, 2048),
                    ragged=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    d = rng.choice([128, 128, 128, 64, 64, 96, 32, 256])
    g = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    elem = 4 if dtype == "f32" else 2
    c = dict(op=op, q_heads=hkv * g, kv_heads=hkv, head_dim=d, dtype=dtype, block_size=bs,
             slots=min(1024, max(1, _log(rng, 64, 32768) // bs)), context=_log(rng, 1, 60000),
             ragged=rng.random() < 0.5, weigh=rng.random() < 0.3)
    windowed = rng.random() < 0.4
    c.update(window=_log(rng, 16, 4096) if windowed else 0, sinks=rng.choice([0, 4, 64]) if windowed else 0)
    unit = hkv * c["slots"] * 2 * bs * d * elem
    c["R"] = _log(rng, 1, max(1, min(128, 1_000_000_000 // unit)))
    rows = (2 if dtype == "f32" else 100) * 10_000_000_000 // (c["R"] * c["q_heads"] * c["slots"] * bs * d)
    c["T"] = _log(rng, 1, max(1, min(2048, rows)))
    return c


def _lengths(case):
    """Tokens of each request before the new ones, and its new tokens: of the case alone."""
    R, T, n = case["R"], case["T"], case["context"]
    if not case["ragged"]:
        return [n] * R, [T] * R
    lengths = [(n * (r * 37 % 101)) // 100 for r in range(R)]  # 0 .. n, request 0 has nothing
    if case["op"] == "evict":
        return lengths, [T] * R
    return lengths, [T - (r * 5 % (T + 1)) for r in range(R)]  # T .. 0


def _held(case, length, new):
    """What the pool holds of a request: tokens [0, a) and [b, end), and full blocks anywhere between
    them, at random. Under a window the newest blocks and the first ones, else the new tokens'."""
    bs, kb, end = case["block_size"], case["slots"], length + new
    nb = -(-end // bs)
    if nb <= kb:
        return 0, 0, 0, end
    first = min(kb - 1, -(-case["sinks"] // bs))
    own_blocks = nb - length // bs if new else 1
    newest = kb - first if case["window"] else min(kb - first, own_blocks)
    newest = min(newest, nb - first)
    return first * bs, (nb - newest) * bs, kb - first - newest, end


def _overlap(a, b, c, d):
    return max(0, min(b, d) - max(a, c))


def _visible(case, held, lo, hi):
    """Tokens of `held` that positions lo .. hi see, of any of them."""
    a, b, blocks, end = held
    w, k = case["window"] or end + 1, case["sinks"]
    start, stop = max(0, lo - w + 1), hi + 1
    sink = min(k, stop, start)  # first tokens before the window
    n = sum(_overlap(x, y, start, stop) + _overlap(x, y, 0, sink) for x, y in ((0, a), (b, end)))
    return n + (blocks * case["block_size"] if not case["window"] else 0)


def work(case):
    lengths, counts = _lengths(case)
    hkv, kb = case["kv_heads"], case["slots"]
    table = case["R"] * hkv * kb * 4
    if case["op"] == "evict":
        return {"bytes": 4 * table, "flops": case["R"] * hkv * kb}
    e = 4 if case["dtype"] == "f32" else 2
    d, hq = case["head_dim"], case["q_heads"]
    moved, pairs = table + case["R"] * 8 + (2 * table if case["weigh"] else 0), 0
    for n, t in zip(lengths, counts):
        if t:
            held = _held(case, n, t)
            moved += 2 * hkv * d * e * _visible(case, held, n, n + t - 1) + t * hq * (2 * d * e + 4)
            pairs += sum(_visible(case, held, n + i, n + i) for i in range(t))
    return {"bytes": moved, "flops": 4 * d * hq * pairs}


# ---- inputs --------------------------------------------------------------------------------------

def _slots(case, gen, dev):
    """Slot tables [R][Hkv][Kb]: the blocks of _held in any order; a request that fits lies in order. Of an
    evict case: before the new tokens, with one slot in 32 empty."""
    R, H, kb, bs = case["R"], case["kv_heads"], case["slots"], case["block_size"]
    evict = case["op"] == "evict"
    sb = torch.full((R, H, kb), -1, dtype=torch.int32, device=dev)
    for r, (n, t) in enumerate(zip(*_lengths(case))):
        t = 0 if evict else t
        nb = -(-(n + t) // bs)
        if nb <= kb:
            sb[r, :, :nb] = torch.arange(nb, dtype=torch.int32, device=dev)
            continue
        if evict:
            a, b, rest = 0, (nb - 1) * bs, kb - 1
        else:
            a, b, rest, _ = _held(case, n, t)
        first, last = a // bs, b // bs
        ids = torch.empty(H, kb, dtype=torch.int32, device=dev)
        ids[:, :first] = torch.arange(first, dtype=torch.int32, device=dev)
        ids[:, first:kb - rest] = torch.arange(last, nb, dtype=torch.int32, device=dev)
        between = torch.rand(H, last - first, generator=gen, device=dev).argsort(-1)[:, :rest]
        ids[:, kb - rest:] = (first + between).to(torch.int32)
        sb[r] = ids.gather(-1, torch.rand(H, kb, generator=gen, device=dev).argsort(-1))
    if evict:
        gone = torch.rand(R, H, kb, generator=gen, device=dev) < 1 / 32
        tail = sb == (torch.tensor(_lengths(case)[0], device=dev, dtype=torch.int32) // bs)[:, None, None]
        sb = torch.where(gone & ~tail, -1, sb)
    return sb


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    R, T, H, kb, bs = case["R"], case["T"], case["kv_heads"], case["slots"], case["block_size"]
    lengths, counts = _lengths(case)
    s = {"case": dict(case), "lengths": torch.tensor(lengths, device=dev, dtype=torch.int32),
         "counts": torch.tensor(counts, device=dev, dtype=torch.int32), "slot_block": _slots(case, gen, dev)}
    # what the slots have drawn so far: a few a lot, most little, many alike
    drawn = torch.rand(R, H, kb, generator=gen, device=dev).pow_(-0.7).sub_(1)
    s["weight"] = torch.where(s["slot_block"] < 0, 0.0, (drawn * 64).round_() / 64)
    s["weight_out"] = torch.zeros_like(s["weight"])
    if case["op"] == "evict":
        s["slot_block_out"] = torch.zeros_like(s["slot_block"])
        return s
    dtype, d, hq = _DTYPES[case["dtype"]], case["head_dim"], case["q_heads"]
    s["pool"] = torch.empty(R, H, kb, 2, bs, d, device=dev, dtype=dtype).normal_(generator=gen)
    s["q"] = (2 * torch.randn(R, T, hq, d, generator=gen, device=dev)).to(dtype)  # scores of spread 2
    s["out"] = torch.zeros(R, T, hq, d, device=dev, dtype=dtype)
    s["lse"] = torch.zeros(R, T, hq, device=dev)
    return s


# ---- one pass ------------------------------------------------------------------------------------

def _plain_chunk(s, r0, r1):
    """out, lse and slot weights of requests r0 .. r1 - 1."""
    c = s["case"]
    T, H, kb, bs, d = c["T"], c["kv_heads"], c["slots"], c["block_size"], c["head_dim"]
    g, dev = c["q_heads"] // H, s["q"].device
    length, count = s["lengths"][r0:r1].long(), s["counts"][r0:r1].long()
    t = torch.arange(T, device=dev)
    at = (length[:, None] + t)[:, None, :, None]                                        # [r][1][T][1]
    block = s["slot_block"][r0:r1].long()[..., None]
    pos = (block * bs + torch.arange(bs, device=dev)).flatten(2)                        # [r][H][Kb bs]
    held = (block >= 0).expand(-1, -1, -1, bs).flatten(2) & (pos < (length + count)[:, None, None])
    pos = pos[:, :, None]
    sees = held[:, :, None] & (pos <= at)                                               # [r][H][T][Kb bs]
    if c["window"]:
        sees &= (at - pos < c["window"]) | (pos < c["sinks"])
    q = s["q"][r0:r1].float().unflatten(2, (H, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [r][H][T g][d]
    k = s["pool"][r0:r1, :, :, 0].flatten(2, 3).float()
    score = (q @ torch.where(held[..., None], k, 0.0).transpose(2, 3)).unflatten(2, (T, g))
    score = (score * (1 / math.sqrt(d))).masked_fill_(~sees[:, :, :, None], float("-inf"))
    del k, sees
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(total == 0, 1.0, total))
    v = torch.where(held[..., None], s["pool"][r0:r1, :, :, 1].flatten(2, 3).float(), 0.0)
    o = (p.flatten(2, 3) @ v).unflatten(2, (T, g)).permute(0, 2, 1, 3, 4).flatten(2, 3).to(s["q"].dtype)
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).flatten(2, 3)
    fresh = (t < count[:, None])[..., None]
    drawn = None
    if c["weigh"]:
        p.mul_((t < count[:, None])[:, None, :, None, None])
        drawn = s["weight"][r0:r1] + p.sum((2, 3)).unflatten(-1, (kb, bs)).sum(-1)
    return torch.where(fresh[..., None], o, s["out"][r0:r1]), torch.where(fresh, lse, s["lse"][r0:r1]), drawn


def _run_chunk(s):
    c = s["case"]
    if own:
        from sparse_kv_cache_draft_gb300 import attend_chunk_static
        weigh = dict(weight=s["weight"], weight_out=s["weight_out"]) if c["weigh"] else {}
        attend_chunk_static(s["pool"], s["slot_block"], s["lengths"], s["counts"], s["q"], s["out"], s["lse"],
                            q_heads=c["q_heads"], kv_heads=c["kv_heads"], head_dim=c["head_dim"],
                            block_size=c["block_size"], slots=c["slots"], window=c["window"], sinks=c["sinks"], **weigh)
        return (s["out"], s["lse"], s["weight_out"]) if c["weigh"] else (s["out"], s["lse"])
    each = c["q_heads"] * c["T"] * c["slots"] * c["block_size"]
    step = max(1, 2_000_000_000 // each)  # requests at a time, by the room that their scores take
    parts = [_plain_chunk(s, r, min(r + step, c["R"])) for r in range(0, c["R"], step)]
    outs = [torch.cat(x) if len(x) > 1 else x[0] for x in zip(*parts) if x[0] is not None]
    return tuple(outs)


def _run_evict(s):
    c = s["case"]
    if own:
        from sparse_kv_cache_draft_gb300 import evict_static
        evict_static(s["slot_block"], s["weight"], s["lengths"], s["counts"], s["slot_block_out"], s["weight_out"],
                     n_new=c["T"], kv_heads=c["kv_heads"], block_size=c["block_size"], slots=c["slots"],
                     sinks=c["sinks"], recent=c["recent"])
        return s["slot_block_out"], s["weight_out"]
    bs, kb, sb, dev = c["block_size"], c["slots"], s["slot_block"].long(), s["weight"].device
    length, end = s["lengths"].long()[:, None, None], (s["lengths"] + s["counts"]).long()[:, None, None]
    begin, stop = (length + bs - 1) // bs, (end + bs - 1) // bs            # the blocks that the new tokens begin
    # which of them no slot holds, the last Kb of them
    room = c["T"] // bs + 2
    new = begin + torch.arange(room, device=dev)                           # [R][1][room]
    at = sb - begin
    there = torch.zeros(c["R"], c["kv_heads"], room + 1, device=dev, dtype=torch.bool)
    there.scatter_(2, torch.where((sb >= 0) & (at >= 0) & (at < room), at, room), True)
    wanted = (new < stop) & ~there[..., :room]
    # the order in which slots are taken: empty ones, then by weight, ties by slot
    empty = (sb < 0) | ((sb * bs >= length) & ((sb < begin) | (sb >= stop)))
    kept = ~empty & ((sb * bs < c["sinks"]) | ((sb + 1) * bs > length - c["recent"]))
    weight = torch.where(empty, float("-inf"), torch.where(kept, float("inf"), s["weight"]))
    order = torch.sort(weight, dim=-1, stable=True).indices
    n = torch.minimum(wanted.sum(-1), (~kept).sum(-1))[..., None]          # [R][Hkv][1]
    rank = torch.empty_like(order).scatter_(2, order, torch.arange(kb, device=dev).expand_as(order).contiguous())
    taken = rank < n
    # the n newest wanted blocks, in order, into the taken slots, in order
    behind = wanted.flip(-1).cumsum(-1).flip(-1)
    placed = wanted & (behind <= n)
    nth = placed.cumsum(-1)
    by_order = torch.zeros(*sb.shape[:2], kb + 1, device=dev, dtype=torch.long)
    by_order.scatter_(2, torch.where(placed, nth - 1, kb), new.expand_as(wanted).contiguous())
    got = by_order.gather(2, (taken.cumsum(-1) - 1).clamp_(min=0))
    return torch.where(taken, got, sb).to(torch.int32), torch.where(taken, 0.0, s["weight"])


def run(state):
    return {"chunk": _run_chunk, "evict": _run_evict}[state["case"]["op"]](state)


# ---- the definitions in binary64 -----------------------------------------------------------------

def _exact_evict(s):
    c = s["case"]
    bs, table, weight = c["block_size"], s["slot_block"].tolist(), s["weight"].double().tolist()
    for r, (n, t) in enumerate(zip(*_lengths(c))):
        new = [b for b in range(n // bs, (n + t - 1) // bs + 1) if b * bs >= n]
        for sb, w in zip(table[r], weight[r]):
            held = set(sb)
            wanted = [b for b in new if b not in held]
            rank = []
            for i, b in enumerate(sb):
                if b < 0 or (b * bs >= n and b not in new):
                    rank.append((0, 0.0, i))
                elif b * bs >= c["sinks"] and (b + 1) * bs <= n - c["recent"]:
                    rank.append((1, w[i], i))
            m = min(len(wanted), len(rank))
            if m:
                for i, b in zip(sorted(x[2] for x in sorted(rank)[:m]), wanted[-m:]):
                    sb[i], w[i] = b, 0.0
    dev = s["weight"].device
    return torch.tensor(table, dtype=torch.int32, device=dev), torch.tensor(weight, dtype=torch.float64, device=dev)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(s)
    H, kb, bs, d = case["kv_heads"], case["slots"], case["block_size"], case["head_dim"]
    g, dev = case["q_heads"] // H, s["q"].device
    out, lse, weight = s["out"].double(), s["lse"].double(), s["weight"].double()
    for r, (n, t) in enumerate(zip(*_lengths(case))):
        for h in range(H if t else 0):
            first = s["slot_block"][r, h].long()[:, None] * bs
            where = (first + torch.arange(bs, device=dev)).reshape(-1)
            keep = ((first >= 0).expand(kb, bs).reshape(-1) & (where < n + t)).nonzero()[:, 0]
            where = where[keep]
            k = s["pool"][r, h, :, 0].reshape(-1, d)[keep].double()
            v = s["pool"][r, h, :, 1].reshape(-1, d)[keep].double()
            drawn = torch.zeros(kb * bs, device=dev, dtype=torch.float64)
            for i0 in range(0, t, 512):  # rows at a time
                i1 = min(t, i0 + 512)
                mine = torch.arange(n + i0, n + i1, device=dev)[:, None]
                no = where > mine
                if case["window"]:
                    no = no | ((where <= mine - case["window"]) & (where >= case["sinks"]))
                for j in range(h * g, h * g + g):
                    z = (s["q"][r, i0:i1, j].double() @ k.T / math.sqrt(d)).masked_fill(no, -math.inf)
                    lse[r, i0:i1, j] = torch.logsumexp(z, -1)
                    p = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)  # a row that sees nothing is zero
                    out[r, i0:i1, j] = p @ v
                    drawn.index_add_(0, keep, p.sum(0))
            weight[r, h] += drawn.view(kb, bs).sum(-1)
    return (out, lse, weight) if case["weigh"] else (out, lse)
