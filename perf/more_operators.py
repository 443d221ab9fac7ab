"""The operators of a decode step with drafted tokens, measured: which cases, their plain forms, and what they cost at least.

One step of speculative decoding over the int8 key/value cache:

* rotary: rotary positions on the heads of each token;
* append: keys, rotated on the way, and values into the cache (read back, so that what it holds is seen);
* tree: attention of a tree of drafted tokens at the end of each sequence over the cache;
* verify: which drafted tokens are kept and which one follows them, from given random numbers.

``run`` computes the plain form in elementary torch operations, or, where ``own``
is true, calls the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
TINY = float(np.finfo(np.float32).tiny)


# ------------------------------------------------------------------- cases ---

def _rotary(name, rows, heads, head_dim, rotary_dim, interleaved, far, magnitude, dtype):
    return {"name": name, "op": "rotary", "rows": rows, "heads": heads, "head_dim": head_dim, "rotary_dim": rotary_dim,
            "interleaved": interleaved, "far": far, "magnitude": magnitude, "dtype": dtype}


def _append(name, batch, kv_heads, head_dim, rotary_dim, interleaved, block, start, new, reach, dtype):
    return {"name": name, "op": "append", "batch": batch, "kv_heads": kv_heads, "head_dim": head_dim,
            "rotary_dim": rotary_dim, "interleaved": interleaved, "magnitude": 1.0, "block": block, "lo": start[0],
            "hi": start[1], "new_lo": new[0], "new_hi": new[1], "reach": reach, "dtype": dtype}


def _tree(name, batch, heads, kv_heads, head_dim, block, prefix, nodes, reach, dtype, window=0, lse=False):
    return {"name": name, "op": "tree", "batch": batch, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "block": block, "lo": prefix[0], "hi": prefix[1], "new_lo": nodes[0], "new_hi": nodes[1], "reach": reach,
            "dtype": dtype, "window": window, "lse": lse}


def _verify(name, batch, nodes, reach, vocab, dtype, drawn=True):
    return {"name": name, "op": "verify", "batch": batch, "lo": 0, "hi": 0, "new_lo": nodes[0], "new_hi": nodes[1],
            "reach": reach, "vocab": vocab, "dtype": dtype, "drawn": drawn}


def listed():
    return [
        # a decode batch's query heads: latency
        _rotary("rotary 64 tokens", 64, 32, 128, 128, False, 8000, 1.0, "bf16"),
        # prompts at far positions of a scaled context, 64 heads: bytes
        _rotary("rotary 16384 tokens", 16384, 64, 128, 128, False, 131071, 1.2079, "bf16"),
        # fp32, neighbours as pairs, part of a head whose size is no power of two
        _rotary("rotary part of the head, fp32", 1777, 12, 80, 32, True, 4000, 1.0, "f32"),
        # a decode step: 64 sequences append one token each to partly filled blocks
        _append("append, 64 sequences", 64, 8, 128, 128, False, 16, (1, 4095), (1, 1), 0, "bf16"),
        # chunked prompts of several users, some far into their contexts
        _append("append prompts", 16, 8, 128, 128, False, 64, (0, 50000), (1000, 4099), 0, "bf16"),
        # drafted trees of a small-headed model in fp32: positions are depths, part of the head turns
        _append("append trees, fp32", 61, 12, 64, 32, True, 32, (0, 700), (1, 64), 5, "f32"),
        # one user's drafted tree over a short context: latency
        _tree("tree 1 sequence", 1, 32, 8, 128, 16, (1000, 1000), (16, 16), 4, "bf16"),
        # ragged trees of a batch of grouped heads
        _tree("tree 16 sequences", 16, 32, 8, 128, 64, (500, 8000), (24, 64), 6, "bf16"),
        # a large batch over long contexts, 8 query heads for each of keys and values: matrix rate
        _tree("tree 64 sequences", 64, 64, 8, 128, 64, (100, 16001), (33, 64), 8, "bf16"),
        # fp32 queries of a small-headed model, sliding window, single tokens among the trees
        _tree("tree window, fp32", 9, 12, 12, 64, 32, (0, 2047), (1, 61), 5, "f32", window=300, lse=True),
        # one user's drafts: latency
        _verify("verify 1 sequence", 1, (8, 8), 3, 32000, "f32"),
        # a batch of trees over a large vocabulary: the rows that decide
        _verify("verify 48 sequences", 48, (16, 48), 5, 128256, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "tree", "tree", "tree", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotary":
        heads, dim = rng.choice([1, 5, 8, 12, 32, 64]), rng.choice([64, 80, 96, 128, 128, 256])
        rows = _log(rng, 1, max(1, 16384 * 64 * 128 // (heads * dim * (2 if dtype == "f32" else 1))))
        case = _rotary("", rows, heads, dim, rng.choice([dim, dim // 2, 2 * rng.randint(1, dim // 2)]), rng.random() < 0.4,
                       _log(rng, 10, 1000000), rng.choice([1.0, 1.0, 1.1386, 1.2079]), dtype)
    elif op == "append":
        batch, heads, dim = rng.randint(1, 64), rng.choice([1, 2, 4, 5, 8, 12]), rng.choice([64, 128, 128, 256])
        trees = rng.random() < 0.4
        most = max(1, min(64 if trees else 4099, 4 * 8 * 128 * 4096 // (batch * heads * dim)))
        hi, start = _log(rng, 1, most), _log(rng, 1, 20000) - 1
        case = _append("", batch, heads, dim, rng.choice([dim, dim, dim // 2, 2 * rng.randint(1, dim // 2)]),
                       rng.random() < 0.4, rng.choice([16, 32, 64, 128]), (start // 2, start), (rng.randint(1, hi), hi),
                       rng.randint(1, 8) if trees else 0, dtype)
    elif op == "tree":
        batch, kv, dim = rng.randint(1, 64), rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 256])
        group, nodes = rng.choice([1, 2, 3, 4, 7, 8]), _log(rng, 2, 64)
        most = max(16, min(16000, 64 * 8 * 128 * 3000 // (batch * kv * dim)))
        hi = _log(rng, 16, most)
        case = _tree("", batch, kv * group, kv, dim, rng.choice([16, 32, 64, 128]), (rng.choice([0, rng.randint(1, hi), hi]), hi),
                     (rng.randint(1, nodes), nodes), rng.randint(1, 8), dtype, rng.choice([0, 0, 0, _log(rng, 4, 2000)]),
                     rng.random() < 0.4)
    else:
        batch, vocab = rng.randint(1, 48), rng.choice([32000, 128256, _log(rng, 100, 152000) | 1])
        most = max(1, min(64, 48 * 30 * 128256 // (batch * vocab)))
        nodes = _log(rng, 1, most)
        case = _verify("", batch, (rng.randint(1, nodes), nodes), rng.randint(1, 8), vocab, dtype, rng.random() < 0.7)
    del case["name"]
    return case


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], both met when n > 1, in a mixed order: the same for every seed."""
    order = sorted(range(n), key=lambda i: (i * 0.6180339887498949) % 1.0)
    return [hi if n == 1 else lo + (hi - lo) * k // (n - 1) for k in order]


def _lengths(case):
    """(tokens before, tokens of the call) of each sequence."""
    n = case["batch"]
    return _spread(n, case["lo"], case["hi"]), _spread(n, case["new_lo"], case["new_hi"])[::-1]


def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "rotary":
        values, pairs = case["rows"] * case["heads"] * case["head_dim"], case["rows"] * case["rotary_dim"] // 2
        return {"bytes": 2 * values * e + 4 * case["rows"] + 4 * case["rotary_dim"], "flops": 6.0 * pairs * case["heads"]}
    a, b = _lengths(case)
    if case["op"] == "verify":       # the root's probabilities, at least, against the draft's
        return {"bytes": case["batch"] * case["vocab"] * e * (1 + case["drawn"]) + 16 * sum(b) + 8 * case["batch"],
                "flops": 3.0 * case["batch"] * case["vocab"]}
    h, d, bs = case["kv_heads"], case["head_dim"], case["block"]
    if case["op"] == "append":
        back = sum(s % bs + n for s, n in zip(a, b))
        blocks = sum(-(-(s % bs + n) // bs) for s, n in zip(a, b))
        return {"bytes": 2 * sum(b) * h * d * (e + 1) + 2 * back * h * d * 3 + 16 * blocks * h + 4 * sum(b),
                "flops": sum(b) * h * (6.0 * d + 3.0 * case["rotary_dim"])}
    pairs = keys = blocks = 0
    for prefix, n in zip(a, b):
        seen = min(prefix, case["window"]) if case["window"] else prefix
        pairs, keys, blocks = pairs + n * seen + 2 * n - 1, keys + seen + n, blocks + -(-(seen + n) // bs)
    rows = sum(b) * case["heads"]
    return {"bytes": 2 * keys * h * d + 8 * blocks * h + 2 * rows * d * e + 4 * rows * case["lse"] + 4 * sum(b),
            "flops": 4.0 * pairs * case["heads"] * d}


# ------------------------------------------------------------------ inputs ---

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _offsets(v):
    return _ints(np.concatenate([[0], np.cumsum(v)]).tolist())


def _cache(case, length, gen):
    """A cache that holds `length` tokens of each sequence in shuffled blocks: codes of normal values, and scales."""
    h, d, bs = case["kv_heads"], case["head_dim"], case["block"]
    blocks = [-(-n // bs) for n in length]
    nb = sum(blocks) + 3
    ids = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32)
    used, table = 0, torch.full((len(length), max(1, max(blocks))), -1, dtype=torch.int32, device=DEV)
    for b, m in enumerate(blocks):
        table[b, :m] = ids[used:used + m]
        used += m
    code = lambda *shape: (torch.randn(shape, generator=gen, device=DEV) * 36).round_().clamp_(-127, 127).to(torch.int8)
    scale = lambda x: x / 36 * torch.exp(0.3 * torch.randn((nb, h), generator=gen, device=DEV))
    return (code(nb, h, bs, d), code(nb, h, d, bs), scale(1.0), scale(0.5)), table


def _trees(nodes, reach, gen):
    """Parents and depths of one tree a sequence, row after row: node 0 is the root, a node hangs below one of the
    `reach` nodes before it."""
    width = max(nodes)
    i = torch.arange(width, device=DEV)
    back = (torch.rand((len(nodes), width), generator=gen, device=DEV) * torch.minimum(i, _ints(reach))).long()
    parents = i - 1 - back
    parents[:, 0] = -1
    depth = torch.zeros_like(parents)
    for k in range(1, width):
        depth[:, k] = depth.gather(1, parents[:, k:k + 1])[:, 0] + 1
    there = i < _ints(nodes)[:, None]
    return parents[there].int(), depth[there].int()


def _frequencies(n):
    return 10000.0 ** (-torch.arange(0, n, 2, dtype=torch.float64, device=DEV) / n)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[case["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)
    if case["op"] == "rotary":
        rows = case["rows"]
        first = torch.randint(0, case["far"] + 1, (rows // 1000 + 1, 1), generator=gen, device=DEV)
        run_of = (first + torch.arange(1000, device=DEV)).reshape(-1)[:rows]     # stretches of up to 1000 positions
        return {"case": case, "x": normal(rows, case["heads"], case["head_dim"]).to(t), "positions": run_of.int(),
                "frequencies": _frequencies(case["rotary_dim"])}
    a, b = _lengths(case)
    offsets = _offsets(b)
    if case["op"] == "verify":
        parents, _ = _trees(b, case["reach"], gen)
        vocab, rows = case["vocab"], sum(b)
        logits = normal(rows, vocab) * 2.5
        target = torch.softmax(logits, 1)
        draft = torch.softmax(logits.add_(normal(rows, vocab), alpha=0.8), 1)
        del logits
        tokens = torch.zeros(rows, dtype=torch.int32, device=DEV)
        at = 0
        for n in b:      # each node's token is drawn from the draft at its parent
            up = parents[at:at + n].clamp(min=0).long() + at
            noise = torch.empty((n, vocab), device=DEV).exponential_(generator=gen)
            tokens[at:at + n] = (draft[up] / noise).argmax(1)
            at += n
        uniform = lambda n: torch.rand(n, generator=gen, device=DEV)
        return {"case": case, "target": target.to(t), "draft": draft.to(t) if case["drawn"] else None, "tokens": tokens,
                "parents": parents, "offsets": offsets, "u": uniform(rows), "r": uniform(case["batch"]), "width": max(b)}
    cache, table = _cache(case, [s + n for s, n in zip(a, b)], gen)
    h, d, bs = case["kv_heads"], case["head_dim"], case["block"]
    st = {"case": case, "cache": cache, "table": table, "offsets": offsets}
    if case["op"] == "tree":
        st["parents"], _ = _trees(b, case["reach"], gen)
        st |= {"q": (1.5 * normal(sum(b), case["heads"], d)).to(t), "lengths": _ints([s + n for s, n in zip(a, b)]),
               "width": max(b), "keys": max(s + n for s, n in zip(a, b))}
        return st
    back = [s % bs + n for s, n in zip(a, b)]
    # heads of different spread, some tokens several times larger than the rest
    big = 1 + 3 * (torch.rand((sum(b), 1, 1), generator=gen, device=DEV) < 0.05)
    spread = torch.exp(0.3 * normal(1, h, 1))
    st |= {"k": (normal(sum(b), h, d) * big * spread).to(t), "v": (0.5 * normal(sum(b), h, d) * spread).to(t),
           "starts": _ints(a), "back_offsets": _offsets(back), "back_rows": sum(back),
           "back_starts": _ints([s - s % bs for s in a]), "frequencies": _frequencies(case["rotary_dim"]), "positions": None}
    if case["reach"]:
        _, depth = _trees(b, case["reach"], gen)
        st["positions"] = (torch.repeat_interleave(st["starts"], _ints(b)) + depth).int()
    return st


# ------------------------------------------------------------- plain forms ---

def _rows(offsets, starts, rows):
    """Sequence and position of each row of a ragged batch."""
    r = torch.arange(rows, dtype=torch.int32, device=DEV)
    seq = torch.searchsorted(offsets, r, right=True, out_int32=True).sub_(1)
    return seq, starts[seq] + r - offsets[seq]


def _turn(x, positions, frequencies, case):
    """The pairs of x [rows, heads, dim] turned by position times frequency, in fp32."""
    x, n = x.float(), case["rotary_dim"]
    angle = positions.double()[:, None] * frequencies
    cos, sin = ((f(angle) * case["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if case["interleaved"] else (x[..., :n // 2], x[..., n // 2:n])
    pair = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(pair, -1).flatten(-2) if case["interleaved"] else torch.cat(pair, -1)
    return torch.cat([turned, x[..., n:]], -1)


def _scale(amax):
    s = amax / torch.full_like(amax, 127.0)
    return torch.where(s < TINY, torch.zeros_like(s), s)


def _inverse(s):
    return torch.where(s > 0, torch.reciprocal(s), torch.zeros_like(s))


def _plain_write(st, x, codes, scales, transposed):
    """Quantize the rows x into one of the cache's halves (codes [nb, h, bs, d], or [nb, h, d, bs])."""
    bs = st["case"]["block"]
    starts, table = st["starts"], st["table"]
    seq, pos = _rows(st["offsets"], starts, x.shape[0])
    block, slot = table[seq, pos // bs].long(), (pos % bs).long()
    amax = torch.zeros_like(scales).index_reduce_(0, block, x.abs().amax(2), "amax")
    # blocks that hold earlier tokens of their sequence keep at least their scale; their codes follow it when it grows
    part = (starts % bs > 0) & (st["offsets"][1:] > st["offsets"][:-1])
    first = table[torch.arange(len(starts), device=DEV), torch.where(part, starts // bs, 0)].long()[part]
    new = _scale(amax)
    new[first] = torch.maximum(new[first], scales[first])
    old = codes[first].float()
    ratio = torch.where(new[first] > scales[first], scales[first] * _inverse(new[first]), torch.ones_like(new[first]))
    held = torch.arange(bs, device=DEV)[None, :] < (starts % bs)[part][:, None]
    held = held[:, None, None, :] if transposed else held[:, None, :, None]
    codes[first] = torch.where(held, (old * ratio[:, :, None, None]).round(), old).to(torch.int8)
    scales[block] = new[block]
    c = (x * _inverse(new[block])[:, :, None]).round().clamp(-127, 127).to(torch.int8)
    if transposed:
        codes[block, :, :, slot] = c
    else:
        codes[block, :, slot] = c


def _plain_read(st, codes, scales, transposed):
    seq, pos = _rows(st["back_offsets"], st["back_starts"], st["back_rows"])
    bs = st["case"]["block"]
    block, slot = st["table"][seq, pos // bs].long(), (pos % bs).long()
    c = codes[block, :, :, slot] if transposed else codes[block, :, slot]
    return (c.float() * scales[block][:, :, None]).to(torch.bfloat16)


def _plain_append(st):
    k, v, ks, vs = st["cache"]
    positions = st["positions"] if st["positions"] is not None else _rows(st["offsets"], st["starts"], st["k"].shape[0])[1]
    _plain_write(st, _turn(st["k"], positions, st["frequencies"], st["case"]), k, ks, False)
    _plain_write(st, st["v"].float(), v, vs, True)
    return _plain_read(st, k, ks, False), _plain_read(st, v, vs, True)


def _padded(st, rows):
    """Row of each node of each sequence [batch, width], and which of them there are."""
    at = torch.arange(st["width"], device=DEV)
    return (st["offsets"][:-1, None] + at).clamp(max=rows - 1).long(), at < (st["offsets"][1:] - st["offsets"][:-1])[:, None]


def _plain_tree(st):
    case = st["case"]
    h, d, bs, heads, width = case["kv_heads"], case["head_dim"], case["block"], case["heads"], st["width"]
    k, v, ks, vs = st["cache"]
    table, q = st["table"].clamp(min=0).long(), st["q"].float()
    batch, n = table.shape[0], table.shape[1] * bs
    keys = (k[table].float() * ks[table][..., None, None]).permute(0, 2, 4, 1, 3).reshape(batch, h, d, n)
    vals = (v[table].float() * vs[table][..., None, None]).permute(0, 2, 1, 4, 3).reshape(batch, h, n, d)
    # queries padded to [batch, kv head, group * nodes, d]
    row, there = _padded(st, q.shape[0])
    pad = q[row].reshape(batch, width, h, heads // h, d).permute(0, 2, 3, 1, 4).reshape(batch, h, -1, d)
    s = torch.matmul(pad.contiguous() * (1 / math.sqrt(d)), keys.contiguous()).reshape(batch, heads, width, n)
    # the path from each node up: steps[b, i, j] = how far above node i its ancestor j is, -1 where it is none
    steps = torch.full((batch, width, width + 1), -1, device=DEV)
    up, node = torch.where(there, st["parents"][row], -1), torch.arange(width, device=DEV).repeat(batch, 1)
    depth = torch.zeros_like(node)
    for far in range(width):
        steps.scatter_(2, torch.where(node >= 0, node, width)[..., None], far)
        node = torch.where(node >= 0, up.gather(1, node.clamp(min=0)), -1)
        depth += node >= 0
    base = st["lengths"] - there.sum(1)
    j = torch.arange(n, device=DEV)
    in_tree = (j - base[:, None]).clamp(0, width)      # column `width` is nobody's ancestor
    far = steps.scatter(2, torch.full_like(steps[..., :1], width), -1).gather(2, in_tree[:, None].expand(-1, width, -1))
    before = j < base[:, None, None]
    gap = torch.where(before, base[:, None, None] + depth[..., None] - j, far)
    seen = before | (far >= 0)
    if case["window"]:
        seen = seen & (gap < case["window"])
    s.masked_fill_(~seen[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(torch.where(m > -math.inf, m, 0)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(batch, h, -1, n), vals.contiguous()).reshape(batch, heads, width, d)
    o = o / torch.where(total > 0, total, 1)
    seq, i = _rows(st["offsets"], torch.zeros_like(st["lengths"]), q.shape[0])
    out = o[seq, :, i].to(st["q"].dtype)
    return (out, (m + torch.log(total))[seq, :, i, 0]) if case["lse"] else out


def _plain_verify(st):
    target, draft, offsets = st["target"], st["draft"], st["offsets"]
    rows, vocab = target.shape
    batch = len(offsets) - 1
    row, there = _padded(st, rows)
    b, first = torch.arange(batch, device=DEV), offsets[:-1].long()
    cur, z = torch.zeros_like(first), torch.ones(batch, dtype=torch.float64, device=DEV)
    left = target[row[:, 0]].double().clamp(min=0)      # what the token is drawn from, times z
    kept = torch.zeros_like(there)
    kept[:, 0] = there[:, 0]
    for i in range(1, st["width"]):
        at = row[:, i]
        x = st["tokens"][at].long()
        tried = there[:, i] & (st["parents"][at] == cur) & (x >= 0) & (x < vocab)
        x = x.clamp(0, vocab - 1)
        q = draft[first + cur].double() if draft is not None else torch.zeros_like(left).scatter_(1, x[:, None], 1.0)
        take = tried & (st["u"][at].double() * z * q[b, x] < left[b, x])
        drop = tried & ~take
        rest = (left - z[:, None] * q).clamp(min=0) if draft is not None else left.scatter(1, x[:, None], 0.0)
        z_rest = rest.sum(1) if draft is not None else z - left[b, x]
        left = torch.where(take[:, None], target[at].double().clamp(min=0), torch.where(drop[:, None], rest, left))
        z = torch.where(take, 1.0, torch.where(drop, z_rest, z))
        cur = torch.where(take, i, cur)
        kept[:, i] = take
    none = left.sum(1, keepdim=True) == 0
    left = torch.where(none, target[first + cur].double().clamp(min=0), left)
    run_sum = left.cumsum(1)
    total = run_sum[:, -1:]
    at = torch.arange(vocab, device=DEV)
    over = torch.where(run_sum > st["r"].double()[:, None] * total, at, vocab).amin(1)
    last = torch.where(left > 0, at, -1).amax(1)
    token = torch.where(over < vocab, over, last)
    counts = kept.sum(1)
    token = torch.where((counts > 0) & (total[:, 0] > 0) & torch.isfinite(total[:, 0]), token, -1)
    path = torch.where(kept, torch.arange(st["width"], device=DEV), st["width"]).sort(1).values
    path = torch.where(path < st["width"], path, -1)
    return {"path": path[there].int(), "counts": counts.int(), "next": token.int()}


def run(state):
    case = state["case"]
    if own:
        from post_int4_weight_amd import api
        if case["op"] == "verify":
            path, counts, token = api.verify_drafts(state["target"], state["tokens"], state["parents"], state["offsets"],
                                                    state["u"], state["r"], draft=state["draft"])
            return {"path": path, "counts": counts, "next": token}
        if case["op"] != "tree":
            rotary = api.Rotary(state["frequencies"], case["magnitude"], case["interleaved"])
        if case["op"] == "rotary":
            return api.rotary_apply(state["x"], rotary, state["positions"])
        cache = api.KVCacheInt8(*state["cache"])
        if case["op"] == "tree":
            return api.attention_int8_tree(state["q"], cache, state["offsets"], state["lengths"], state["table"],
                                           state["parents"], window=case["window"], return_lse=case["lse"])
        api.kv_cache_append_int8(cache, state["k"], state["v"], state["offsets"], state["starts"], state["table"], rotary,
                                 positions=state["positions"])
        k, v = api.kv_cache_read_int8(cache, state["back_offsets"], state["back_starts"], state["table"],
                                      state["back_rows"])
    else:
        if case["op"] == "verify":
            return _plain_verify(state)
        if case["op"] == "rotary":
            return _turn(state["x"], state["positions"], state["frequencies"], case).to(state["x"].dtype)
        if case["op"] == "tree":
            return _plain_tree(state)
        k, v = _plain_append(state)
    # the codes come back as the values they stand for; the scales are the cache's own buffers
    return {"k": k, "v": v, "k_scales": state["cache"][2], "v_scales": state["cache"][3]}


# ---------------------------------------------------------- in 64 bits -------

def _exact_turn(x, positions, frequencies, case):
    """As complex numbers: a pair turns by a product with e^(i t)."""
    y, n = x.double().clone(), case["rotary_dim"]
    t = torch.outer(positions.double(), frequencies)
    factor = torch.polar(torch.full_like(t, case["magnitude"]), t)[:, None, :]
    pick = (slice(0, n, 2), slice(1, n, 2)) if case["interleaved"] else (slice(0, n // 2), slice(n // 2, n))
    z = torch.complex(y[..., pick[0]].contiguous(), y[..., pick[1]].contiguous()) * factor
    y[..., pick[0]], y[..., pick[1]] = z.real, z.imag
    return y


def _exact_append(st):
    """Sequence by sequence and block by block, from the definition; values of the blocks that are read back."""
    case = st["case"]
    bs = case["block"]
    a, b = _lengths(case)
    where = st["positions"] if case["reach"] else torch.cat([torch.arange(s, s + n, device=DEV) for s, n in zip(a, b)])
    rows_of = {"k": _exact_turn(st["k"], where, st["frequencies"], case), "v": st["v"].double()}
    table, given = st["table"].tolist(), {}
    found = {"k_scales": st["cache"][2].double(), "v_scales": st["cache"][3].double()}
    for half, at in (("k", 0), ("v", 1)):
        codes, scales, rows, first = st["cache"][at], found[half + "_scales"], [], 0
        for i, (start, new) in enumerate(zip(a, b)):
            lo, end = start - start % bs, start + new
            ids = torch.tensor([table[i][p // bs] for p in range(lo, end, bs)], device=DEV)
            held = codes[ids].double()
            held = held.transpose(2, 3) if half == "v" else held            # [blocks, h, bs, d]
            x = torch.zeros(len(ids) * bs, *st[half].shape[1:], dtype=torch.float64, device=DEV)
            x[start - lo:end - lo] = rows_of[half][first:first + new]
            x = x.reshape(len(ids), bs, *x.shape[1:]).transpose(1, 2)
            s = x.abs().amax((2, 3)) / 127.0
            if start > lo:
                s[0] = torch.maximum(s[0], scales[ids[0]])
                x[0, :, :start - lo] = held[0, :, :start - lo] * scales[ids[0]][:, None, None]
            scales[ids] = s
            s = s[:, :, None, None]
            value = torch.round(x / torch.where(s > 0, s, 1.0)) * s
            rows.append(value.transpose(1, 2).reshape(-1, *value.shape[1:2], value.shape[3])[:end - lo])
            first += new
        given[half] = torch.cat(rows)
    return {**given, **found}


def _exact_tree(st):
    """Node by node which keys it sees, then a softmax for each sequence and kv head."""
    case = st["case"]
    h, d, bs, window = case["kv_heads"], case["head_dim"], case["block"], case["window"]
    k, v, ks, vs = st["cache"]
    parents, outs, lses, first = st["parents"].tolist(), [], [], 0
    for b, (prefix, n) in enumerate(zip(*_lengths(case))):
        mask = np.zeros((n, prefix + n), dtype=bool)
        for i in range(n):
            line, j = [], i
            while j >= 0:
                line.append(j)
                j = parents[first + j]
            depth = len(line) - 1
            mask[i, max(0, prefix + depth - window + 1) if window else 0:prefix] = True
            mask[i, [prefix + x for x in (line[:window] if window else line)]] = True
        seen = torch.tensor(mask, device=DEV)
        q = st["q"][first:first + n].double().reshape(n, h, -1, d)
        first += n
        ids = st["table"][b, :-(-(prefix + n) // bs)].long()
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device=DEV)
        for g in range(h):
            key = (k[ids, g].double() * ks[ids, g].double()[:, None, None]).reshape(-1, d)[:prefix + n]
            val = (v[ids, g].double() * vs[ids, g].double()[:, None, None]).transpose(1, 2).reshape(-1, d)[:prefix + n]
            logit = (q[:, g].reshape(-1, d) @ key.T / math.sqrt(d)).reshape(n, -1, prefix + n)
            logit = logit.masked_fill(~seen[:, None], -math.inf)
            out[:, g] = (torch.softmax(logit, 2).reshape(-1, prefix + n) @ val).reshape(n, -1, d)
            lse[:, g] = torch.logsumexp(logit, 2)
        outs.append(out.reshape(n, -1, d))
        lses.append(lse.reshape(n, -1))
    return (torch.cat(outs), torch.cat(lses)) if case["lse"] else torch.cat(outs)


def _exact_verify(st):
    """Sequence by sequence: the walk down the tree, on one row of probabilities at a time."""
    offsets, parents, tokens = st["offsets"].tolist(), st["parents"].tolist(), st["tokens"].tolist()
    u, r, vocab = st["u"].tolist(), st["r"].tolist(), st["target"].shape[1]
    path, counts, after = [], [], []
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        line, node, taken = [], 0 if hi > lo else None, True
        while taken and node is not None:
            line.append(node)
            weight, z, taken = st["target"][lo + node].double().clamp(min=0), 1.0, False
            for i in range(node + 1, hi - lo):
                x = tokens[lo + i]
                if parents[lo + i] != node or not 0 <= x < vocab:
                    continue
                q = 1.0 if st["draft"] is None else float(st["draft"][lo + node, x])
                if u[lo + i] * z * q < float(weight[x]):
                    node, taken = i, True
                    break
                if st["draft"] is None:
                    z -= float(weight[x])
                    weight[x] = 0
                else:
                    weight = torch.relu(weight - z * st["draft"][lo + node].double())
                    z = float(weight.sum())
        path += line + [-1] * (hi - lo - len(line))
        counts.append(len(line))
        token = -1
        if line:
            if float(weight.sum()) == 0:
                weight = st["target"][lo + line[-1]].double().clamp(min=0)
            sums = torch.cumsum(weight, 0)
            total = float(sums[-1])
            if 0 < total < math.inf:
                token = int(torch.searchsorted(sums, torch.tensor(r[b] * total, dtype=torch.float64, device=DEV), right=True))
                token = token if token < vocab else int(torch.nonzero(weight)[-1])
        after.append(token)
    return {"path": _ints(path), "counts": _ints(counts), "next": _ints(after)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_turn(st["x"], st["positions"], st["frequencies"], case)
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify}[case["op"]](st)
