"""GPU: which drafted tokens are kept (verify_drafts) against the fp64 oracle (oracle/drafts.py): whole numbers, equal.

Both form products and sums of fp32 (bf16) probabilities in fp64 and differ in the order of sums alone, by 2^-53 of a sum a
term; a decision could differ only within that of its border, where random inputs of 24 bits do not fall. Inputs in
multiples of 2^-10, whose sums are exact, test the borders themselves.
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import drafts as ref
from test_gpu_14_kv_cache_int8 import DTYPES, _ints, _offsets
from test_gpu_22_attention_tree import _trees

pytestmark = pytest.mark.gpu


def _roots(trees):
    """One root each: nodes without a parent hang below node 0."""
    return [[-1] + [max(p, 0) for p in t[1:]] if t else [] for t in trees]


def _inputs(nodes, vocab, dtype, drawn, seed, gpu, near=0.8, reach=3):
    gen = torch.Generator().manual_seed(seed)
    rows, trees = sum(nodes), _roots(_trees(nodes, reach, seed))
    logits = 2.5 * torch.randn(rows, vocab, generator=gen)
    target = torch.softmax(logits, 1).to(DTYPES[dtype])
    draft = torch.softmax(logits + near * torch.randn(rows, vocab, generator=gen), 1).to(DTYPES[dtype])
    tokens, first = np.zeros(rows, dtype=np.int64), 0
    for t in trees:
        for i, p in enumerate(t):
            if i:
                tokens[first + i] = int(torch.multinomial(draft[first + p].float(), 1, generator=gen))
        first += len(t)
    u, r = torch.rand(rows, generator=gen), torch.rand(len(nodes), generator=gen)
    return dict(target=target.to(gpu), draft=draft.to(gpu) if drawn else None, tokens=tokens, trees=trees, u=u, r=r)


def _call(api, d, gpu, **out):
    flat = [p for t in d["trees"] for p in t]
    off = _offsets([len(t) for t in d["trees"]])
    return api.verify_drafts(d["target"], _ints(d["tokens"], gpu), _ints(flat, gpu), _ints(off, gpu), d["u"].to(gpu),
                             d["r"].to(gpu), draft=d["draft"], **out)


def _check(api, d, gpu):
    path, counts, token = (t.cpu().tolist() for t in _call(api, d, gpu))
    off = _offsets([len(t) for t in d["trees"]])
    target, draft = to64(d["target"]), None if d["draft"] is None else to64(d["draft"])
    for b, t in enumerate(d["trees"]):
        at = slice(off[b], off[b + 1])
        kept, after = ref.verify(target[at], None if draft is None else draft[at], d["tokens"][at], t,
                                 d["u"][at].double().numpy(), float(d["r"][b]))
        assert path[at] == kept + [-1] * (len(t) - len(kept)), (b, path[at], kept)
        assert counts[b] == len(kept) and token[b] == after, (b, token[b], after)
    return counts


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 63, 257, 4096, 4099, 32000, 50257, 131073])
def test_trees(gpu, vocab, dtype, drawn):
    from post_int4_weight_amd import api
    announce(f"verify vocab={vocab} {dtype} drawn={drawn}")
    nodes = [1, 5, 0, 9, 17, 2, 33, 4]
    counts = _check(api, _inputs(nodes, vocab, dtype, drawn, vocab + drawn, gpu), gpu)
    if vocab > 60 and drawn:      # drafts near the target are kept, and far ones are not
        assert sum(_check(api, _inputs(nodes, vocab, dtype, drawn, 7, gpu, near=0.0, reach=1), gpu)) == sum(nodes)
        assert sum(counts) < sum(nodes)


@pytest.mark.parametrize("drawn", [True, False])
def test_many_children(gpu, drawn):
    """Bushes whose nodes have up to hundreds of children, the largest trees, the same token twice among siblings."""
    from post_int4_weight_amd import api
    announce(f"verify, many children drawn={drawn}")
    d = _inputs([512, 300, 65, 64], 700, "f32", drawn, 3, gpu, near=3.0, reach=500)
    d["trees"][1] = [-1] + [0] * 299
    d["tokens"][513:812] = np.arange(299) % 40 + 600
    d["u"][513:812] = 0.9999
    _check(api, d, gpu)


def test_borders(gpu):
    """Probabilities in multiples of 2^-10 and random numbers on the borders: kept below, not kept at them."""
    from post_int4_weight_amd import api
    announce("verify, borders")
    vocab, e = 5000, 2.0 ** -24
    p, q = np.zeros(vocab), np.zeros(vocab)
    p[[3, 40, 700, 2048, 4999]] = np.array([256, 128, 512, 64, 64]) / 1024
    q[[3, 40, 700, 2048, 4000]] = np.array([512, 128, 128, 128, 128]) / 1024
    cum = np.cumsum(p)
    cases = [(3, 0.5 - e, 0), (3, 0.5, 0), (40, 1 - e, 0), (4000, 0, 0)] + [
        (3, 0.75, r) for x in (0, 128, 384) for r in (x / 512, x / 512 + e, max(0, x / 512 - e), 1 - e)]
    for drawn in (True, False):
        todo = cases if drawn else [(700, 0.5 - e, 0), (700, 0.5, 0)] + [(4000, 0.75, float(r)) for c in np.unique(cum)[1:-1]
                                                                           for r in (c, c - e, c + e)]
        n = len(todo)
        both = lambda x: torch.tensor(np.tile(x, (2 * n, 1)), dtype=torch.float32).to(gpu)
        tokens = np.array([t for x, _, _ in todo for t in (0, x)])
        d = dict(target=both(p), draft=both(q) if drawn else None, tokens=tokens, trees=[[-1, 0]] * n,
                 u=torch.tensor([v for _, u, _ in todo for v in (0.5, u)]), r=torch.tensor([r for _, _, r in todo]))
        _check(api, d, gpu)


def test_nothing_left_and_not_finite(gpu):
    """Where nothing is left the target itself is drawn from; sums that are no positive number give -1; tokens outside the
    vocabulary, parents that are none and negative probabilities count for nothing."""
    from post_int4_weight_amd import api
    announce("verify, nothing left, not finite")
    vocab = 1000
    for drawn in (True, False):
        for dtype in DTYPES:
            d = _inputs([6] * 8, vocab, dtype, drawn, 11, gpu)
            t = d["target"]
            if drawn:      # the draft covers the target: nothing is left after a rejection
                d["draft"][0:6] = t[0:6] * 2
            else:
                t[0:6] = 0
                t[0:6, 17] = 1
                d["tokens"][0:6] = 17
            d["u"][0:6] = 1.0 if not drawn else 0.75
            t[6:12] = 0                                    # nothing at all
            t[18:24, 5] = -1.0                             # not a probability
            d["tokens"][24:30] = [0, -1, vocab, 2 ** 31 - 1, -2 ** 31, 3]
            d["trees"][5] = [-1, 1, 5, -7, 2 ** 31 - 1, 0]
            d["trees"][6] = [3, 0, 0, 1, 1, 2]             # a root with a parent
            with np.errstate(invalid="ignore"):
                _check(api, d, gpu)
            t[12:18, 100] = float("nan")
            t[42:48, 999] = float("inf")
            path, counts, token = _call(api, d, gpu)
            torch.cuda.synchronize()
            assert token[1] == -1 and token[2] == -1 and token[7] == -1
            assert (token[[0, 3, 4, 5, 6]] >= 0).all() and (token < vocab).all() and (counts >= 1).all()


def test_too_many_nodes_and_wrong_offsets(gpu):
    from post_int4_weight_amd import api
    announce("verify, too many nodes, wrong offsets")
    d = _inputs([513, 4], 64, "f32", True, 5, gpu)
    path, counts, token = _call(api, d, gpu)
    assert counts[0] == 0 and token[0] == -1 and (path[:513] == -1).all() and counts[1] > 0
    args = (d["target"][:9], _ints(d["tokens"][:9], gpu), _ints([-1] + [0] * 8, gpu))
    u, r = d["u"][:9].to(gpu), torch.rand(3).to(gpu)
    path = torch.full((9,), 77, dtype=torch.int32, device=gpu)
    for off, n in (([0, 10 ** 9, 5, -3], [9, 0, 0]), ([2, 4, 4, 7], [2, 0, 3])):
        path.fill_(77)
        _, counts, token = api.verify_drafts(*args, _ints(off, gpu), u, r, draft=d["draft"][:9], path=path)
        torch.cuda.synchronize()
        assert [int(c) > 0 for c in counts] == [x > 0 for x in n] and [int(t) >= 0 for t in token] == [x > 0 for x in n]
    assert (path[:2] == 77).all() and (path[7:] == 77).all() and (path[2:7] != 77).all()


def test_strides_streams_and_graphs(gpu):
    from post_int4_weight_amd import api
    announce("verify, strides, streams and graphs")
    nodes, vocab = [5, 9, 3], 1003
    sets = [_inputs(nodes, vocab, "bf16", True, s, gpu) for s in (1, 2)]
    for d in sets:
        d["trees"] = sets[0]["trees"]
    want = [_call(api, d, gpu) for d in sets]
    torch.cuda.synchronize()
    wide = torch.full((17, 2 * vocab + 5), 3.0, dtype=torch.bfloat16, device=gpu)
    d = dict(sets[0])
    wide[:, 1:vocab + 1], wide[:, vocab + 3:2 * vocab + 3] = d["target"], d["draft"]
    d["target"], d["draft"] = wide[:, 1:vocab + 1], wide[:, vocab + 3:2 * vocab + 3]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _call(api, d, gpu)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[0]))
    flat, off = _ints([p for t in d["trees"] for p in t], gpu), _ints(_offsets(nodes), gpu)
    held = [sets[0]["target"].clone(), sets[0]["draft"].clone(), _ints(sets[0]["tokens"], gpu), sets[0]["u"].to(gpu),
            sets[0]["r"].to(gpu)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = api.verify_drafts(held[0], held[2], flat, off, held[3], held[4], draft=held[1])
    for i in (1, 0, 1, 0):
        s = sets[i]
        for x, y in zip(held, (s["target"], s["draft"], _ints(s["tokens"], gpu), s["u"], s["r"])):
            x.copy_(y)
        for x in out:
            x.fill_(99)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want[i])), i


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 700, 4099, 131073])
@pytest.mark.parametrize("shares", [1, 2, 3, 4])
def test_workgroups_of_a_sequence(gpu, shares, vocab, dtype, drawn):
    """The same by any number of workgroups, calls that follow each other included (the state that they share starts anew)."""
    from post_int4_weight_amd import api
    announce(f"verify shares={shares} vocab={vocab} {dtype} drawn={drawn}")
    far = _inputs([9, 0, 30, 1, 600, 7], vocab, dtype, drawn, 5, gpu, near=3.0, reach=30)      # many are not kept
    far["u"].mul_(0.3).add_(0.7)
    whole = _inputs([4, 4], vocab, dtype, drawn, 6, gpu)
    if drawn:      # nothing is left
        whole["draft"][:] = whole["target"] * 2
        whole["u"][:] = 1.0
    for d in (far, whole, far):
        off = _offsets([len(t) for t in d["trees"]])
        args = (d["target"], _ints(d["tokens"], gpu), _ints([p for t in d["trees"] for p in t], gpu), _ints(off, gpu),
                d["u"].to(gpu), d["r"].to(gpu))
        path, counts, token = (x.cpu().tolist() for x in api._test_verify_drafts(shares, *args, draft=d["draft"]))
        target, draft = to64(d["target"]), to64(d["draft"]) if drawn else None
        for b, t in enumerate(d["trees"]):
            at = slice(off[b], off[b + 1])
            kept, after = [], -1
            if len(t) <= 512:
                kept, after = ref.verify(target[at], draft[at] if drawn else None, d["tokens"][at], t,
                                         d["u"][at].double().numpy(), float(d["r"][b]))
            assert path[at] == kept + [-1] * (len(t) - len(kept)) and (counts[b], token[b]) == (len(kept), after), b


def test_calls_at_once(gpu):
    """Calls on several streams, more workgroups than the card holds: each walks on whether its helpers run or not."""
    from post_int4_weight_amd import api
    announce("verify, calls at once")
    nodes, vocab, streams = [3] * 60, 100003, 6
    d = _inputs(nodes, vocab, "f32", True, 9, gpu, near=3.0, reach=1)
    d["u"].mul_(0.2).add_(0.8)
    args = (d["target"], _ints(d["tokens"], gpu), _ints([p for t in d["trees"] for p in t], gpu), _ints(_offsets(nodes), gpu),
            d["u"].to(gpu), d["r"].to(gpu))
    want = api._test_verify_drafts(4, *args, draft=d["draft"])
    assert all(torch.equal(x, y) for x, y in zip(want, _call(api, d, gpu)))
    torch.cuda.synchronize()
    side, got = [torch.cuda.Stream() for _ in range(streams)], []
    for _ in range(5):
        for s in side:
            with torch.cuda.stream(s):
                got.append(api._test_verify_drafts(4, *args, draft=d["draft"]))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, want))
