"""GPU: two bounds of the decode step with drafted tokens, taken as closely as they can be derived.

 * What the cache holds of the kept tokens after several steps. Each append rounds what it writes, and what it recodes, to
   whole steps of the block's scale, which only grows while the block holds earlier tokens: half a step of the final scale
   each. A step has two appends, the tree's and the kept rows'; the prompt's comes first. 2^-10 of a step for the roundings of
   the quotients (127 2^-23), of the turned keys (16 2^-24 of the largest value, 127 steps) and of the values read (127 2^-24).
 * Calls of verify_drafts on several streams at once give what one workgroup a sequence does, which shares no sum with
   another, and what the fp64 oracle does.
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import drafts as ref
from test_gpu_14_kv_cache_int8 import DTYPES, _ints, _offsets, _table
from test_gpu_22_attention_tree import _trees
from test_gpu_23_verify_drafts import _call, _inputs

pytestmark = pytest.mark.gpu
KV, DIM, BS = 2, 128, 16


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_cache_after_steps(gpu, dtype, interleaved):
    from post_int4_weight_amd import api
    gen, rng = torch.Generator().manual_seed(5), np.random.default_rng(6)
    rotary = api.Rotary.make(DIM, interleaved=interleaved, device=gpu)
    done = [[], [], []]      # (key, value) of the kept tokens
    batch, most = len(done), 150
    table = _table([most] * batch, BS, batch * -(-most // BS) + 1, seed=2)
    cache, tab = api.KVCacheInt8.empty(batch * -(-most // BS) + 1, KV, DIM, BS, device=gpu), _ints(table, gpu)

    def rows(n, grow):
        return [(grow * torch.randn(n, KV, DIM, generator=gen)).to(DTYPES[dtype]) for _ in range(2)]

    def append(new, positions=None):
        k, v = (torch.cat([x[i] for x in new]).to(gpu) for i in (0, 1))
        off, starts = _offsets([len(x[0]) for x in new]), [len(d) for d in done]
        api.kv_cache_append_int8(cache, k, v, _ints(off, gpu), _ints(starts, gpu), tab, rotary,
                                 positions=None if positions is None else _ints(positions, gpu))

    touched = 0
    for step, nodes in enumerate(([37, 3, 90], [9, 4, 20], [1, 17, 6], [12, 12, 3], [5, 5, 5])):
        announce(f"cache after draft step {step} {dtype} interleaved={interleaved}")
        new = [rows(n, 1 + 0.3 * step) for n in nodes]      # later rows are larger: scales grow, codes are recoded
        if step:      # a tree, of which a line is kept
            trees = [[-1] + [max(p, 0) for p in t[1:]] for t in _trees(nodes, 3, step)]
            append(new, [len(d) + len(ref.line(t, i)) - 1 for d, t in zip(done, trees) for i in range(len(t))])
            lines = [ref.line(t, int(rng.integers(0, len(t))))[::-1] for t in trees]
            new = [[x[line] for x in pair] for pair, line in zip(new, lines)]
        append(new)
        touched += 2 if step else 1
        for d, (k, v) in zip(done, new):
            d += list(zip(k, v))
        lens = [len(d) for d in done]
        at = _offsets(lens)
        k, v = api.kv_cache_read_int8(cache, _ints(at, gpu), _ints([0] * batch, gpu), tab, at[-1], out_dtype=torch.float32)
        torch.cuda.synchronize()
        for b, d in enumerate(done):
            want = [to64(torch.stack([row[i] for row in d])) for i in (0, 1)]
            want[0] = ref.turn(want[0], range(len(d)), to64(rotary.inv_freq.cpu()), 1.0, interleaved)
            ids = table[b, np.arange(len(d)) // BS]
            for got, exact, scales in ((k, want[0], cache.k_scales), (v, want[1], cache.v_scales)):
                tol = to64(scales)[ids][:, :, None] * (0.5 * touched + 2.0 ** -10)
                assert np.all(np.abs(to64(got[at[b]:at[b + 1]]) - exact) <= tol), (step, b)


@pytest.mark.parametrize("drawn", [True, False])
def test_verify_calls_at_once(gpu, drawn):
    from post_int4_weight_amd import api
    announce(f"verify, calls at once against one workgroup a sequence drawn={drawn}")
    nodes, vocab = [3] * 60, 100003
    d = _inputs(nodes, vocab, "f32", drawn, 9, gpu, near=3.0, reach=1 if drawn else 3)
    d["u"].mul_(0.2).add_(0.8)
    off = _offsets(nodes)
    args = (d["target"], _ints(d["tokens"], gpu), _ints([p for t in d["trees"] for p in t], gpu), _ints(off, gpu),
            d["u"].to(gpu), d["r"].to(gpu))
    want = api._test_verify_drafts(1, *args, draft=d["draft"])
    torch.cuda.synchronize()
    path, counts, token = (x.cpu().tolist() for x in want)
    for b, t in enumerate(d["trees"]):
        a = slice(off[b], off[b + 1])
        kept, after = ref.verify(to64(d["target"][a]), to64(d["draft"][a]) if drawn else None, d["tokens"][a], t,
                                 d["u"][a].double().numpy(), float(d["r"][b]))
        assert path[a] == kept + [-1] * (len(t) - len(kept)) and (counts[b], token[b]) == (len(kept), after), b
    side, got = [torch.cuda.Stream() for _ in range(6)], []
    for _ in range(5):
        for s in side:
            with torch.cuda.stream(s):
                got.append(api._test_verify_drafts(4, *args, draft=d["draft"]))
                got.append(_call(api, d, gpu))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, want))
