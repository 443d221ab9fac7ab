"""GPU: a decode step with drafted tokens as it is run, the operators one after the other: queries turn (rotary_apply), the
trees' keys turn and are appended with their values (kv_cache_append_int8, positions their depths), the nodes attend
(attention_int8_tree), what is kept is decided (verify_drafts), and the kept rows are appended again where the trees began.

Each operator's outputs are held against the fp64 oracle (oracle/drafts.py) on what the ones before it left. What the cache
holds of the kept tokens is off by half a step of its block's scale for each append that touched the block, at most (each
write, and each growth of the scale, rounds to whole steps of a scale that only grows while the block holds earlier tokens;
2^-10 for the roundings of a quotient).
"""
import numpy as np
import pytest
import torch

from gpu_util import announce, to64
from oracle import drafts as ref
from test_gpu_14_kv_cache_int8 import DTYPES, _ints, _offsets, _table
from test_gpu_22_attention_tree import _check, _trees

pytestmark = pytest.mark.gpu
HEADS, KV, DIM, BS, VOCAB, WORDS = 8, 2, 128, 16, 700, 97


class Model:
    """One attention layer's rows and the two models' probabilities, each a table over words (token % WORDS)."""

    def __init__(self, dtype, gpu):
        gen = torch.Generator().manual_seed(3)
        rand = lambda *s: torch.randn(*s, generator=gen).to(DTYPES[dtype]).to(gpu)
        self.q, self.k, self.v = rand(WORDS, HEADS, DIM), rand(WORDS, KV, DIM), rand(WORDS, KV, DIM)
        logits = 1.5 * torch.randn(WORDS, VOCAB, generator=gen)
        self.target = torch.softmax(logits, 1).to(DTYPES[dtype]).to(gpu)
        self.draft = torch.softmax(logits + 0.5 * torch.randn(WORDS, VOCAB, generator=gen), 1).to(DTYPES[dtype]).to(gpu)

    def propose(self, trees, last, gen):
        """Tokens of the trees' nodes: the root is the last token, the others are drawn from their parents' rows."""
        tokens = []
        for parents, root in zip(trees, last):
            mine = [root]
            for p in parents[1:]:
                mine.append(int(torch.multinomial(self.draft[mine[p] % WORDS].float().cpu(), 1, generator=gen)))
            tokens += mine
        return tokens


def _forward(api, model, cache, rotary, words, offsets, starts, lens, depths, table, parents, tokens, u, r):
    Q = api.rotary_apply(model.q[words], rotary, depths)
    api.kv_cache_append_int8(cache, model.k[words], model.v[words], offsets, starts, table, rotary, positions=depths)
    O, lse = api.attention_int8_tree(Q, cache, offsets, lens, table, parents, return_lse=True)
    kept = api.verify_drafts(model.target[words], tokens, parents, offsets, u, r, draft=model.draft[words])
    return (Q, O, lse) + kept


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps(gpu, dtype, interleaved):
    from post_int4_weight_amd import api
    model, gen = Model(dtype, gpu), torch.Generator().manual_seed(17)
    rotary = api.Rotary.make(DIM, interleaved=interleaved, scaling="yarn", factor=4.0, original_length=64, device=gpu)
    prompts = [[int(x) for x in torch.randint(0, VOCAB, (n,), generator=gen)] for n in (40, 3, 129)]
    most, batch = 200, len(prompts)
    table = _table([most] * batch, BS, batch * -(-most // BS) + 1, seed=1)
    cache = api.KVCacheInt8.empty(batch * -(-most // BS) + 1, KV, DIM, BS, device=gpu)
    tab = _ints(table, gpu)
    row = lambda tokens: torch.tensor([t % WORDS for t in tokens], device=gpu)
    flat = row([t for p in prompts for t in p])
    api.kv_cache_append_int8(cache, model.k[flat], model.v[flat], _ints(_offsets([len(p) for p in prompts]), gpu),
                             _ints([0] * batch, gpu), tab, rotary)
    done, last, touched = [list(p) for p in prompts], [5, 6, 7], 1
    total_kept = 0
    for step, nodes in enumerate(([9, 4, 20], [1, 17, 6], [12, 12, 3])):
        announce(f"draft step {step} {dtype} interleaved={interleaved}")
        trees = [[-1] + [max(p, 0) for p in t[1:]] for t in _trees(nodes, 3, step)]
        tokens, starts, off = model.propose(trees, last, gen), [len(d) for d in done], _offsets(nodes)
        depths = [s + len(ref.line(t, i)) - 1 for s, t in zip(starts, trees) for i in range(len(t))]
        u, r = torch.rand(sum(nodes), generator=gen), torch.rand(batch, generator=gen)
        args = (row(tokens), _ints(off, gpu), _ints(starts, gpu), _ints([s + n for s, n in zip(starts, nodes)], gpu),
                _ints(depths, gpu), tab, _ints([p for t in trees for p in t], gpu), _ints(tokens, gpu), u.to(gpu), r.to(gpu))
        before = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
        Q, O, lse, path, counts, token = _forward(api, model, cache, rotary, *args)
        torch.cuda.synchronize()
        # attention, on what the cache holds; the tables end in rows that belong to no sequence
        lens = [s + n for s, n in zip(starts, nodes)]
        k, v = api.kv_cache_read_int8(cache, _ints(_offsets(lens), gpu), _ints([0] * batch, gpu), tab, sum(lens),
                                      out_dtype=torch.float32)
        at = _offsets(lens)
        vals = [(to64(k[a:b]), to64(v[a:b])) for a, b in zip(at, at[1:])]
        _check(O, lse, Q, vals, trees, HEADS, KV, DIM ** -0.5, 0)
        # what is kept
        words, path, counts, token = [t % WORDS for t in tokens], path.tolist(), counts.tolist(), token.tolist()
        target, draft = to64(model.target), to64(model.draft)
        for b, t in enumerate(trees):
            a = slice(off[b], off[b + 1])
            kept, after = ref.verify(target[words[a]], draft[words[a]], tokens[a], t, u[a].double().numpy(), float(r[b]))
            assert path[a] == kept + [-1] * (nodes[b] - len(kept)) and (counts[b], token[b]) == (len(kept), after)
        # the same step from a graph, over the cache as it was
        with torch.cuda.graph(graph := torch.cuda.CUDAGraph()):
            out = _forward(api, model, cache, rotary, *args)
        now = [t.clone() for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
        for _ in range(3):
            for t, x in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), before):
                t.copy_(x)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[1], O) and out[3].tolist() == path and out[5].tolist() == token
            assert all(torch.equal(t, x) for t, x in zip((cache.k, cache.v, cache.k_scales, cache.v_scales), now))
        # the kept rows again, behind what was there
        rows = [off[b] + i for b in range(batch) for i in path[off[b]:off[b + 1]] if i >= 0]
        kept = row([tokens[i] for i in rows])
        api.kv_cache_append_int8(cache, model.k[kept], model.v[kept], _ints(_offsets(counts), gpu), _ints(starts, gpu), tab,
                                 rotary)
        touched += 5      # the eager append, three replays, and this one
        for b in range(batch):
            done[b] += [tokens[off[b] + i] for i in path[off[b]:off[b + 1]] if i >= 0]
        last = token
        total_kept += sum(counts)
        lens, at = [len(d) for d in done], _offsets([len(d) for d in done])
        k, v = api.kv_cache_read_int8(cache, _ints(at, gpu), _ints([0] * batch, gpu), tab, sum(lens), out_dtype=torch.float32)
        torch.cuda.synchronize()
        ks, vs = to64(cache.k_scales), to64(cache.v_scales)
        for b, d in enumerate(done):
            words = [t % WORDS for t in d]
            want = ref.turn(to64(model.k)[words], range(len(d)), to64(rotary.inv_freq), rotary.magnitude, interleaved)
            ids = table[b, np.arange(len(d)) // BS]
            for got, exact, scales in ((k, want, ks), (v, to64(model.v)[words], vs)):
                tol = scales[ids][:, :, None] * (0.5 * touched + 2.0 ** -10)
                assert np.all(np.abs(to64(got[at[b]:at[b + 1]]) - exact) <= tol)
    assert total_kept > 3 * batch      # drafts among them, not the roots alone
