"""The engine's steps over 4-bit caches with several rows a sequence: chains and trees of drafts against single steps
along each row's path, and speculative decoding (step, verification, commit) against plain greedy decoding."""
import numpy as np
import pytest
import torch

import drafts_ref as dr
from latency_moe_decode_gb300 import synth
from tests.parity import LOGIT_MAX_ABS
from tests.test_gpu_step_kvq import DENSE, _ints, _setup, _step, _tables

pytestmark = pytest.mark.gpu


def _rows(eng, caches, lens, table, toks, cu, parents=None, **kw):
    c = eng.cfg
    n = len(toks)
    logits = torch.empty(n, c.vocab, device="cuda")
    nxt = torch.empty(n, dtype=torch.int32, device="cuda")
    eng.step_kvq(caches, _ints(lens), table, tokens=_ints(toks), logits=logits, next_tokens=nxt, cu_tokens=_ints(cu),
                 parents=None if parents is None else _ints(parents), **kw)
    eng.sync()
    caches[0].check()
    return logits, nxt


def _roomy(seed, page=16):
    """The engine's histories in tables with room for 24 more positions each."""
    _, eng, caches, table, lens, _ = _setup(DENSE, 5, seed, page)
    wide, n_pages = _tables([l + 24 for l in lens], page, 3, seed + 1)
    big = eng.kvq_caches(n_pages, page)
    for b in range(5):
        eng.kvq_store(b, big, wide[b].contiguous())
    return eng, big, wide, lens


@pytest.mark.parametrize("sizes", [[4, 1, 6, 3, 8], [2, 0, 13, 1, 5]])
@pytest.mark.parametrize("tree", [True, False])
def test_rows_match_single_steps_along_their_paths(sizes, tree):
    eng, caches, table, lens = _roomy(3)
    g = np.random.default_rng(sum(sizes))
    parents = [dr.random_parents(g, n, 3 if tree else 1) if n else [] for n in sizes]
    toks = synth.gen_tokens(sum(sizes), DENSE.vocab, seed=17).tolist()
    cu = np.cumsum([0] + sizes).tolist()
    before = [k.pages.clone() for k in caches]
    logits, nxt = _rows(eng, caches, lens, table, toks, cu, [p for ps in parents for p in ps] if tree else None, max_tokens=max(sizes))
    again, _ = _rows(eng, caches, lens, table, toks, cu, [p for ps in parents for p in ps] if tree else None)
    assert (again - logits).abs().max().item() <= 2 * LOGIT_MAX_ABS  # (a bound of 22 rows may choose another kernel)
    rows = logits.double().cpu().numpy()
    assert np.array_equal(nxt.cpu().numpy(), rows.argmax(1))
    for b, ps in enumerate(parents):
        done = {}
        for j, path in enumerate(dr.paths(ps)):
            for i, r in enumerate(path):  # single steps from the root (those already made are not repeated)
                if tuple(path[:i + 1]) in done:
                    continue
                if i == 0 or tuple(path[:i]) != done.get("last"):
                    for k, p in zip(caches, before):
                        k.pages.copy_(p)
                    for i2, r2 in enumerate(path[:i]):
                        _step(eng, caches, [lens[b] + i2], table[b:b + 1], [toks[cu[b] + r2]])
                lg, _, _ = _step(eng, caches, [lens[b] + i], table[b:b + 1], [toks[cu[b] + r]])
                done[tuple(path[:i + 1])] = lg[0]
                done["last"] = tuple(path[:i + 1])
            # (each side is within LOGIT_MAX_ABS of the restatement of its own cache, and a code of the row's
            # history that rounds the other way moves logits by less)
            assert np.abs(rows[cu[b] + j] - done[tuple(path)]).max() <= 2 * LOGIT_MAX_ABS, (b, j)


def test_speculative_decoding_gives_the_greedy_text():
    """Trees whose drafts are partly the text that single steps generate: steps of trees, verification and commits give
    that text. A token that differs has to be a near tie of its own step's logits."""
    from latency_moe_decode_gb300 import ops
    eng, caches, table, lens = _roomy(5)
    batch, steps = 3, 9
    lens, table = lens[1:1 + batch], table[1:1 + batch].contiguous()
    first = synth.gen_tokens(batch, DENSE.vocab, seed=40).tolist()
    start = [k.pages.clone() for k in caches]
    text, t, ln = [[x] for x in first], list(first), list(lens)
    for _ in range(steps):
        lg, nx, _ = _step(eng, caches, ln, table, t)
        t, ln = nx.tolist(), [l + 1 for l in ln]
        for b in range(batch):
            text[b].append(t[b])
    for k, p in zip(caches, start):
        k.pages.copy_(p)
    length, cur, out = _ints(lens), list(first), [[x] for x in first]
    g = np.random.default_rng(1)
    calls = 0
    while min(len(o) for o in out) <= steps - 4 and calls < 20:
        calls += 1
        toks, parents, cu = [], [], [0]
        for b in range(batch):
            ahead = text[b][len(out[b]):len(out[b]) + 2]
            wrong = g.integers(0, DENSE.vocab, 3).tolist()
            # root; a wrong draft and the right one beside each other; below the right one a wrong and a right one
            toks += [cur[b], wrong[0], ahead[0], wrong[1], ahead[1], wrong[2]]
            parents += [-1, 0, 0, 2, 2, 1]
            cu.append(len(toks))
        logits, _ = _rows(eng, caches, length.tolist(), table, toks, cu, parents, max_tokens=6)
        got = ops.verify_drafts(logits, _ints(toks), torch.rand(len(toks), device="cuda"), _ints(cu), parents=_ints(parents),
                                temperature=torch.zeros(batch, device="cuda"), max_tokens=6)
        for cache in caches:
            cache.move(got.path, got.count, table, start=length)
        length = length + got.count
        for b in range(batch):
            path = got.path[b, :int(got.count[b])].tolist()
            new = [toks[cu[b] + r] for r in path[1:]] + [int(got.next_tokens[b])]
            for r, x in zip(path, new):
                want = text[b][len(out[b])]
                row = logits[cu[b] + r]
                assert x == int(row.argmax())
                if x != want:  # greedy texts part at a near tie
                    assert (row[x] - row[want]).item() <= 4 * LOGIT_MAX_ABS
                    pytest.skip("a near tie parted the texts")
                out[b].append(x)
            cur[b] = out[b][-1]
    for b in range(batch):
        assert out[b] == text[b][:len(out[b])] and len(out[b]) > steps - 4
    assert calls < steps - 3  # (most calls gave three tokens)
    caches[0].check()


def test_refusals_and_padded_rows():
    from latency_moe_decode_gb300.capi import DecError
    eng, caches, table, lens = _roomy(7)
    tok = synth.gen_tokens(8, DENSE.vocab, seed=2).tolist()
    cu = [0, 2, 3, 3, 5, 8]
    logits, _ = _rows(eng, caches, lens, table, tok, cu, [-1, 0, -1, -1, 0, -1, 0, 0])
    # rows of no sequence around them change nothing for the others, and are finite
    pad = [3, 4] + tok + [5]
    lg2, _ = _rows(eng, caches, lens, table, pad, [c + 2 for c in cu], [7, 7, -1, 0, -1, -1, 0, -1, 0, 0, 9])
    assert torch.isfinite(lg2).all()
    assert (lg2[2:10] - logits).abs().max().item() <= 2 * LOGIT_MAX_ABS
    for bad in (lambda: eng.step_kvq(caches, _ints(lens), table, tokens=_ints(tok[:5]), parents=_ints([-1] * 5)),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=_ints(tok), cu_tokens=_ints(cu[:4])),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=_ints(tok), cu_tokens=_ints(cu), parents=_ints([0] * 7)),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=_ints(tok), cu_tokens=_ints(cu), max_tokens=0),
                lambda: eng.step_kvq(caches, _ints(lens), table, cu_tokens=_ints(cu)),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=_ints(tok * 4), cu_tokens=_ints(cu))):
        with pytest.raises((DecError, ValueError)):
            bad()
    eng.sync()


def test_captured_verify_steps():
    """A whole round (step of a tree, verification, commit of every layer, new lengths) captured once and replayed."""
    from latency_moe_decode_gb300 import ops
    eng, caches, table, lens = _roomy(9)
    cu, parents = _ints([0, 4, 8, 12, 16, 20]), _ints([-1, 0, 0, 2] * 5)
    tok = synth.gen_tokens(20, DENSE.vocab, seed=3).to(torch.int32).cuda()
    u = torch.rand(20, device="cuda")
    length = _ints(lens)
    logits = torch.empty(20, DENSE.vocab, device="cuda")

    def round_(s):
        eng.step_kvq(caches, length, table, tokens=tok, logits=logits, cu_tokens=cu, parents=parents, max_tokens=4, stream=s)
        got = ops.verify_drafts(logits, tok, u, cu, parents=parents, max_tokens=4)
        for cache in caches:
            cache.move(got.path, got.count, table, start=length)
        length.add_(got.count)
        return got

    start = [k.pages.clone() for k in caches]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        a = [round_(s), round_(s)]
        want_len, want_logits = length.clone(), logits.clone()
    torch.cuda.synchronize()
    want_pages = [k.pages.clone() for k in caches]
    for k, p in zip(caches, start):
        k.pages.copy_(p)
    length.copy_(_ints(lens))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = round_(s)
    for i in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, a[i]))
    assert torch.equal(length, want_len) and torch.equal(logits, want_logits)
    assert all(torch.equal(k.pages, p) for k, p in zip(caches, want_pages))
    eng.sync()
    caches[0].check()
