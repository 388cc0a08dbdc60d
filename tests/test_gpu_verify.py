"""Verification of drafted tokens on the GPU (verify_drafts) against a walk in 64 bits."""
import numpy as np
import pytest
import torch

import drafts_ref as dr
from test_gpu_kvq import BF, F32, _cu, _ints

pytestmark = pytest.mark.gpu


def _case(sizes, vocab, dtype, probs, width, seed, temps=None, peaked=8.0):
    g, r = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    n = sum(sizes)
    x = 2.0 * torch.randn(n, vocab, generator=g)
    x.scatter_add_(1, torch.randint(0, vocab, (n, 2), generator=g), torch.full((n, 2), peaked))
    x = x.to(dtype)
    parents = [dr.random_parents(r, m, width) if m else [] for m in sizes]
    t = torch.ones(len(sizes)) if temps is None else torch.tensor([temps[b % len(temps)] for b in range(len(sizes))])
    per = torch.repeat_interleave(t, torch.tensor(sizes))[:, None]
    draft = (x.float() + 0.7 * torch.randn(n, vocab, generator=g)) / torch.where((per > 0) & (per < 100), per, torch.ones_like(per))
    q = torch.softmax(draft, 1)
    first = np.repeat(np.cumsum([0] + sizes[:-1]), sizes)
    flat = np.array([p for ps in parents for p in ps], np.int64)
    up = torch.from_numpy(np.maximum(first + flat, 0))
    tokens = torch.multinomial(q[up], 1, generator=g)[:, 0].to(torch.int32) if n else torch.zeros(0, dtype=torch.int32)
    u = torch.rand(n, generator=g)
    return x, tokens, u, parents, t, q if probs else None


def _same(got, x, tokens, u, parents, t, q, near=2.0 ** -33):
    """Every sequence's path, count and next token; where a decision of the 64-bit walk lies within `near` of the
    other one the kernel's may be either. Sums of pairs of floats are held to about 36 bits (a weight's terms round to
    2^-38, a whole sum's low parts to 2^-24 of themselves); the walk's own roundings are far smaller."""
    path, count, nxt = (z.cpu().numpy() for z in got)
    row = skipped = 0
    for b, ps in enumerate(parents):
        n = len(ps)
        if n == 0:
            assert count[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
            continue
        want, token, off = dr.verify(x[row:row + n].double().numpy(), tokens[row:row + n].tolist(), u[row:row + n].tolist(), ps,
                                     float(t[b]), None if q is None else q[row:row + n].numpy())
        row += n
        if off < near:
            skipped += 1
            continue
        assert path[b, :count[b]].tolist() == want, b
        assert (path[b, count[b]:] == -1).all() and nxt[b] == token, (b, nxt[b], token, off)
    assert skipped <= 1 + len(parents) // 20


CASES = [
    # rows, vocabulary, type, draft probabilities, width
    ([8], 32000, F32, True, 1),
    ([1], 32000, F32, False, 1),
    ([64], 32000, BF, False, 8),
    ([5, 8, 1, 3] * 10, 1001, F32, True, 1),
    ([30, 1, 0, 17] * 5, 1000, BF, True, 5),
    ([9, 64, 2] * 20, 257, F32, False, 6),
    ([4, 4], 1, F32, True, 2),
    ([6] * 30, 2, BF, True, 3),
    ([12] * 12, 33, F32, True, 4),
    ([3, 7], 128001, F32, True, 2),
    ([7] * 80, 5000, BF, False, 2),
    ([1024, 3], 300, F32, True, 40),
]


@pytest.mark.parametrize("sizes,vocab,dtype,probs,width", CASES)
def test_verify(sizes, vocab, dtype, probs, width):
    from latency_moe_decode_gb300 import ops
    for seed in (0, 1):
        temps = [1.0, 0.0, 0.4, 2.5, float("inf"), 1e-6] if seed else None
        x, tok, u, parents, t, q = _case(sizes, vocab, dtype, probs, width, seed, temps)
        flat = _ints([p for ps in parents for p in ps])
        pad = torch.randn(x.shape[0], vocab + 3).to(dtype).cuda()  # rows that are not aligned
        pad[:, 1:vocab + 1] = x.cuda()
        args = dict(parents=flat if width > 1 else None, temperature=t.cuda() if seed else None,
                    draft_probs=None if q is None else q.cuda())
        got = ops.verify_drafts(x.cuda(), tok.cuda(), u.cuda(), _cu(sizes), max_tokens=max(sizes), **args)
        _same(got, x, tok, u, parents, t, q)
        again = ops.verify_drafts(pad[:, 1:vocab + 1], tok.cuda(), u.cuda(), _cu(sizes), **args)
        assert torch.equal(again.count, got.count) and torch.equal(again.next_tokens, got.next_tokens)
        assert torch.equal(again.path[:, :max(sizes)], got.path) and (again.path[:, max(sizes):] == -1).all()


@pytest.mark.parametrize("vocab", [50, 32000])
@pytest.mark.parametrize("probs", [True, False])
def test_acceptance_at_the_border(vocab, probs):
    """Random numbers beside p / q, one fp32 step (2^-24 of it and more) each way: what fp32 sums leave open is decided
    as 64 bits say."""
    from latency_moe_decode_gb300 import ops
    batch = 40
    x, tok, u, parents, t, q = _case([3] * batch, vocab, F32, probs, 1 if probs else 2, 5, peaked=3.0)
    parents = [[-1, 0, 1 if probs else 0]] * batch
    for b in range(batch):
        p = dr.softmax(x[3 * b].double().numpy(), 1.0)
        d = int(tok[3 * b + 1])
        qd = float(q[3 * b, d]) if probs else 1.0
        edge = np.float32(min(p[d] / qd, 1 - 2.0 ** -24))
        for _ in range(b % 4):
            edge = np.nextafter(edge, np.float32(b % 2))
        u[3 * b + 1] = float(edge)
    got = ops.verify_drafts(x.cuda(), tok.cuda(), u.cuda(), _cu([3] * batch), parents=_ints([p for ps in parents for p in ps]),
                            draft_probs=None if q is None else q.cuda(), max_tokens=3)
    _same(got, x, tok, u, parents, t, q)
    assert len(set(got.count.tolist())) > 1


@pytest.mark.parametrize("vocab", [7, 1000, 32000])
def test_next_tokens_at_borders(vocab):
    """Logits of which the weights are whole powers of two: the sums are exact, and random numbers that fall on one
    belong to the next id. 0 gives the first id that has a probability, the largest one below 1 the last."""
    from latency_moe_decode_gb300 import ops
    log2 = float(np.log(2.0))
    w = np.zeros(vocab)
    ids = np.linspace(1, vocab - 2, 5).astype(int)  # (the first and the last id have no probability)
    x = torch.full((6, vocab), -float("inf"))
    x[:, ids] = 0.0
    w[ids] = 0.2
    u = torch.tensor([0.0, 0.25, 0.5, 0.5, 0.75, 1 - 2.0 ** -24])
    x4 = x.clone()
    x4[:, ids[4]] = -float("inf")  # four of a quarter each: borders at 0.25, 0.5, 0.75
    got = ops.verify_drafts(x4.cuda(), _ints([0] * 6), u.cuda(), _cu([1] * 6), max_tokens=1)
    assert got.next_tokens.tolist() == [ids[0], ids[1], ids[2], ids[2], ids[3], ids[3]]
    got = ops.verify_drafts(x.cuda(), _ints([0] * 6), u.cuda(), _cu([1] * 6), max_tokens=1)
    assert got.next_tokens.tolist() == [ids[0], ids[1], ids[2], ids[2], ids[3], ids[4]]
    assert log2 > 0 and w.sum() > 0.99


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab", [3, 17, 1000, 32003])
def test_greedy_ties_wherever_a_row_begins(dtype, vocab):
    """The first of equal logits, at every offset of a row from 16 bytes: ties with the row's first and last ids, which
    lie in words that it shares."""
    from latency_moe_decode_gb300 import ops
    for off in range(1, 9):
        pad = torch.zeros(4, vocab + 16, dtype=dtype, device="cuda")
        x = pad[:, off:off + vocab]
        x[1, 0], x[1, vocab // 2] = -1.0, 2.0
        x[1, vocab - 1] = 2.0
        x[2, vocab - 1] = 1.0
        x[3, :vocab - 1] = -5.0
        got = ops.verify_drafts(x, _ints([0] * 4), torch.zeros(4, device="cuda"), _cu([1] * 4), max_tokens=1,
                                temperature=torch.zeros(4, device="cuda"))
        assert got.next_tokens.tolist() == [0, vocab // 2, vocab - 1, vocab - 1], off


@pytest.mark.parametrize("probs", [True, False])
def test_tokens_are_distributed_as_the_targets(probs):
    """The property that verification is for: over many sequences the first token that comes out (an accepted draft or
    the next token) follows the target's distribution, whatever drafted it. 40000 sequences; a frequency's standard
    deviation is sqrt(p (1 - p) / 40000) at most 0.0025, and 5.5 of them are met by all 24 ids but once in a million."""
    from latency_moe_decode_gb300 import ops
    g = torch.Generator().manual_seed(11)
    batch, vocab, kids = 40000, 24, 3
    x0 = torch.randn(vocab, generator=g)
    q0 = torch.softmax(x0 + torch.randn(vocab, generator=g), 0)
    x = torch.randn(batch * (kids + 1), vocab, generator=g)
    x[::kids + 1] = x0
    if probs:
        drafts = torch.multinomial(q0.expand(batch, -1), kids, replacement=True, generator=g)
    else:
        drafts = torch.tensor([3, 9, 3]).expand(batch, -1)
    tok = torch.cat([torch.zeros(batch, 1, dtype=torch.int64), drafts], 1).flatten().to(torch.int32)
    cu = torch.arange(batch + 1, dtype=torch.int32) * (kids + 1)
    got = ops.verify_drafts(x.cuda(), tok.cuda(), torch.rand(batch * (kids + 1), generator=g).cuda(), cu.cuda(),
                            parents=_ints([-1, 0, 0, 0] * batch), max_tokens=kids + 1,
                            draft_probs=q0.expand(batch * (kids + 1), -1).contiguous().cuda() if probs else None)
    count, path, nxt = (z.cpu().long() for z in (got.count, got.path, got.next_tokens))
    first = torch.where(count > 1, tok.view(batch, -1).long().gather(1, path[:, 1:2].clamp(min=0))[:, 0], nxt)
    p = torch.softmax(x0.double(), 0)
    freq = torch.bincount(first, minlength=vocab).double() / batch
    assert ((freq - p).abs() <= 5.5 * (p * (1 - p) / batch).sqrt()).all()
    # drafts that are certain are accepted as often as the target has them (3 again: never)
    rate, want = (count > 1).double().mean().item(), (p[3] + p[9]).item()
    assert 0.2 < rate < 1 if probs else abs(rate - want) <= 5.5 * (want * (1 - want) / batch) ** 0.5


def test_masked_rows_ties_and_rows_without_a_distribution():
    from latency_moe_decode_gb300 import ops
    vocab, inf, nan = 4099, float("inf"), float("nan")
    g = torch.Generator().manual_seed(2)
    x = torch.randn(12, vocab, generator=g)
    x[0, ::2] = -inf                      # a masked half
    x[1] = -inf                           # nothing left
    x[2, 77] = nan
    x[3, 78] = inf
    x[4] = torch.finfo(F32).min           # the type's lowest value, and one id above it
    x[4, 1234] = 0.0
    x[5] = torch.finfo(F32).min           # nothing but it: every id alike
    x[6, 10], x[6, 4000] = 50.0, 50.0     # a tie of two
    u = torch.rand(12, generator=g)
    t = torch.ones(12)
    t[6] = 0.0
    # each a sequence of one row; then as parents of a draft
    got = ops.verify_drafts(x.cuda(), _ints([0] * 12), u.cuda(), _cu([1] * 12), temperature=t.cuda(), max_tokens=1)
    _same(got, x, torch.zeros(12, dtype=torch.int32), u, [[-1]] * 12, t, None)
    assert got.next_tokens[1:4].tolist() == [-1] * 3 and got.next_tokens[4] == 1234 and got.next_tokens[6] == 10
    tok = torch.tensor([0, 1, 0, 77, 0, 78, 0, 1234, 0, 4000, 0, 5], dtype=torch.int32)
    order = [0, 7, 1, 8, 2, 9, 4, 10, 6, 11, 5, 7]
    y, ps = x[order].contiguous(), [[-1, 0]] * 6
    t2 = torch.tensor([1.0, 1, 1, 1, 0, 1])
    q = torch.softmax(torch.randn(12, vocab, generator=g), 1)
    for probs in (None, q):
        got = ops.verify_drafts(y.cuda(), tok.cuda(), u.cuda(), _cu([2] * 6), temperature=t2.cuda(), max_tokens=2,
                                draft_probs=None if probs is None else probs.cuda())
        _same(got, y, tok, u, ps, t2, probs)
        # (nothing left, a NaN: no draft is accepted and no token follows; 4000 only ties with 10)
        assert got.count[1:3].tolist() == [1, 1] and got.next_tokens[1:3].tolist() == [-1, -1]
        assert got.count[3] == 2 and got.count[4] == 1 and got.next_tokens[4] == 10


def test_odd_drafts_and_bounds():
    """Tokens outside the vocabulary, parents that are none, the same draft twice, rows beyond max_tokens, sequences
    without rows, rows of no sequence; a draft model that is the target."""
    from latency_moe_decode_gb300 import ops
    vocab = 500
    x, tok, u, _, t, q = _case([10, 10, 10, 10], vocab, F32, True, 3, 21, peaked=2.0)
    parents = [[-1, 0, 0, 0, 1, 2, 3, 4, 4, 9], [5, 0, 0, 0, 0, 0, 0, 0, 0, 0], [-1] + [8] * 8 + [0], [-1, 0, 1, 2, 3, 4, 5, 6, 7, 8]]
    tok[1], tok[2], tok[11:20], tok[31] = -4, vocab, 17, 2 ** 31 - 1
    flat = _ints([p for ps in parents for p in ps])
    for probs in (None, q):
        dp = None if probs is None else probs.cuda()
        for most in (10, 4, 1):
            got = ops.verify_drafts(x.cuda(), tok.cuda(), u.cuda(), _cu([10] * 4), parents=flat, draft_probs=dp, max_tokens=most)
            cut = [ps[:most] for ps in parents]
            pick = [10 * b + j for b in range(4) for j in range(most)]
            _same(got, x[pick], tok[pick], u[pick], cut, t, None if probs is None else probs[pick])
        # rows 10 .. 29 in two sequences between empty ones, others' rows around them
        cu = _ints([10, 10, 20, 20, 30, 30])
        got = ops.verify_drafts(x.cuda(), tok.cuda(), u.cuda(), cu, parents=flat, draft_probs=dp, max_tokens=10)
        pick = list(range(10, 30))
        _same(got, x[pick], tok[pick], u[pick], [[], parents[1], [], parents[2], []], torch.ones(5), None if probs is None else probs[pick])
    # the target's own probabilities: u p < p, every draft of the chain is accepted
    p = torch.softmax(x.double(), 1).float()
    chain = torch.multinomial(p, 1)[:, 0].to(torch.int32)
    tok2 = torch.cat([torch.zeros(1, dtype=torch.int32), chain[:-1]])
    got = ops.verify_drafts(x.cuda(), tok2.cuda(), (u * 0.999).cuda(), _cu([40]), draft_probs=p.cuda(), max_tokens=40)
    assert got.count.tolist() == [40]
    # no rows at all
    got = ops.verify_drafts(x[:0].cuda(), tok[:0].cuda(), u[:0].cuda(), _ints([0, 0, 0]))
    assert got.count.tolist() == [0, 0] and got.next_tokens.tolist() == [-1, -1] and got.path.shape == (2, 0)


def test_streams_graphs_and_repeats():
    from latency_moe_decode_gb300 import ops
    sizes = [8] * 20
    x, tok, u, parents, t, q = (z.cuda() if torch.is_tensor(z) else z for z in _case(sizes, 9000, F32, True, 1, 3))
    cu = _cu(sizes)
    want = ops.verify_drafts(x, tok, u, cu, draft_probs=q, max_tokens=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ops.verify_drafts(x, tok, u, cu, draft_probs=q, max_tokens=8, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ops.verify_drafts(x, tok, u, cu, draft_probs=q, max_tokens=8)
        more = ops.verify_drafts(x, tok, u, cu, max_tokens=8)
    u2 = torch.rand(u.shape, device="cuda")
    u.copy_(u2)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ops.verify_drafts(x, tok, u, cu, draft_probs=q, max_tokens=8), got))
    assert all(torch.equal(a, b) for a, b in zip(ops.verify_drafts(x, tok, u, cu, max_tokens=8), more))
