"""Verification's sums where they are hardest to hold."""
import numpy as np
import pytest
import torch

import drafts_ref as dr
from test_gpu_kvq import BF, F32, _cu, _ints
from test_gpu_verify import _same

pytestmark = pytest.mark.gpu

# temperature, the largest logit
SCALES = [(1.0, 12.0), (1.0, 300.0), (1.0, -200.0), (0.4, 30.0), (0.05, 30.0), (0.01, 30.0), (0.001, 30.0), (1e-4, 20.0),
          (1e-6, -5.0), (30.0, 1e4), (1e-3, 1e-3), (1e3, 1e6), (2.5, 1e7), (1e-35, 2e-33)]


def _rows(t, top, vocab, seed):
    """A row of logits at temperature t (fp32): a dozen ids of some weight each, among others of next to none."""
    r = np.random.default_rng(seed)
    x = (top - t * (30.0 + 50.0 * r.random(vocab))).astype(np.float32)
    ids = np.sort(r.choice(vocab, 12, replace=False))
    x[ids] = (top - t * 4.0 * r.random(12)).astype(np.float32)
    x[ids[r.integers(12)]] = top
    x[r.choice(vocab, vocab // 8, replace=False)] = -np.inf
    x[ids[:2]] = np.float32(top)
    return x, ids


def _steps(v):
    """The two fp32 numbers beside v, in [0, 1)."""
    a = np.float32(v)
    b = np.nextafter(a, np.float32(0.0 if a > v else 1.0))
    return [float(np.clip(z, 0.0, np.float32(1 - 2.0 ** -24))) for z in (a, b)]


@pytest.mark.parametrize("t,top", SCALES)
@pytest.mark.parametrize("vocab", [64, 5000])
def test_next_tokens_beside_every_border(t, top, vocab):
    """Random numbers one fp32 step or less from the borders between ids: sums hold 36 bits at any temperature and
    wherever the logits lie."""
    from latency_moe_decode_gb300 import ops
    t = float(np.float32(t))
    xs, us = [], []
    for seed in range(4):
        x, ids = _rows(t, top, vocab, seed)
        c = np.cumsum(dr.softmax(x.astype(np.float64), t))
        for i in ids:
            for u in _steps(c[i] / c[-1]):
                xs.append(x)
                us.append(u)
    n = len(us)
    x, u, tt = torch.from_numpy(np.stack(xs)), torch.tensor(us, dtype=F32), torch.full((n,), t)
    got = ops.verify_drafts(x.cuda(), _ints([0] * n), u.cuda(), _cu([1] * n), temperature=tt.cuda(), max_tokens=1)
    _same(got, x, torch.zeros(n, dtype=torch.int32), u, [[-1]] * n, tt, None)


@pytest.mark.parametrize("t,top", SCALES)
@pytest.mark.parametrize("probs", [True, False])
def test_acceptance_beside_the_border(t, top, probs):
    """The same of acceptances: random numbers one fp32 step or less from p / q."""
    from latency_moe_decode_gb300 import ops
    t, vocab = float(np.float32(t)), 777
    xs, us, tok, qs = [], [], [], []
    r = np.random.default_rng(9)
    for seed in range(4):
        x, ids = _rows(t, top, vocab, seed)
        p = dr.softmax(x.astype(np.float64), t)
        for i in ids[p[ids] > 0]:
            q = np.float32(p * np.exp(0.3 * r.standard_normal(vocab)))
            q[i] = np.float32(min(1.0, p[i] * (1.0 + r.random())))
            for u in _steps(p[i] / float(q[i]) if probs else p[i]):
                xs += [x, x]
                us += [0.4, u]
                tok += [0, i]
                qs += [q, q]
    n = len(us) // 2
    x, u, tt = torch.from_numpy(np.stack(xs)), torch.tensor(us, dtype=F32), torch.full((n,), t)
    q = torch.from_numpy(np.stack(qs)) if probs else None
    tok = torch.tensor(tok, dtype=torch.int32)
    got = ops.verify_drafts(x.cuda(), tok.cuda(), u.cuda(), _cu([2] * n), temperature=tt.cuda(), max_tokens=2,
                            draft_probs=None if q is None else q.cuda())
    _same(got, x, tok, u, [[-1, 0]] * n, tt, q)
    assert len(set(got.count.tolist())) == 2


def test_acceptance_after_long_chains_of_additions():
    """2^24 ids, in the few parts that many rows get: 256 ids of one weight, where the parts' lanes begin, and behind them
    weights that are lost one by one when they are added in fp32 (16 of them are less than half a step of 1). The
    draft is one of the 256, its random number 2^-13 from p each way; the sums that lose the others are 2^-12 short."""
    from latency_moe_decode_gb300 import ops
    vocab, batch = 1 << 24, 1217
    row = torch.full((vocab,), -19.5, dtype=BF)
    ids = (torch.arange(8)[:, None] * (vocab // 8) + 8 * torch.arange(32)).flatten()
    row[ids] = 0.0
    w = torch.exp(row.double())
    z = w.sum().item()
    d = int(ids[100])
    assert 16 * float(w[1]) < 2.0 ** -24 and z > 256.05
    x = row.cuda().expand(2 * batch, vocab)
    up = torch.tensor([(1 + 2.0 ** -13) / z if b % 2 else (1 - 2.0 ** -13) / z for b in range(batch)])
    u = torch.stack([torch.full((batch,), 0.3), up], 1).flatten()
    tok = torch.tensor([0, d] * batch, dtype=torch.int32)
    got = ops.verify_drafts(x, tok.cuda(), u.cuda(), _cu([2] * batch), max_tokens=2)
    want = [1 if b % 2 else 2 for b in range(batch)]
    assert got.count.tolist() == want
    for b in (0, 1):
        c = torch.cumsum(w if b == 0 else torch.where(torch.arange(vocab) == d, 0.0, w), 0)
        at = int(torch.searchsorted(c, float(u[0]) * c[-1].item(), right=True))
        assert abs(c[at].item() / c[-1].item() - 0.3) > 2.0 ** -20
        assert set(got.next_tokens[b::2].tolist()) == {at}


@pytest.mark.parametrize("vocab", [900, 32000])
def test_drafts_from_all_but_the_target(vocab):
    """Draft probabilities that differ from the target's by an fp32 step or less, but for the refused draft and one
    other id (2^-9 of the sum): what is left of the other ids is 2^-24 of the sum, and whether an id has something left
    must not go by sums that are off by as much. Random numbers a tenth beside the border that they make; the id that
    comes out holds them within 2^-26 (a weight's 2^-36, over the 2^-9 that are left, and what roundings add)."""
    from latency_moe_decode_gb300 import ops
    xs, us, tok, qs, lefts = [], [], [], [], []
    for seed, step in enumerate([0.0, 2.0 ** -24, -2.0 ** -24, 2.0 ** -23, -2.0 ** -23, -2.0 ** -22] * 6):
        r = np.random.default_rng(seed)
        x = (1.5 * r.standard_normal(vocab)).astype(np.float32)
        a, d = vocab // 2 + seed, vocab // 3
        x[a] = x[d] = np.float32(np.log(np.exp(x.astype(np.float64)).sum() * 0.02))
        p = dr.softmax(x.astype(np.float64), 1.0)
        q = (p * (1 + step)).astype(np.float32)
        q[a], q[d] = np.float32(p[a] - 2.0 ** -9), np.float32(4 * p[d])
        left = np.maximum(p - q.astype(np.float64), 0)
        edge = left[:a].sum() / left.sum()
        for u0 in (0.9 * edge, 1.1 * edge):
            xs += [x, x]
            us += [u0, 0.9]
            tok += [0, d]
            qs += [q, q]
            lefts.append(left)
    n = len(us) // 2
    x, u, q = torch.from_numpy(np.stack(xs)), torch.tensor(us, dtype=F32), torch.from_numpy(np.stack(qs))
    got = ops.verify_drafts(x.cuda(), _ints(tok), u.cuda(), _cu([2] * n), max_tokens=2, draft_probs=q.cuda())
    assert got.count.tolist() == [1] * n
    far = []
    for b, i in enumerate(got.next_tokens.tolist()):
        c = np.cumsum(lefts[b]) / lefts[b].sum()
        want = float(u[2 * b])
        assert lefts[b][i] > 0
        far.append(max((c[i - 1] if i else 0.0) - want, want - c[i], 0.0))
    assert max(far) <= 2.0 ** -26, (np.log2(max(far)), far)


def test_sums_over_many_equal_weights():
    """2^24 ids of one weight that is no whole power of two: a random number half an id's share from the borders picks
    that id. (A lane's remainders, all alike, round alike: in one chain they are off by 2^-20 of the sum and more.)"""
    from latency_moe_decode_gb300 import ops
    vocab, batch = 1 << 24, 100
    at = torch.from_numpy(np.sort(np.random.default_rng(0).choice(vocab // 2, batch, replace=False)))
    for value, t in ((0.3, 1.0), (-7.7, 1.0), (0.123, 0.9)):
        row = torch.full((vocab,), value, device="cuda")
        u = ((at.double() + 0.5) / vocab).to(F32)
        assert torch.equal(u.double() * vocab, at + 0.5)
        got = ops.verify_drafts(row.expand(batch, vocab), _ints([0] * batch), u.cuda(), _cu([1] * batch), max_tokens=1,
                                temperature=torch.full((batch,), t).cuda())
        assert got.next_tokens.tolist() == at.tolist()
        # behind a refused draft, the first id, where all of the draft probability lies: the others are left
        u2 = torch.stack([u, torch.full((batch,), 0.5)], 1).flatten()
        q = torch.zeros(vocab, device="cuda")
        q[:1] = 1.0
        got = ops.verify_drafts(row.expand(2 * batch, vocab), _ints([0] * 2 * batch), u2.cuda(), _cu([2] * batch),
                                draft_probs=q.expand(2 * batch, vocab), max_tokens=2, temperature=torch.full((batch,), t).cuda())
        assert got.count.tolist() == [1] * batch
        for i, v in zip(got.next_tokens.tolist(), u.tolist()):
            want = (vocab - 1) * v  # (in ids; exact)
            if abs(want - round(want)) > 0.1:
                assert i == 1 + int(want)
