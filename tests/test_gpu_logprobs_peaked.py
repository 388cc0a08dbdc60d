"""dec_logprobs where cancellation would show: rows that one token leads, far from the row's first elements,
at offsets that logits may have, and rows whose largest logit is of any magnitude."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def _exact(x):
    x = x.double().cpu().numpy()
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    s = e.sum(-1, keepdims=True)
    lp = (x - m) - np.log(s)
    p = e / s
    with np.errstate(invalid="ignore"):
        ent = -np.where(p > 0, p * lp, 0.0).sum(-1)
    return lp, ent, (x - m), 1 - p.max(-1)


def _check(x, t, n):
    """Units of 2^-24. A term's exponential: 4 (the approximation's 2^-22) and 5.6 for its argument, within -16 .. 0
    where it counts; a power of two's 4, logarithm, its correction and product 3: 17 for all, 20 taken. Each of the
    additions, at most vocab / 512 + 32 one after another, loses no more than half a unit of the sum or, where one term
    is nearly all of it, than what is added: the rest of the row's mass. x - M and the result round once each. The entropy
    is the difference of log2 S and U / S, of magnitude 16 + log2(vocab) at most and, in a row with little else than one
    term, 16 (16 and 8 units, with the division 28); U's additions round sixteen times as much, and lose the rest's mass
    times its exponents, up to 70."""
    from latency_moe_decode_gb300 import ops
    vocab = x.shape[1]
    lp, ent, below, rest = _exact(x)
    r = ops.logprobs(x, torch.from_numpy(t).cuda(), top_n=n)
    rows, chain = np.arange(len(x)), (vocab / 512 + 32) * U
    lost = np.minimum(rest, chain)
    got, want = r.logprob.double().cpu().numpy(), lp[rows, t]
    assert (got <= 0).all()
    assert (np.abs(got - want) <= 20 * U + lost + U * (np.abs(below[rows, t]) + np.abs(want))).all(), np.abs(got - want).max()
    h = r.entropy.double().cpu().numpy()
    assert (h >= 0).all()
    off = (40 + 4 * np.log2(vocab) * np.minimum(1, 100 * rest) + 2 * ent) * U + np.minimum(70 * rest, 17 * chain)
    assert (np.abs(h - ent) <= off).all(), np.abs(h - ent).max()
    if n:
        ids = np.argsort(-x.double().cpu().numpy(), axis=-1, kind="stable")[:, :n]
        assert np.array_equal(r.top_ids.cpu().numpy(), ids)
        got, want, b = r.top_logprobs.double().cpu().numpy(), np.take_along_axis(lp, ids, 1), np.take_along_axis(below, ids, 1)
        assert (got <= 0).all() and (np.diff(got, axis=1) <= 0).all()
        assert (np.abs(got - want) <= 20 * U + lost[:, None] + U * (np.abs(b) + np.abs(want))).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab,n", [(5000, 0), (32000, 20), (32001, 0), (128256, 5), (280000, 32)])
@pytest.mark.parametrize("offset", [0, 300, -300, 3000, -3000, 8185, -8150, 9000, -9000, 1e5, -1e6])
def test_rows_that_one_token_leads(offset, vocab, n, dtype):
    rows = 24
    g = torch.Generator().manual_seed(vocab)
    x = 3 * torch.randn(rows, vocab, generator=g)
    at = torch.randint(vocab // 3, vocab, (rows,), generator=g)
    at[0], at[1], at[2] = vocab - 1, 0, vocab // 2
    x[torch.arange(rows), at] = torch.linspace(8, 55, rows)
    x = (x + offset).to(dtype).cuda()
    t = at.to(torch.int32).numpy()
    t[-4:] = [5, vocab // 2 + 1, vocab - 2, 17]  # tokens that trail far behind
    _check(x, t, n)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab,n", [(777, 3), (33000, 0), (70000, 20)])
def test_rows_of_any_magnitude(vocab, n, dtype):
    """Maxima on both sides of where another pass takes over, rows around it, the type's ends, equal logits."""
    g = torch.Generator().manual_seed(3)
    big = torch.finfo(dtype).max
    noise = torch.randn(vocab, generator=g)
    rows = [noise + c for c in (8150.0, -8195.0, -8300.0, -8448.0, -8500.0)]
    for m in (8192.0, 8191.5, -8192.0, -8191.5, -8448.0, -8449.0):
        rows += [torch.full((vocab,), m), torch.where(torch.arange(vocab) % 3 == 0, m, m - 7.0)]
    rows += [torch.full((vocab,), -big), torch.full((vocab,), big), torch.where(torch.arange(vocab) == vocab - 2, big, -big),
             torch.where(torch.arange(vocab) < 5, 0.0, -big), torch.where(torch.arange(vocab) == 9, -8000.0, -8460.0),
             noise * 1e30, noise * 1e-30]
    x = torch.stack(rows).to(dtype).cuda()
    t = torch.randint(0, vocab, (len(rows),), generator=g).to(torch.int32).numpy()
    t[-4] = 3
    lp = _exact(x)[0]
    t = np.where(lp[np.arange(len(t)), t] < -3.4e38, x.argmax(-1).cpu().numpy(), t).astype(np.int32)  # (beyond fp32's range)
    _check(x, t, min(n, 1))


@pytest.mark.parametrize("value", [0.0, 9000.0])
def test_the_longest_rows(value):
    """2^31 - 1025 equal logits: a second look at the whole row for its alternatives, another for its sums where they lie
    far from 0."""
    from latency_moe_decode_gb300 import ops
    vocab = 2 ** 31 - 1025
    x = torch.full((1, vocab), value, dtype=BF, device="cuda")
    x[0, 5] = -torch.inf
    r = ops.logprobs(x, torch.tensor([vocab - 1], dtype=torch.int32, device="cuda"), top_n=1)
    want = -np.log(vocab - 1)
    # every sum is of ones or of one power of two, exact up to 2^24 of them: a thread has 2^20 to 2^23
    assert abs(r.logprob.item() - want) <= 40 * U * -want and abs(r.top_logprobs.item() - want) <= 40 * U * -want
    assert abs(r.entropy.item() + want) <= 80 * U * -want
    assert r.rank.item() == vocab - 2 and r.top_ids.item() == 0
