"""dec_logprobs against a plain 64-bit form."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _ref(x, t, n):
    x = x.double().cpu().numpy()
    bad = ~(x < np.inf).all(-1)  # a NaN or +infinity
    key = np.where(np.isnan(x), -np.inf, x)
    order = np.argsort(-key, axis=-1, kind="stable")
    m = np.where(np.isfinite(key.max(-1)), key.max(-1), 0)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = m + np.log(np.exp(key - m[:, None]).sum(-1))
        lp = np.where(key == -np.inf, -np.inf, key - lse[:, None])
        p = np.exp(lp)
        ent = -np.where(p > 0, p * lp, 0).sum(-1)
    lp[bad], ent[bad] = np.nan, np.nan
    r = np.arange(len(x))
    tt = np.clip(t, 0, x.shape[1] - 1)
    inside = (t >= 0) & (t < x.shape[1])
    mine = np.where(inside, lp[r, tt], np.nan)
    rank = np.where(inside, np.argmax(order == tt[:, None], axis=1), -1)
    ids = order[:, :n]
    return mine, rank, ent, ids, np.take_along_axis(lp, ids, 1), lse


def _close(got, want, tol):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fin = np.isfinite(want)
    assert (np.abs(got[fin] - want[fin]) <= np.broadcast_to(tol, want.shape)[fin]).all()


def _check(x, t, n, r=None):
    from latency_moe_decode_gb300 import ops
    if r is None:
        r = ops.logprobs(x, None if t is None else torch.from_numpy(t).cuda(), top_n=n)
    tt = np.zeros(len(x), np.int32) if t is None else t
    mine, rank, ent, ids, tops, lse = _ref(x, tt, n)
    # sums of up to `vocab` fp32 terms by chains of at most a few hundred, exponentials of arguments
    # rounded to fp32: 2^-24 of the row's spread each
    xf = x.double().cpu().numpy()
    spread = np.array([np.ptp(v[np.isfinite(v)]) if np.isfinite(v).any() else 0.0 for v in xf])
    lse = np.where(np.isfinite(lse), lse, 0)
    tol = 2.0 ** -24 * (16 + 4 * spread + 4 * np.abs(lse) + np.sqrt(x.shape[1]))
    if t is not None:
        _close(r.logprob, mine, tol)
        assert np.array_equal(r.rank.cpu().numpy(), rank)
    else:
        assert r.logprob is None and r.rank is None
    _close(r.entropy, ent, tol * (2 + spread))
    if n:
        assert np.array_equal(r.top_ids.cpu().numpy(), ids)
        _close(r.top_logprobs, tops, tol[:, None])
    return r


def _targets(g, rows, vocab):
    return torch.randint(0, vocab, (rows,), generator=g).to(torch.int32).numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,n", [(1, 1, 1), (1, 2, 2), (3, 31, 31), (2, 1000, 32), (1, 32000, 5), (7, 1023, 0),
                                          (5, 4097, 20), (64, 32000, 20), (3, 128256, 8), (300, 257, 3), (2, 200001, 32), (1, 300007, 20)])
def test_logprobs(rows, vocab, n, dtype):
    g = torch.Generator().manual_seed(rows + vocab)
    x = (3 * torch.randn(rows, vocab, generator=g)).to(dtype).cuda()
    _check(x, _targets(g, rows, vocab), n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [50, 5000, 70000, 280000])
def test_ties_masks_and_orders(vocab, dtype):
    """Equal logits, ascending and descending rows, masked rows, rows of nothing, NaN and infinities."""
    g = torch.Generator().manual_seed(vocab)
    n = 20
    x = torch.zeros(12, vocab)
    x[1] = torch.arange(vocab) * 0.01
    x[2] = -torch.arange(vocab) * 0.01
    x[3] = torch.randint(0, 3, (vocab,), generator=g).float()
    x[4] = float("-inf")
    x[5] = float("-inf")
    x[5, vocab - 1] = 2.0
    x[6] = torch.where(torch.rand(vocab, generator=g) < 0.9, -torch.inf, torch.randn(vocab, generator=g))
    x[7, vocab // 2] = float("nan")
    x[8, 3] = float("inf")
    x[9] = torch.finfo(dtype).min
    x[10] = torch.where(torch.arange(vocab) % 7 == 0, torch.finfo(dtype).min, 1.0)
    x[11] = torch.randn(vocab, generator=g) * 1e4
    x = x.to(dtype).cuda()
    t = _targets(g, 12, vocab)
    t[0], t[5], t[9] = vocab - 1, vocab - 1, 0
    _check(x, t, n)
    t[:] = -1
    t[1], t[2] = vocab, 2 ** 31 - 1
    _check(x, t, n)
    _check(x, None, 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_rows(dtype):
    g = torch.Generator().manual_seed(9)
    big = torch.randn(6, 3001, generator=g).to(dtype).cuda()
    t = _targets(g, 6, 2999)
    for x in (big[:, 1:3000], big[:, :2999], big[::2, 2:], big[:, ::3][:, :900]):
        _check(x, np.minimum(t, x.shape[1] - 1)[:len(x)], 7)


def test_rows_beyond_32_bit_offsets():
    from latency_moe_decode_gb300 import ops
    g = torch.Generator().manual_seed(5)
    rows, vocab = 70000, 32001  # 2.2 thousand million elements
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    x[-3:] = (3 * torch.randn(3, vocab, generator=g)).to(torch.bfloat16).cuda()
    t = torch.full((rows,), 7, dtype=torch.int32, device="cuda")
    r = ops.logprobs(x, t, top_n=4)
    # (against the 64-bit form: a copy of the rows elsewhere is summed in another order, since a thread's
    # vectors are the row's aligned ones)
    _check(x[-3:], t[-3:].cpu().numpy(), 4, ops.LogProbs(*(a[-3:] for a in r)))
    assert (r.rank[:-3] == 7).all() and (r.top_ids[:-3] == torch.arange(4, device="cuda")).all()
    assert (r.logprob[:-3] + np.log(vocab)).abs().max().item() < 2.0 ** -24 * (16 + np.log(vocab) * 4 + np.sqrt(vocab))


def test_captured_and_on_two_streams():
    from latency_moe_decode_gb300 import ops
    x = torch.randn(4, 50000, device="cuda")
    t = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device="cuda")
    want = ops.logprobs(x, t, top_n=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = ops.logprobs(x, t, top_n=9)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    runs = []
    for _ in range(10):
        runs.append(ops.logprobs(x, t, top_n=9, stream=s))
        runs.append(ops.logprobs(x, t, top_n=9))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in runs for a, b in zip(r, want))


def test_refusals():
    from latency_moe_decode_gb300 import ops
    from latency_moe_decode_gb300.capi import DecError
    x = torch.zeros(2, 40, device="cuda")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (lambda: ops.logprobs(x.half()), lambda: ops.logprobs(x[0]), lambda: ops.logprobs(x.cpu()),
                lambda: ops.logprobs(x, t.long()), lambda: ops.logprobs(x, t[:1]), lambda: ops.logprobs(x, t.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.logprobs(x, t, top_n=41), lambda: ops.logprobs(torch.zeros(1, 100, device="cuda"), top_n=33)):
        with pytest.raises(DecError):
            bad()
    r = ops.logprobs(x[:0], t[:0], top_n=3)
    assert r.logprob.shape == (0,) and r.top_ids.shape == (0, 3)
