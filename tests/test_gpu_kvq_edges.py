"""Calls at the edges of what the paged 4-bit cache's operators are given."""
import numpy as np
import pytest
import torch

import kvq_ref as ref
from tests.test_gpu_kvq import _cache, _check, _cu, _filled, _ints, _np, _rnd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("batch", [0, 2])
def test_no_rows(batch):
    cache, table = _cache([20, 20], 2, 128, 16)
    pages = cache.pages.clone()
    kv, q = (torch.zeros(0, h, 128, dtype=BF, device="cuda") for h in (2, 8))
    ln, t = _ints([3, 5][:batch]), table[:batch]
    cu = _cu([0] * batch) if batch else None
    for kw in (dict(), dict(q=q), dict(q=q, q_out=torch.empty_like(q))):
        out = cache.append(kv, kv, ln, t, cu_tokens=cu, **kw)
        assert out is None if not kw else out.shape == (0, 8, 128) and out.dtype == BF
    k, v = cache.gather(ln, t, 0, cu_tokens=cu)
    out, lse = cache.attention(q, ln, t, cu_tokens=cu, return_lse=True)
    assert k.shape == v.shape == (0, 2, 128) and out.shape == (0, 8, 128) and lse.shape == (0, 8)
    cache.check()
    assert torch.equal(pages, cache.pages)


@pytest.mark.parametrize("dtype,hd,rot", [(BF, 128, 128), (F32, 64, 32)])
@pytest.mark.parametrize("status", [True, False])
def test_rows_beyond_the_rotation_table_are_not_appended_by_half(dtype, hd, rot, status):
    """Rows inside the page table and beyond the rotation table leave the page and their queries' place as they
    were, values included; rows before it are appended as ever. Also where no status word is kept."""
    from latency_moe_decode_gb300 import ops
    from latency_moe_decode_gb300.capi import DecError
    g = torch.Generator().manual_seed(hd)
    n, hkv, hq, reach = 30, 2, 4, 21
    cache, table = _cache([n], hkv, hd, 16)
    q, k, v = (_rnd(g, n, h, hd, dtype=dtype).cuda() for h in (hq, hkv, hkv))
    ln, rope = _ints([0]), ops.rope_table(n, rot, 1e4)
    cache.append(k, v, ln, table, cu_tokens=_cu([n]), rope=rope)
    k2, v2 = (torch.randn(n, hkv, hd, generator=g).to(dtype).cuda() for _ in range(2))
    if not status:
        cache.c.status = None
    pages = cache.pages.clone()
    out = torch.full((n, hq, hd), 9.0, dtype=BF, device="cuda")
    cache.append(k2[reach:], v2[reach:], _ints([reach]), table, cu_tokens=_cu([n - reach]), q=q[reach:], q_out=out[reach:],
                 rope=rope[:reach])
    assert torch.equal(pages, cache.pages) and (out == 9).all()
    cache.append(k2, v2, ln, table, cu_tokens=_cu([n]), q=q, q_out=out, rope=rope[:reach])
    want = _cache([n], hkv, hd, 16)
    want[0].append(k, v, ln, want[1], cu_tokens=_cu([n]), rope=rope)
    qo = want[0].append(k2[:reach], v2[:reach], ln, want[1], cu_tokens=_cu([reach]), q=q[:reach], rope=rope)
    assert torch.equal(out[:reach], qo) and (out[reach:] == 9).all()
    for a, b in zip(cache.gather(ln, table, n, cu_tokens=_cu([n])), want[0].gather(ln, want[1], n, cu_tokens=_cu([n]))):
        assert torch.equal(a, b)
    if status:
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == -8


@pytest.mark.parametrize("hd,dtype,norm,rot,inter", [(128, BF, True, 128, False), (128, F32, False, 128, False),
                                                     (64, BF, False, 32, False), (64, F32, True, 64, True), (128, BF, False, 16, False)])
@pytest.mark.parametrize("size", [30.0, 300.0, 3e4])
def test_codes_of_runs_that_a_rotation_leaves_small(hd, dtype, norm, rot, inter, size):
    """Pairs of large values that turn into one small and one large one: the small one keeps the large ones'
    roundings, and is held as the formula in 64 bits says all the same. (One pair or all pairs of a run; runs of
    adjacent pairs hold both values.)"""
    from latency_moe_decode_gb300 import ops
    n, hkv = 2 ** 18 // hd, 8
    g = torch.Generator().manual_seed(hd + rot)
    k = torch.randn(n, hkv, hd, generator=g)
    rope = ops.rope_table(n, rot, 1e6)
    c, s = rope.cpu().unbind(-1)
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    r = size * (0.5 + torch.rand(n, hkv, rot // 2, generator=g))
    r[:, ::2] *= (torch.rand(n, hkv // 2, rot // 2, generator=g) < 0.1)  # some heads: a pair of a run now and then
    k[..., a] += r * s[:, None]
    k[..., b] += r * c[:, None]  # a cos - b sin: what the rounding to the type and the noise leave
    k = k.to(dtype)
    kn = (1 + 0.2 * torch.randn(hd, generator=g)).to(BF) if norm else None
    if norm:  # (a pair's two weights alike, or the norm undoes the angle)
        kn[b] = kn[a]
    cache, table = _cache([n], hkv, hd, 64)
    cache.append(k.cuda(), k.cuda(), _ints([0]), table, cu_tokens=_cu([n]), k_norm=None if kn is None else kn.cuda(),
                 rope=rope, interleaved=inter)
    got = _np(cache.gather(_ints([0]), table, n, cu_tokens=_cu([n]))[0])
    cache.check()
    held = ref.store(ref.norm_rotate(_np(k), None if kn is None else _np(kn), 1e-6, _np(rope), np.arange(n), inter))[0]
    wrong = got != held
    assert not wrong.any(), (wrong.sum(), got[wrong][:4], held[wrong][:4])


def test_the_public_way_to_the_current_stream(monkeypatch):
    """The handle that a torch without the short cut would give is the same, on any stream."""
    from latency_moe_decode_gb300 import ops
    cache, table, _, _, g = _filled([40], 2, 128, 16, 3)
    q = _rnd(g, 1, 8, 128).cuda()
    s = torch.cuda.Stream()
    want = cache.attention(q, _ints([39]), table)
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), s):
        with torch.cuda.stream(stream):
            assert ops._current_raw_stream(0) == ops._raw_stream(0) == stream.cuda_stream
    monkeypatch.setattr(ops, "_raw_stream", ops._current_raw_stream)
    ln = _ints([39])
    torch.cuda.synchronize()
    got = cache.attention(q, ln, table, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_raw_streams_through_every_call():
    from latency_moe_decode_gb300 import ops
    cache, table, _, _, g = _filled([40], 2, 128, 16, 4)
    kv, q = _rnd(g, 1, 2, 128).cuda(), _rnd(g, 1, 8, 128).cuda()
    logits, t = torch.randn(3, 500, generator=g).cuda(), _ints([1, 2, 3])
    ln = _ints([39])

    def calls(stream):
        qo = cache.append(kv, kv, ln, table, q=q, stream=stream)
        got = [qo, *cache.gather(ln, table, 1, stream=stream), cache.attention(q, ln, table, stream=stream)]
        got += [x for x in ops.logprobs(logits, t, top_n=3, stream=stream)]
        torch.cuda.synchronize()
        return got

    s = torch.cuda.Stream()
    want = calls(None)
    for stream in (s, s.cuda_stream, 0, torch.cuda.default_stream()):
        assert all(torch.equal(a, b) for a, b in zip(calls(stream), want))
    with pytest.raises(ValueError):
        ops.logprobs(logits.cpu(), stream=s)


@pytest.mark.parametrize("hd,hq,hkv", [(128, 8, 2), (64, 8, 1)])
def test_the_default_bound_takes_decode_batches_to_their_own_kernel(hd, hq, hkv):
    """cu_tokens without max_tokens: the same bits as with the rows that the sequences have."""
    for new in ([1] * 40, [2, 1] * 9 + [0], [30, 41, 25]):
        lens = [(37 * i) % 300 for i in range(len(new))]
        cache, table, _, _, g = _filled([l + n for l, n in zip(lens, new)], hkv, hd, 16, 8)
        q = _rnd(g, sum(new), hq, hd).cuda()
        a = cache.attention(q, _ints(lens), table, cu_tokens=_cu(new), return_lse=True)
        b = cache.attention(q, _ints(lens), table, cu_tokens=_cu(new), max_tokens=max(new), return_lse=True)
        cache.check()
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_more_rows_than_were_likely():
    """Every kernel takes any number of rows: one sequence of many among single tokens; and a call whose rows would
    not fit the list of the likely kernel goes to the other one."""
    from latency_moe_decode_gb300 import ops
    from latency_moe_decode_gb300.capi import DecKvqAttentionArgs
    hd, hq, hkv = 128, 8, 2
    new = [1] * 30 + [50] + [1] * 9
    lens = [(53 * i) % 200 for i in range(len(new))]
    cache, table, k, v, g = _filled([l + n for l, n in zip(lens, new)], hkv, hd, 16, 9)
    q = _rnd(g, sum(new), hq, hd)
    out, lse = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(new), return_lse=True)
    cache.check()
    _check(_np(out), _np(lse), _np(q), k, v, new, lens, True, hd ** -0.5, hd)
    # rows 3 .. a million belong to no sequence; the table could reach a million positions
    n = 1 << 20
    wide = torch.zeros(1, n // 16, dtype=torch.int32, device="cuda")
    wide[0, :table.shape[1]] = table[30]
    ln, cu, dev, res = _ints([50]), _cu([3]), q.cuda(), []
    for rows, likely in ((3, 0), (n, 1)):
        o = torch.zeros(3, hq, hd, dtype=BF, device="cuda")
        ws = torch.empty(cache.lib.dec_kvq_attention_workspace(cache.c, hq, 1, rows), dtype=torch.uint8, device="cuda")
        a = DecKvqAttentionArgs(hq, dev.data_ptr(), hq * hd, hd, o.data_ptr(), hq * hd, hd, None, 0.0, 1, rows, ws.data_ptr(),
                                ws.numel(), likely)
        s = cache._seqs(ln, wide, cu, rows)
        assert cache.lib.dec_kvq_attention(cache.c, s, a, None) == 0, cache.lib.dec_op_error()
        torch.cuda.synchronize()
        res.append(o.float())
    cache.check()
    assert res[0].abs().sum() > 0 and (res[0] - res[1]).abs().max() < 0.05  # (as bounds of other kernels: 0.044)


@pytest.mark.parametrize("m", [1, 3, 20])
@pytest.mark.parametrize("bounds", [[0, 2, 1, 4], [4, 3, 2, 0], [-1, 1, 2, 4], [0, 3, 3, 2]])
def test_token_bounds_that_do_not_ascend(bounds, m):
    """Reported, and nothing computed, by each of the kernels (as few, more and many rows choose them)."""
    from latency_moe_decode_gb300.capi import DecError
    lens = [30, 5, 90]
    cache, table, _, _, g = _filled([l + 2 * m for l in lens], 2, 128, 16, 10)
    q = _rnd(g, 4 * m, 8, 128).cuda()
    out = torch.full_like(q, 3.0)
    cu = _ints([b * m for b in bounds])
    cache.attention(q, _ints(lens), table, cu_tokens=cu, max_tokens=m, out=out)
    with pytest.raises(DecError) as e:
        cache.check()
    assert e.value.status == -1 and (out == 3).all()
    good = _ints([0, m, 2 * m, 2 * m])
    cache.attention(q, _ints(lens), table, cu_tokens=good, max_tokens=m, out=out)
    cache.check()
    assert (out[:2 * m] != 3).any(-1).all() and (out[2 * m:] == 3).all()
