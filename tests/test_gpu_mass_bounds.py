"""Attention mass at the bounds of what it says: sequences that pass the end of their page table (nothing beyond it is
read or written), queries of far apart values, sequences beside others."""
import numpy as np
import pytest
import torch

from test_gpu_keep import _mass_want, _paged
from test_gpu_kvq import _cu, _ints, _rnd

pytestmark = pytest.mark.gpu

# hd, hq, hkv, page, pages of a table's row, rows of the sequence that passes it, by how many positions
PAST = [
    (128, 16, 2, 16, 3, 4, 4),     # 52 positions of 48, many query rows
    (128, 16, 2, 16, 21, 64, 1),
    (128, 16, 2, 16, 21, 64, 100),  # (the whole of them, and what was there before)
    (64, 8, 1, 16, 9, 40, 37),
    (128, 8, 2, 64, 3, 30, 1),
    (64, 16, 2, 64, 5, 100, 100),
    (128, 8, 8, 32, 7, 17, 9),
    (128, 8, 2, 16, 3, 2, 1),      # few query rows
    (64, 4, 2, 16, 5, 4, 3),
    (128, 8, 1, 64, 1, 1, 1),
]


@pytest.mark.parametrize("hd,hq,hkv,page,pages,n,past", PAST)
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("decay", [0.0, 0.5])
def test_mass_past_the_page_table(hd, hq, hkv, page, pages, n, past, last, decay):
    """Sequence 0 (or the last one) has `past` rows more than its table's row holds. What lies behind the row, guard
    pages' numbers or the next sequence's, is left as it is; the other sequence's masses are those of a call in which this
    one keeps within its table, bit for bit; its own are the formula's over the positions that it has."""
    from latency_moe_decode_gb300 import ops
    from latency_moe_decode_gb300.capi import DecError
    g = torch.Generator().manual_seed(n + past)
    most, m = pages * page, max(1, n // 2)
    guards = 16
    for guarded in (False, True):
        cache = ops.KvqCache(2 * pages + 2 * guards, hkv, hd, page_tokens=page)
        ids = torch.randperm(2 * pages, generator=g).view(2, pages)
        wide = torch.cat([ids, torch.arange(2 * pages, 2 * pages + 2 * guards).view(2, guards)], 1).to(torch.int32).cuda()
        table = wide[:, :pages] if guarded else wide[:, :pages].contiguous()
        k, v = _rnd(g, 2 * most, hkv, hd, scale=1.5), _rnd(g, 2 * most, hkv, hd)
        cache.append(k.cuda(), v.cuda(), _ints([0, 0]), table, cu_tokens=_cu([most, most]))
        cache.check()
        bad, good = (1, 0) if last else (0, 1)
        new, lens = [0, 0], [0, 0]
        new[bad], lens[bad] = n, most - n + past
        new[good], lens[good] = m, most - m
        q, lse = _rnd(g, n + m, hq, hd), 6 + torch.randn(n + m, hq, generator=g)
        was = torch.rand((cache.n_pages, hkv, page), generator=g).cuda()
        call = lambda ln: cache.attention_mass(q.cuda(), lse.cuda(), _ints(ln), table, was, cu_tokens=_cu(new), max_tokens=max(n, m),
                                               decay=decay, out=torch.full_like(was, -3.0))
        got = call(lens)
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == -8
        within = list(lens)
        within[bad] = most - n
        other = call(within)
        cache.check()
        own = ids[good].tolist()
        assert (got[2 * pages:] == -3.0).all() and torch.equal(got[own], other[own])
        want, bound = _mass_want(q, k, lse, new, lens, [most, most], True, bad, bad * most, 0 if bad == 0 else m, decay,
                                 _paged(was, table, [most, most], page)[bad])
        assert (np.abs(_paged(got, table, [most, most], page)[bad] - want) <= bound).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n,low", [(1, -17), (2, -17), (5, -40)])
def test_queries_enter_exactly(hd, n, low):
    """Each head's largest query value meets keys of 0, and all others are 2^low of it and less, with eight bits each: in calls
    of up to 16 query rows a KV head down to 2^-17, in those of more at any distance. Their scores alone count."""
    from latency_moe_decode_gb300 import ops
    hkv, group, page, length = 2, 8, 32, 200
    hq = hkv * group
    g = torch.Generator().manual_seed(n + hd)
    k = torch.randint(-7, 8, (length + n, hkv, hd), generator=g).float()
    k[..., ::16] = 7.0  # (every run's scale is 1: codes are values)
    k[..., 1] = 0.0
    q = torch.randint(128, 256, (n, hq, hd), generator=g).float() * 2.0 ** (low - 7)  # in [2^low, 2^(low + 1))
    q[..., 1] = 1.5
    q *= torch.where(torch.rand(q.shape, generator=g) < 0.5, -1.0, 1.0)
    scale = 2.0 ** -low / hd
    cache = ops.KvqCache(16, hkv, hd, page_tokens=page)
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None]
    cache.append(k.to(torch.bfloat16).cuda(), k.to(torch.bfloat16).cuda(), _ints([0]), table, cu_tokens=_cu([length + n]))
    lse = torch.full((n, hq), 3.0)
    mass = cache.new_mass()
    cache.attention_mass(q.to(torch.bfloat16).cuda(), lse.cuda(), _ints([length]), table, mass, cu_tokens=_cu([n]), max_tokens=n,
                         decay=0.0, scale=scale)
    cache.check()
    got = _paged(mass, table, [length + n], page)[0]
    s = torch.einsum("jhgd,phd->hjgp", q.view(n, hkv, group, hd).double(), k.double()) * scale
    pos, row = torch.arange(length + n), torch.arange(n)
    e = torch.exp(s - 3.0).masked_fill((pos > length + row[:, None])[None, :, None], 0.0)
    # fp32: products' sums (hd terms of 2^(low + 1) 7), the exponent's roundings, the sum over rows
    big = hd * 14 / hd
    tol = hd * 2.0 ** -23 * big + 2.0 ** -21 * (big + 4) + 2.0 ** -23 * (n * group + 8)
    want = e.sum((1, 2)).numpy()
    assert (np.abs(got - want) <= want * tol + 2.0 ** -126).all()


@pytest.mark.parametrize("hd,hq,hkv,n", [(128, 8, 2, 1), (128, 8, 2, 4), (64, 16, 2, 30)])
def test_sequences_beside_others(hd, hq, hkv, n):
    """A sequence's masses are the same bits alone (with rows of no sequence behind it, so that the call's size chooses the
    same kernel) and between others."""
    from test_gpu_keep import _mass_case
    new, lens, page = [n, max(1, n // 2), n], [300, 511, 77], 16
    cache, table, q, k, lse, held = _mass_case(hd, hq, hkv, page, new, lens, True)
    was = torch.rand((cache.n_pages, hkv, page), device="cuda")
    out = cache.attention_mass(q.cuda(), lse, _ints(lens), table, was, cu_tokens=_cu(new), max_tokens=n, decay=0.5,
                               out=torch.zeros_like(was))
    for b in range(3):
        at = [0, new[0], new[0] + new[1]][b]
        one = cache.attention_mass(q.cuda(), lse, _ints(lens[b:b + 1]), table[b:b + 1], was, cu_tokens=_ints([at, at + new[b]]),
                                   max_tokens=n, decay=0.5, out=torch.zeros_like(was))
        assert np.array_equal(_paged(one, table[b:b + 1], held[b:b + 1], page)[0], _paged(out, table[b:b + 1], held[b:b + 1], page)[0])
