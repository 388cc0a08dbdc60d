"""Attention mass of sequences that pass the end of their page table: nothing beyond it is read or written."""
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
