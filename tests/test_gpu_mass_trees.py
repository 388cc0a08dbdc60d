"""Attention mass after a step over trees of drafts: the accepted rows, moved into place, weigh as a chain."""
import numpy as np
import pytest
import torch

import drafts_ref as dr
from test_gpu_keep import _paged
from test_gpu_kvq import _cache, _cu, _ints, _np, _rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,hq,hkv", [(128, 8, 2), (64, 16, 1)])
def test_mass_of_accepted_paths(hd, hq, hkv):
    """Append with a tree's positions, attention under its mask, the path moved, the mass of its rows: what each row gives
    the positions that it saw, and nothing to its siblings, which are gone. Every row and head gives 1 in all."""
    from latency_moe_decode_gb300 import ops
    page, sizes, lens = 16, [9, 5, 12], [40, 0, 133]
    g, r = torch.Generator().manual_seed(hd), np.random.default_rng(hd)
    n = sum(sizes)
    cache, table = _cache([a + b for a, b in zip(sizes, lens)], hkv, hd, page)
    k, v = _rnd(g, sum(lens), hkv, hd), _rnd(g, sum(lens), hkv, hd)
    cache.append(k.cuda(), v.cuda(), _ints([0] * 3), table, cu_tokens=_cu(lens))
    parents = [dr.random_parents(r, m, 4) for m in sizes]
    rope = ops.rope_table(200, hd, 1e4)
    cu = _cu(sizes)
    tree = ops.draft_tree(_ints([p for ps in parents for p in ps]), _ints(lens), cu, max_tokens=max(sizes))
    q = cache.append(_rnd(g, n, hkv, hd).cuda(), _rnd(g, n, hkv, hd).cuda(), _ints(lens), table, cu_tokens=cu,
                     q=_rnd(g, n, hq, hd).cuda(), rope=rope, positions=tree.positions)
    _, lse = cache.attention(q, _ints(lens), table, cu_tokens=cu, max_tokens=max(sizes), return_lse=True, tree_mask=tree.mask)
    paths = [dr.paths(ps)[-1] for ps in parents]
    count = [len(p) for p in paths]
    index = torch.full((3, max(sizes)), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        index[b, :len(p)] = torch.tensor(p)
    cache.move(index.cuda(), _ints(count), table, start=_ints(lens))
    first = np.cumsum([0] + sizes)
    rows = torch.tensor([int(first[b]) + j for b, p in enumerate(paths) for j in p]).cuda()
    mass = cache.new_mass()
    cache.attention_mass(q[rows], lse[rows].contiguous(), _ints(lens), table, mass, cu_tokens=_cu(count), max_tokens=max(count))
    cache.check()
    total = [l + c for l, c in zip(lens, count)]
    kk, _ = cache.gather(_ints([0] * 3), table, sum(total), cu_tokens=_cu(total))
    at, row = np.cumsum([0] + total), 0
    for b, got in enumerate(_paged(mass, table, total, page)):
        keys, want = _np(kk[at[b]:at[b + 1]]), np.zeros((hkv, total[b]))
        big = 0.0
        for j in range(count[b]):
            for i in range(hq):
                s = keys[:lens[b] + j + 1, i * hkv // hq] @ _np(q[rows[row], i]) * hd ** -0.5
                big = max(big, (np.abs(keys[:lens[b] + j + 1, i * hkv // hq]) @ np.abs(_np(q[rows[row], i]))).max() * hd ** -0.5)
                e = np.exp(s - s.max())
                want[i * hkv // hq, :lens[b] + j + 1] += e / e.sum()
            row += 1
        # (as test_gpu_keep's bounds, and the lse's own: the same scores' errors, and fp32's of a sum of `total` terms)
        tol = 2 * (hd * 2.0 ** -23 * big + 2.0 ** -21 * (big + 8)) + 2.0 ** -22 * (total[b] + hq + 40)
        assert (np.abs(got - want) <= tol * want + 2.0 ** -30).all()
        assert np.abs(got.sum(1) - count[b] * hq / hkv).max() <= count[b] * hq / hkv * tol
