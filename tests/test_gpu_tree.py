"""Trees of drafted tokens over the paged 4-bit cache on the GPU (draft_tree, attention with a mask, append with rotary
positions of its own) against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import drafts_ref as dr
import kvq_ref as ref
from test_gpu_kvq import BF, F32, _cache, _cu, _ints, _np, _rnd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,first", [([1], 0), ([16], 0), ([33, 1, 0, 64, 7], 3), ([1024, 31, 32], 0)])
@pytest.mark.parametrize("width", [1, 5, 2000])
def test_masks_and_positions(sizes, first, width):
    from latency_moe_decode_gb300 import ops
    g = np.random.default_rng(len(sizes) + width)
    parents = [dr.random_parents(g, n, width) if n else [] for n in sizes]
    if len(sizes) > 1:  # parents that are no earlier rows: the row begins a path of its own
        parents[0][5], parents[0][6], parents[0][7] = 5, 900, -3
    lens = [7 * b for b in range(len(sizes))]
    n = first + sum(sizes) + 2  # (rows of no sequence before and behind)
    flat = [0] * first + [p for ps in parents for p in ps] + [0, 0]
    most = max(sizes)
    w = (most + 31) // 32
    tree = ops.draft_tree(_ints(flat), _ints(lens), _cu(sizes, first), max_tokens=most)
    row = first
    for ps, l in zip(parents, lens):
        want = dr.paths(ps)
        if want:
            assert np.array_equal(tree.mask[row:row + len(ps)].cpu().numpy(), dr.words(want, w))
            assert tree.positions[row:row + len(ps)].tolist() == [l + len(a) - 1 for a in want]
        row += len(ps)
    # what belongs to no sequence stays as it was
    from latency_moe_decode_gb300 import capi
    mask = torch.full((n, w + 1), -5, dtype=torch.int32, device="cuda")
    pos = torch.full((n,), -5, dtype=torch.int32, device="cuda")
    pa, ln, cu = _ints(flat), _ints(lens), _cu(sizes, first)
    a = capi.DecDraftTreeArgs(len(sizes), n, cu.data_ptr(), pa.data_ptr(), ln.data_ptr(), most, mask.data_ptr(), w + 1, pos.data_ptr())
    assert capi.lib().dec_draft_tree(a, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert (mask[:, w] == -5).all() and (mask[:first] == -5).all() and (mask[n - 2:] == -5).all()
    assert (pos[:first] == -5).all() and (pos[n - 2:] == -5).all()
    assert torch.equal(mask[first:n - 2, :w], tree.mask[first:n - 2])


TREES = [
    # hd, hq, hkv, page, rows, lengths, width, kind of mask
    (128, 8, 2, 16, [1], [0], 1, "tree"),
    (128, 32, 8, 64, [16], [1000], 4, "tree"),        # 64 query rows a KV head
    (128, 4, 2, 32, [4, 1, 3], [130, 0, 31], 3, "tree"),   # 8: the streaming kernel's first form
    (128, 8, 4, 16, [8, 5, 7, 1], [0, 300, 17, 512], 3, "any"),  # 16: its second
    (128, 4, 4, 64, [70, 3, 40], [129, 1000, 0], 9, "tree"),
    (128, 8, 1, 128, [17, 33], [2000, 5], 4, "any"),
    (64, 4, 2, 16, [13, 1, 2], [301, 0, 40], 3, "any"),
    (64, 8, 2, 64, [33, 64, 20], [127, 0, 700], 6, "tree"),
    (64, 2, 2, 256, [200], [90], 11, "any"),
]


def _tree_case(hd, hq, hkv, page, sizes, lens, width, kind, seed=0):
    g, r = torch.Generator().manual_seed(hd + hq + sum(sizes) + seed), np.random.default_rng(sum(lens) + seed)
    held = [a + b for a, b in zip(sizes, lens)]
    n = sum(sizes)
    chan = 1 + 5 * (torch.rand(hkv, hd, generator=g) < 0.03)
    k, v = (_rnd(g, sum(held), hkv, hd) * chan).to(BF), _rnd(g, sum(held), hkv, hd)
    q = _rnd(g, n, hq, hd, scale=0.8)
    cache, table = _cache(held, hkv, hd, page, seed)
    zero = _ints([0] * len(lens))
    cache.append(k.cuda(), v.cuda(), zero, table, cu_tokens=_cu(held))
    if kind == "tree":
        sees = [a for m in sizes for a in dr.paths(dr.random_parents(r, m, width))]
    else:  # any set of rows, itself or later ones among them, or none
        sees = [[i for i in range(m) if r.random() < 0.4] if j % 5 else [] for m in sizes for j in range(m)]
    return cache, table, q, k, v, held, sees


def _check_rows(out, lse, q, k, v, sizes, lens, held, sees, kept, skip=()):
    at = row = 0
    hd = q.shape[2]
    for m, l, h in zip(sizes, lens, held):
        kk, vv = ref.store(_np(k[at:at + h]))[0], ref.store(_np(v[at:at + h]))[0]
        for j in range(m):
            if row + j in skip:
                continue
            sel = list(range(l)) + [l + i for i in sees[row + j]]
            want, wl, mass, big = ref.attend(_np(q[row + j]), kk[sel], vv[sel], hd ** -0.5, len(sel), kept)
            ob, lb = ref.out_bounds(want, wl, mass, big, hd, len(sel))
            assert (np.abs(out[row + j] - want) <= ob).all(), (row, j)
            if sel:
                assert (np.abs(lse[row + j] - wl) <= lb).all(), (row, j)
            else:
                assert (out[row + j] == 0).all() and (lse[row + j] == -np.inf).all()
        at, row = at + h, row + m


@pytest.mark.parametrize("hd,hq,hkv,page,sizes,lens,width,kind", TREES)
def test_tree_attention(hd, hq, hkv, page, sizes, lens, width, kind):
    cache, table, q, k, v, held, sees = _tree_case(hd, hq, hkv, page, sizes, lens, width, kind)
    most = max(sizes)
    w = (most + 31) // 32
    # words further apart, and bits of rows that are not there
    m = torch.full((sum(sizes), w + 2), -1, dtype=torch.int32)
    m[:, :w] = torch.from_numpy(dr.words(sees, w))
    row = 0
    for s in sizes:
        for i in range(s, w * 32):
            bit = np.array([1 << (i % 32)], np.uint32).view(np.int32)[0]
            m[row:row + s, i // 32] |= int(bit)
        row += s
    m = m.cuda()
    out, lse = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(sizes), max_tokens=most, tree_mask=m[:, :w],
                               return_lse=True)
    rows = most * hq // hkv
    _check_rows(_np(out), _np(lse), q, k, v, sizes, lens, held, sees, 2.0 ** -29 if rows <= (16 if hd == 128 else 32) else 2.0 ** -21)
    # the kernel that the sequences' mean chooses, and words that the tree does not need
    wide = torch.zeros(sum(sizes), w + 3, dtype=torch.int32, device="cuda")
    wide[:, :w] = m[:, :w]
    out2, lse2 = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(sizes), tree_mask=wide, return_lse=True)
    _check_rows(_np(out2), _np(lse2), q, k, v, sizes, lens, held, sees, 2.0 ** -21)
    cache.check()


@pytest.mark.parametrize("hq", [2, 4, 32])
def test_a_chain_is_the_causal_attention(hq):
    """Masks of a chain see what causal rows see: the same kernels, the same bits."""
    from latency_moe_decode_gb300 import ops
    sizes, lens = [8, 3], [100, 0]
    cache, table, q, *_ = _tree_case(128, hq, 2, 32, sizes, lens, 1, "tree")
    tree = ops.draft_tree(_ints([-1] + list(range(7)) + [-1, 0, 1]), _ints(lens), _cu(sizes), max_tokens=8)
    a = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(sizes), max_tokens=8, return_lse=True)
    b = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(sizes), max_tokens=8, tree_mask=tree.mask, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert tree.positions.tolist() == [100 + i for i in range(8)] + [0, 1, 2]


@pytest.mark.parametrize("hd,hq,hkv,sizes", [(128, 2, 2, [7]), (128, 4, 2, [8]), (128, 8, 2, [40]), (64, 4, 1, [9])])
def test_rows_that_are_not_seen_may_hold_anything(hd, hq, hkv, sizes):
    """A draft whose keys and values are NaN or infinite spoils the rows that see it, and no other."""
    lens = [37]
    m = sizes[0]
    cache, table, q, k, v, held, sees = _tree_case(hd, hq, hkv, 16, sizes, lens, 3, "tree")
    bad = m - 2
    for what in (float("nan"), float("inf")):
        for side in (k, v):
            kk, vv = k.clone(), v.clone()
            (kk if side is k else vv)[37 + bad, :, 5] = what
            cache.append(kk.cuda(), vv.cuda(), _ints([0]), table, cu_tokens=_cu(held))
            mask = torch.from_numpy(dr.words(sees, (m + 31) // 32)).cuda()
            out, lse = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(sizes), max_tokens=m, tree_mask=mask, return_lse=True)
            hit = [j for j in range(m) if bad in sees[j]]
            assert bad in hit and len(hit) < m
            _check_rows(_np(out), _np(lse), q, k, v, sizes, lens, held, sees, 2.0 ** -21, skip=hit)
            o = _np(out)[hit]
            assert np.isnan(o if side is k else o[:, :, :16]).all()
    # in the stored prefix every row sees it
    vv = v.clone()
    vv[20, :, 5] = float("nan")
    cache.append(k.cuda(), vv.cuda(), _ints([0]), table, cu_tokens=_cu(held))
    out = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(sizes), max_tokens=m, tree_mask=mask)
    assert torch.isnan(out[:, :, :16]).all()


def test_bad_pages_and_lengths_are_recorded():
    from latency_moe_decode_gb300.capi import DecError
    sizes, lens = [5, 20], [40, 40]
    for most in (5, 20):
        cache, table, q, k, v, held, sees = _tree_case(128, 4, 2, 16, sizes, lens, 3, "tree")
        mask = torch.from_numpy(dr.words(sees, 1)).cuda()
        for t, ln in ((-1, lens), (10 ** 6, lens), (None, [40, -3]), (None, [40, 10 ** 6])):
            tab = table.clone()
            if t is not None:
                tab[1, 1] = t
            out, lse = cache.attention(q.cuda(), _ints(ln), tab, cu_tokens=_cu(sizes), max_tokens=most, tree_mask=mask, return_lse=True)
            with pytest.raises(DecError):
                cache.check()
            _check_rows(_np(out[:5]), _np(lse[:5]), q[:5], k, v, sizes[:1], lens[:1], held[:1], sees[:5], 2.0 ** -21)


@pytest.mark.parametrize("hd,dtype,rot,inter", [(128, BF, 128, False), (128, F32, 64, True), (64, F32, 64, False)])
def test_append_with_positions_of_its_own(hd, dtype, rot, inter):
    """Keys and queries turn by the positions given, and stand where lengths says."""
    from latency_moe_decode_gb300 import ops
    g = torch.Generator().manual_seed(hd + rot)
    sizes, lens, hkv = [5, 1, 9], [17, 0, 300], 2
    n = sum(sizes)
    q, k, v = (_rnd(g, n, h, hd, dtype=dtype) for h in (4, hkv, hkv))
    pos = torch.randint(0, 5000, (n,), generator=g).to(torch.int32)
    rope = ops.rope_table(5000, rot, 1e4)
    cache, table = _cache([a + b for a, b in zip(sizes, lens)], hkv, hd, 16)
    kw = dict(cu_tokens=_cu(sizes), q=q.cuda(), rope=rope, interleaved=inter)
    qo = cache.append(k.cuda(), v.cuda(), _ints(lens), table, positions=pos.cuda(), **kw)
    gk, gv = cache.gather(_ints(lens), table, n, cu_tokens=_cu(sizes))
    # the same rows, each a sequence at that position
    other, t2 = _cache([5000] * n, hkv, hd, 256)
    qo2 = other.append(k.cuda(), v.cuda(), pos.cuda(), t2, q=q.cuda(), rope=rope, interleaved=inter)
    gk2, gv2 = other.gather(pos.cuda(), t2, n)
    assert torch.equal(qo, qo2) and torch.equal(gk, gk2) and torch.equal(gv, gv2)
    cache.check()
    # beyond the table, and negative: the row stays as it was
    from latency_moe_decode_gb300.capi import DecError
    for bad, st in ((5000, -8), (-1, -1)):
        p2 = pos.clone()
        p2[3] = bad
        keep = qo.clone()
        cache.append(k.cuda() * 2, v.cuda() * 2, _ints(lens), table, positions=p2.cuda(), q_out=keep, **kw)
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == st
        a, b = cache.gather(_ints(lens), table, n, cu_tokens=_cu(sizes))
        assert torch.equal(a[3], gk[3]) and torch.equal(b[3], gv[3]) and torch.equal(keep[3], qo[3])
        cache.append(k.cuda(), v.cuda(), _ints(lens), table, positions=pos.cuda(), **kw)
