"""A bounded cache on the GPU (attention_mass, heaviest, move, evict) against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import kvq_ref as ref
from test_gpu_kvq import BF, _cache, _cu, _ints, _np, _rnd

pytestmark = pytest.mark.gpu


def _paged(t, table, lens, page):
    """Each sequence's part of a paged tensor [n_pages, hkv, page]: [hkv, positions]."""
    t, table = _np(t), table.cpu().numpy()
    return [np.concatenate([t[table[b, i]] for i in range((n + page - 1) // page)] + [t[0][:, :0]], 1)[:, :n]
            for b, n in enumerate(lens)]


MASS = [
    # hd, hq, hkv, page, rows, lengths, causal
    (128, 32, 8, 64, [1], [1000], True),
    (128, 8, 2, 16, [1, 1, 1, 1], [0, 15, 16, 4000], True),
    (128, 8, 1, 32, [2, 1, 0], [31, 500, 7], True),         # 16 query rows
    (128, 4, 2, 16, [5, 40, 1], [33, 0, 700], True),        # many
    (128, 16, 2, 128, [64, 100], [3000, 130], True),
    (128, 4, 4, 64, [3, 1], [100, 0], False),
    (64, 4, 2, 16, [1, 2, 1], [301, 0, 40], False),
    (64, 8, 8, 16, [1, 1], [511, 512], True),
    (64, 8, 2, 64, [70, 1, 257], [17, 255, 0], True),
    (64, 4, 1, 256, [9, 3], [700, 0], False),
    (128, 8, 2, 16, [300, 7, 64, 1, 150, 33], [50, 700, 0, 129, 400, 1000], True),  # blocks that see some tiles only
    (64, 16, 1, 64, [130, 40, 2, 0, 65], [3, 1500, 260, 9, 127], True),
]


def _mass_case(hd, hq, hkv, page, new, lens, causal, seed=0):
    g = torch.Generator().manual_seed(hd + hq + sum(new) + seed)
    held = [a + b if causal else b for a, b in zip(new, lens)]
    t = max(1, sum(held))
    k, v = _rnd(g, t, hkv, hd, scale=1.5), _rnd(g, t, hkv, hd)
    q = _rnd(g, sum(new), hq, hd)
    cache, table = _cache([a + b for a, b in zip(new, lens)], hkv, hd, page, seed)
    if sum(held):
        cache.append(k[:sum(held)].cuda(), v[:sum(held)].cuda(), _ints([0] * len(lens)), table, cu_tokens=_cu(held))
    _, lse = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(new), max_tokens=max(new), causal=causal, return_lse=True)
    return cache, table, q, k, lse, held


def _mass_want(q, k, lse, new, lens, held, causal, b, off, row, decay, was):
    """(sums of sequence b's positions, bounds). A term exp(s - l) is off by the factor of its score's error (out_bounds':
    hd 2^-23 of sum |q k| for the products' sums, the queries' scaling, the exponent's rounding) and of l's rounding, 2^-23
    |l| with its product with log2 e; terms and the old weight join in fp32, one rounding of the running sum a term."""
    n, l, h = new[b], lens[b], held[b]
    if h == 0:
        return np.zeros((k.shape[1], 0)), np.zeros((k.shape[1], 0))
    kk = ref.store(_np(k[off:off + h]))[0]
    hq, hd = q.shape[1], q.shape[2]
    hkv = kk.shape[1]
    want, bound = np.zeros((hkv, h)), np.zeros((hkv, h))
    for j in range(n):
        seen = min(h, l + j + 1) if causal else h
        for i in range(hq):
            kv = i // (hq // hkv)
            li = float(lse[row + j, i])
            if not np.isfinite(li) or seen == 0:
                continue
            s = kk[:seen, kv] @ _np(q[row + j, i]) * hd ** -0.5
            big = (np.abs(kk[:seen, kv]) @ np.abs(_np(q[row + j, i]))).max() * hd ** -0.5
            e = np.exp(s - li)
            d = hd * 2.0 ** -23 * big + 2.0 ** -14 / hd * big * 2.0 ** -9 + 2.0 ** -21 * (big + 1) + 2.0 ** -22 * abs(li)
            want[kv, :seen] += e
            bound[kv, :seen] += e * (d + 2.0 ** -23 * (n * (hq // hkv) + 8)) + 2.0 ** -126
    old = np.zeros((hkv, h))
    old[:, :min(l, h)] = was[:, :min(l, h)] if decay else 0.0
    return want + decay * old, bound + 2.0 ** -22 * (decay * old + want)


@pytest.mark.parametrize("hd,hq,hkv,page,new,lens,causal", MASS)
def test_attention_mass(hd, hq, hkv, page, new, lens, causal):
    cache, table, q, k, lse, held = _mass_case(hd, hq, hkv, page, new, lens, causal)
    g = torch.Generator(device="cuda").manual_seed(3)
    was = torch.rand((cache.n_pages, hkv, page), generator=g, device="cuda")
    for decay in (0.0, 1.0, 0.75):
        if decay == 0.0:  # nothing of it is read
            mass = torch.full_like(was, float("nan"))
        else:
            mass = was.clone()
        out = torch.full_like(was, -3.0)
        ret = cache.attention_mass(q.cuda(), lse, _ints(lens), table, mass, cu_tokens=_cu(new), max_tokens=max(new),
                                   causal=causal, decay=decay, out=out)
        assert ret is out
        got = _paged(out, table, held, page)
        before = _paged(was, table, held, page)
        off = row = 0
        for b in range(len(new)):
            if new[b]:
                want, bound = _mass_want(q, k, lse.cpu(), new, lens, held, causal, b, off, row, decay, before[b])
                assert (np.abs(got[b] - want) <= bound).all(), (b, decay)
            else:
                assert (got[b] == -3.0).all()
            off, row = off + held[b], row + new[b]
        assert (out == -3.0).sum().item() == out.numel() - hkv * sum(h for h, n in zip(held, new) if n)
        # in place, and again: the same bits
        again = mass.clone()
        cache.attention_mass(q.cuda(), lse, _ints(lens), table, again, cu_tokens=_cu(new), max_tokens=max(new), causal=causal,
                             decay=decay)
        live = out != -3.0
        assert torch.equal(again[live], out[live])
        if decay:
            assert torch.equal(again[~live], was[~live])
    cache.check()


def test_mass_sums_to_the_rows():
    """Weights of a full softmax: over all positions they add up to the heads of the group, row by row."""
    cache, table, q, k, lse, held = _mass_case(128, 16, 4, 32, [1, 1], [777, 30], True)
    mass = cache.new_mass()
    cache.attention_mass(q.cuda(), lse, _ints([777, 30]), table, mass)
    for m in _paged(mass, table, held, 32):
        assert np.abs(m.sum(1) - 4).max() <= 4 * 2.0 ** -14


def test_mass_of_rows_without_an_lse_and_bad_pages():
    from latency_moe_decode_gb300.capi import DecError
    for new in ([1, 1], [30, 2]):
        lens = [100, 64]
        cache, table, q, k, lse, held = _mass_case(128, 8, 2, 16, new, lens, True)
        lse[0, 3], lse[0, 4], lse[0, 5] = float("nan"), float("inf"), -float("inf")
        mass = cache.new_mass()
        cache.attention_mass(q.cuda(), lse, _ints(lens), table, mass, cu_tokens=_cu(new), max_tokens=max(new), decay=0.0)
        got = _paged(mass, table, held, 16)
        want, bound = _mass_want(q, k, lse.cpu(), new, lens, held, True, 0, 0, 0, 0.0, got[0])
        assert (np.abs(got[0] - want) <= bound).all()
        cache.check()
        for bad in (-1, 10 ** 6):
            tab = table.clone()
            tab[0, 2] = bad
            m2 = torch.full_like(mass, -3.0)
            cache.attention_mass(q.cuda(), lse, _ints(lens), tab, m2, cu_tokens=_cu(new), max_tokens=max(new), decay=0.0)
            with pytest.raises(DecError):
                cache.check()
            other = torch.ones(cache.n_pages, dtype=torch.bool)
            other[table[0, 2].item()] = False
            used = torch.zeros_like(other)
            used[table[table >= 0].cpu().long()] = True
            pick = (other & used).nonzero()[:, 0].tolist()
            live = m2[pick] != -3.0
            assert live.any() and torch.equal(m2[pick][live], mass[pick][live])


def _heaviest_want(w, n, budget, sinks, recent):
    out = np.full((w.shape[0], budget), -1, np.int32)
    for h in range(w.shape[0]):
        if n <= budget:
            out[h, :n] = np.arange(n)
            continue
        mid = np.arange(sinks, n - recent)
        order = mid[np.argsort(-np.where(np.isnan(w[h, mid]), -np.inf, w[h, mid]), kind="stable")]
        # (a NaN orders below everything, -infinity included)
        x = w[h, order]
        order = np.concatenate([order[~np.isnan(x)], order[np.isnan(x)]])
        out[h] = np.sort(np.concatenate([np.arange(sinks), order[:budget - sinks - recent], np.arange(n - recent, n)]))
    return out


@pytest.mark.parametrize("lens,budget,sinks,recent,page,hkv", [
    ([1000], 100, 4, 32, 64, 2), ([33, 32, 31, 0, 1, 5000], 32, 1, 7, 16, 3), ([700, 90], 64, 0, 0, 32, 1),
    ([700, 90], 64, 30, 34, 32, 2), ([257], 256, 3, 5, 256, 1), ([2000, 40], 1, 0, 0, 16, 2), ([60000, 100], 7001, 4, 1000, 128, 2),
    ([130], 129, 0, 129, 16, 8)])
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
def test_heaviest(lens, budget, sinks, recent, page, hkv, kind):
    cache, table = _cache(lens, hkv, 64, page)
    g = torch.Generator().manual_seed(budget)
    mass = torch.exp(3 * torch.randn(cache.n_pages, hkv, page, generator=g))
    if kind == "ties":
        mass = (mass * 2).round().clamp(max=3) * torch.where(torch.rand(mass.shape, generator=g) < 0.5, 0.0, 1.0)
    if kind == "odd":
        r = torch.rand(mass.shape, generator=g)
        for lo, x in ((0.0, float("nan")), (0.1, float("inf")), (0.2, -float("inf")), (0.3, -1e-40), (0.4, -0.0), (0.5, 1e-42), (0.6, -2.5)):
            mass[(r >= lo) & (r < lo + 0.1)] = x
    mass = mass.cuda()
    kept, count = cache.heaviest(mass, _ints(lens), table, budget, sinks=sinks, recent=recent)
    cache.check()
    assert count.tolist() == [min(n, budget) for n in lens]
    for b, w in enumerate(_paged(mass, table, lens, page)):
        assert np.array_equal(kept[b].cpu().numpy(), _heaviest_want(w, lens[b], budget, sinks, recent)), b


def test_heaviest_of_bad_sequences():
    from latency_moe_decode_gb300.capi import DecError
    cache, table = _cache([200, 200], 2, 64, 16)
    mass = torch.rand((cache.n_pages, 2, 16), device="cuda")
    want, _ = cache.heaviest(mass, _ints([200, 200]), table, 50)
    for ln, st in (([200, -1], -1), ([200, 10 ** 6], -8)):
        kept, count = cache.heaviest(mass, _ints(ln), table, 50)
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == st
        assert torch.equal(kept[0], want[0]) and count.tolist() == [50, 0] and (kept[1] == -1).all()
    tab = table.clone()
    tab[1, 3] = 10 ** 6  # positions 48 .. 63 weigh nothing
    kept, count = cache.heaviest(mass, _ints([200, 200]), tab, 50, sinks=50)
    with pytest.raises(DecError):
        cache.check()
    assert torch.equal(kept[0], torch.arange(50, dtype=torch.int32, device="cuda").expand(2, -1))
    kept, _ = cache.heaviest(mass, _ints([200, 200]), tab, 50)
    with pytest.raises(DecError):
        cache.check()
    assert not ((kept[1] >= 48) & (kept[1] < 64)).any()


def _filled(lens, hkv, hd, page, seed=0):
    g = torch.Generator().manual_seed(seed + sum(lens))
    cache, table = _cache(lens, hkv, hd, page, seed)
    t = sum(lens)
    k, v = _rnd(g, t, hkv, hd), _rnd(g, t, hkv, hd)
    k[0, 0, 3] = float("nan")
    cache.append(k.cuda(), v.cuda(), _ints([0] * len(lens)), table, cu_tokens=_cu(lens))
    kk, vv = cache.gather(_ints([0] * len(lens)), table, t, cu_tokens=_cu(lens))
    at = np.cumsum([0] + lens)
    mass = torch.rand((cache.n_pages, hkv, page), generator=g).cuda()
    return cache, table, [(kk[at[b]:at[b + 1]], vv[at[b]:at[b + 1]]) for b in range(len(lens))], mass


@pytest.mark.parametrize("hd,hkv,page", [(128, 8, 64), (128, 1, 16), (64, 2, 16), (64, 3, 128)])
@pytest.mark.parametrize("lens,cut", [([70, 16, 40], 0.5), ([4000, 1, 300, 17], 0.3), ([9000], 0.9)])
@pytest.mark.parametrize("where", ["in place", "elsewhere"])
def test_move(hd, hkv, page, lens, cut, where):
    """Lists of every kind: each head's own, or one for all; behind a start; in place or to other pages."""
    cache, table, held, mass = _filled(lens, hkv, hd, page)
    r = np.random.default_rng(len(lens))
    nan_eq = lambda a, b: torch.equal(torch.nan_to_num(a, nan=1234.0), torch.nan_to_num(b, nan=1234.0))
    for heads, start in ((hkv, [0] * len(lens)), (None, [min(n, 5 + 3 * b) for b, n in enumerate(lens)])):
        cache, table, held, mass = _filled(lens, hkv, hd, page)
        w0 = _paged(mass, table, lens, page)
        count = [int((n - s) * cut) for n, s in zip(lens, start)]
        wide = max(count) + 2
        idx = np.full((len(lens), heads or 1, wide), -1, np.int32)
        for b, (n, s, c) in enumerate(zip(lens, start, count)):
            for h in range(heads or 1):
                idx[b, h, :c] = np.sort(r.choice(n - s, c, replace=False))
                idx[b, h, c:] = 7  # (behind the count: not looked at)
        index = torch.from_numpy(idx if heads else idx[:, 0]).cuda()
        if where == "in place":
            to, ttable = None, table
        else:
            need = [(s + c + page - 1) // page for s, c in zip(start, count)]
            # the same cache with more pages
            from latency_moe_decode_gb300 import ops
            more = ops.KvqCache(cache.n_pages + sum(need), hkv, hd, page_tokens=page)
            more.pages[:cache.n_pages * cache.page_bytes] = cache.pages[:cache.n_pages * cache.page_bytes]
            to = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
            at = cache.n_pages
            for b, n in enumerate(need):
                to[b, :n] = torch.arange(at, at + n)
                at += n
            to = ttable = to.cuda()
            mass = torch.cat([mass, torch.zeros(sum(need), hkv, page, device="cuda")])
            cache = more
        pages0 = cache.pages.clone()
        cache.move(index, _ints(count), table, start=None if sum(start) == 0 else _ints(start), to=to, mass=mass)
        cache.check()
        got = cache.gather(_ints(start), ttable, sum(count), cu_tokens=_cu(count))
        got_w = _paged(mass, ttable, [s + c for s, c in zip(start, count)], page)
        row = 0
        for b, (s, c) in enumerate(zip(start, count)):
            for h in range(hkv):
                src = torch.from_numpy(s + idx[b, h if heads else 0, :c]).long()
                for i in (0, 1):
                    assert nan_eq(got[i][row:row + c, h], held[b][i][src.cuda(), h])
                assert np.array_equal(got_w[b][h, s:s + c], w0[b][h, src.numpy()])
            row += c
        if where == "in place":  # what lies before and behind is untouched
            kk, vv = cache.gather(_ints([0] * len(lens)), table, sum(lens), cu_tokens=_cu(lens))
            at = np.cumsum([0] + lens)
            for b, (s, c) in enumerate(zip(start, count)):
                for x, i in ((kk, 0), (vv, 1)):
                    assert nan_eq(x[at[b]:at[b] + s], held[b][i][:s]) and nan_eq(x[at[b] + s + c:at[b + 1]], held[b][i][s + c:])
        else:  # so are the pages that were read
            n = table.max().item() + 1
            assert torch.equal(cache.pages[:n * cache.page_bytes], pages0[:n * cache.page_bytes])


def test_positions_that_stay_are_not_written():
    """Two sequences share their first pages: lists that leave them as they are do not write them."""
    from latency_moe_decode_gb300.capi import DecError
    cache, table, held, mass = _filled([64, 64], 2, 128, 16)
    table[1, :2] = table[0, :2]
    before = cache.pages.clone()
    idx = torch.stack([torch.cat([torch.arange(32), torch.arange(40, 56)]), torch.cat([torch.arange(32), torch.arange(33, 49)])])
    cache.move(idx.to(torch.int32).cuda(), _ints([48, 48]), table)
    cache.check()
    for p in table[0, :2].tolist():
        assert torch.equal(cache.pages[p * cache.page_bytes:(p + 1) * cache.page_bytes], before[p * cache.page_bytes:(p + 1) * cache.page_bytes])
    # pages, starts and indexes out of range are recorded and skipped; the other sequence moves
    for tab, start, i2, st in ((-5, [0, 0], 40, -1), (None, [0, -1], 40, -1), (None, [0, 0], 10 ** 9, -8), (None, [0, 2 ** 31 - 9], 40, -8)):
        cache, table, held, mass = _filled([64, 64], 2, 128, 16)
        t2 = table.clone()
        if tab is not None:
            t2[1, :] = tab
        cache.move(_ints([[3, 40], [3, i2]]), _ints([2, 2]), t2, start=_ints(start))
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == st
        kk, _ = cache.gather(_ints([0]), table[:1].contiguous(), 2, cu_tokens=_ints([0, 2]))
        assert torch.equal(kk, held[0][0][[3, 40]])


def test_evict_then_decode():
    """A bounded cache in use: steps add their weights, the cache is brought down to its budget, later rows keep their
    rotary positions, and attention over what is left is attention over those positions."""
    from latency_moe_decode_gb300 import ops
    hd, hq, hkv, page, budget = 128, 8, 2, 16, 48
    lens = [90, 30, 61]
    g = torch.Generator().manual_seed(4)
    rope = ops.rope_table(200, hd, 1e4)
    cache, table = _cache([n + 8 for n in lens], hkv, hd, page)
    zero = _ints([0] * 3)
    k, v = _rnd(g, sum(lens), hkv, hd), _rnd(g, sum(lens), hkv, hd)
    cache.append(k.cuda(), v.cuda(), zero, table, cu_tokens=_cu(lens), rope=rope)
    mass, length, position = cache.new_mass(), _ints(lens), _ints(lens)
    history = [[cache.gather(zero, table, sum(lens), cu_tokens=_cu(lens))[i].split(lens)[b] for i in (0, 1)] for b in range(3)]
    history = [[h[0].transpose(0, 1), h[1].transpose(0, 1)] for h in history]  # [hkv, positions, hd]
    for step in range(4):
        q, k1, v1 = _rnd(g, 3, hq, hd), _rnd(g, 3, hkv, hd), _rnd(g, 3, hkv, hd)
        qr = cache.append(k1.cuda(), v1.cuda(), length, table, q=q.cuda(), rope=rope, positions=position)
        k2, v2 = cache.gather(length, table, 3)
        for b in range(3):
            history[b] = [torch.cat([history[b][i], x[b][:, None]], 1) for i, x in ((0, k2), (1, v2))]
        out, lse = cache.attention(qr, length, table, return_lse=True)
        cache.attention_mass(qr, lse, length, table, mass)
        for b in range(3):
            n = history[b][0].shape[1]
            for h in range(hkv):
                rows = slice(h * 4, h * 4 + 4)
                kk, vv = (_np(x[h])[:, None] for x in history[b])
                want, wl, m, big = ref.attend(_np(qr[b, rows]), kk, vv, hd ** -0.5, n)
                ob, lb = ref.out_bounds(want, wl, m, big, hd, n)
                assert (np.abs(_np(out[b, rows]) - want) <= ob).all() and (np.abs(_np(lse[b, rows]) - wl) <= lb).all()
        length, position = length + 1, position + 1
        if step % 2 == 1:
            kept, length = cache.evict(mass, length, table, budget, sinks=2, recent=8)
            for b in range(3):
                n = int(length[b])
                history[b] = [torch.stack([x[h][kept[b, h, :n].long()] for h in range(hkv)]) for x in history[b]]
    cache.check()
    assert length.tolist() == [48, 34, 48]


def test_calls_with_work_in_flight_and_from_graphs():
    """heaviest, move and attention_mass read what earlier work on the stream leaves, and run from a captured graph."""
    cache, table, held, mass = _filled([500, 300], 2, 128, 16)
    other, t2, _, _ = _filled([500, 300], 2, 128, 16)
    m2 = mass.clone()
    kept, count = other.evict(m2, _ints([500, 300]), t2, 100, sinks=3, recent=10)
    s = torch.cuda.Stream()
    ln, tab = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros_like(table)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            big = torch.tanh(big @ big)  # (queued work before the lengths and the table are there)
        ln.copy_(_ints([500, 300]))
        tab.copy_(table)
    k3, c3 = cache.evict(mass, ln, tab, 100, sinks=3, recent=10, stream=s)
    s.synchronize()
    assert torch.equal(k3, kept) and torch.equal(c3, count) and torch.equal(mass, m2)
    a, b = cache.gather(_ints([0, 0]), table, 200, cu_tokens=_ints([0, 100, 200])), other.gather(_ints([0, 0]), t2, 200, cu_tokens=_ints([0, 100, 200]))
    assert all(torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)) for x, y in zip(a, b))
    q = torch.randn(2, 4, 128, device="cuda").to(BF)
    ln2 = _ints([100, 100])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = cache.attention(q, ln2, table, causal=False, return_lse=True)
        cache.attention_mass(q, lse, ln2, table, mass, causal=False)
        kept, count = cache.heaviest(mass, ln2, table, 20)
        cache.move(kept, count, table, mass=mass)
    want_m = m2.clone()
    for _ in range(2):
        mass.copy_(m2)
    g.replay()
    torch.cuda.synchronize()
    _, lse2 = other.attention(q, ln2, t2, causal=False, return_lse=True)
    other.attention_mass(q, lse2, ln2, t2, want_m, causal=False)
    k4, c4 = other.heaviest(want_m, ln2, t2, 20)
    other.move(k4, c4, t2, mass=want_m)
    assert torch.equal(k4, kept) and torch.equal(want_m, mass)


def test_heaviest_of_more_than_a_cta_keeps():
    """Many lists, one CTA each, of more positions than their keys have room for in shared memory (sequences that share
    their pages: nothing is written there)."""
    hkv, page, n, batch, budget = 2, 256, 45001, 90, 3000
    cache, row = _cache([n], hkv, 64, page)
    g = torch.Generator(device="cuda").manual_seed(6)
    mass = torch.rand((cache.n_pages, hkv, page), generator=g, device="cuda")
    mass[torch.rand(mass.shape, generator=g, device="cuda") < 0.3] = 0.25  # ties at what may be the border
    lens = [n - 7 * b for b in range(batch)]
    kept, count = cache.heaviest(mass, _ints(lens), row.expand(batch, -1), budget, sinks=3, recent=50)
    cache.check()
    assert (count == budget).all()
    w = _paged(mass, row, [n], page)[0]
    for b in (0, 1, 40, 89):
        assert np.array_equal(kept[b].cpu().numpy(), _heaviest_want(w[:, :lens[b]], lens[b], budget, 3, 50)), b


def test_pages_beyond_32_bit_offsets():
    """A cache of more than 4 GB (and weights of more than 2^31 bytes / 16): the sequence's pages are its last ones."""
    from latency_moe_decode_gb300 import ops
    hkv, hd, page, n = 8, 128, 64, 300
    each = ops.KvqCache(1, hkv, hd, page).page_bytes
    pages = (2 ** 32 + 2 ** 29) // each + 20
    cache = ops.KvqCache(pages, hkv, hd, page)
    table = torch.arange(pages - 1, pages - 7, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    g = torch.Generator().manual_seed(9)
    k, v, q = _rnd(g, n, hkv, hd), _rnd(g, n, hkv, hd), _rnd(g, n, 2 * hkv, hd)
    cache.append(k.cuda(), v.cuda(), _ints([0]), table, cu_tokens=_ints([0, n]))
    small, t2 = _cache([n], hkv, hd, page)
    small.append(k.cuda(), v.cuda(), _ints([0]), t2, cu_tokens=_ints([0, n]))
    for c, t in ((cache, table), (small, t2)):
        m = c.new_mass()
        for rows in (1, n):  # the kernels for few and for many rows
            _, lse = c.attention(q[:rows].cuda(), _ints([n - rows]), t, cu_tokens=_ints([0, rows]), max_tokens=rows, return_lse=True)
            c.attention_mass(q[:rows].cuda(), lse, _ints([n - rows]), t, m, cu_tokens=_ints([0, rows]), max_tokens=rows)
        kept, count = c.evict(m, _ints([n]), t, 100, sinks=2, recent=9)
        got = (kept, count, *c.gather(_ints([0]), t, 100, cu_tokens=_ints([0, 100])), torch.from_numpy(_paged(m[t[0].long()], torch.arange(t.shape[1])[None], [n], page)[0]))
        c.check()
        if c is cache:
            want = got
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("rows,batch,length", [(1, 16, 8000), (5, 12, 6007), (40, 6, 9001), (150, 3, 20000)])
def test_many_tiles_a_cta(rows, batch, length):
    """The kernel for many rows over long stretches of tiles (its rings wrap many times; queries that stay, and blocks in
    turn), against the one for few rows, a few rows at a time. Both are off the definition by at most what _mass_want
    allows, so they are off each other by twice that."""
    hq, hkv, hd = 32, 8, 128
    lens = [length - 131 * b for b in range(batch)]
    g = torch.Generator(device="cuda").manual_seed(rows)
    n = rows * batch
    cache, table = _cache(lens, hkv, hd, 64)
    for b in range(batch):
        k = torch.randn(lens[b], hkv, hd, generator=g, device="cuda").to(BF)
        cache.append(k, k, _ints([0]), table[b:b + 1], cu_tokens=_ints([0, lens[b]]))
    q = torch.randn(n, hq, hd, generator=g, device="cuda").to(BF)
    _, lse = cache.attention(q, _ints(lens), table, cu_tokens=_cu([rows] * batch), max_tokens=rows, causal=False, return_lse=True)
    was = torch.rand((cache.n_pages, hkv, 64), generator=g, device="cuda")
    many = cache.attention_mass(q, lse, _ints(lens), table, was, cu_tokens=_cu([rows] * batch), max_tokens=max(rows, 5), causal=False,
                                out=torch.zeros_like(was))
    few, step = was.clone(), 4
    for r0 in range(0, rows, step):
        m = min(step, rows - r0)
        pick = torch.cat([torch.arange(b * rows + r0, b * rows + r0 + m) for b in range(batch)]).cuda()
        cache.attention_mass(q[pick], lse[pick], _ints(lens), table, few, cu_tokens=_cu([m] * batch), max_tokens=m, causal=False)
    cache.check()
    # |q| and |k| of 128 normal values: sum |q k| / sqrt(128) below 20 (its mean is 7.2, deviation 0.7), |lse| below 32
    d = hd * 2.0 ** -23 * 20 + 2.0 ** -14 / hd * 20 * 2.0 ** -9 + 2.0 ** -21 * 21 + 2.0 ** -22 * 32
    rel = 2 * (d + 2.0 ** -23 * (rows * 4 + 8) + 2.0 ** -22)
    for a, b in zip(_paged(many, table, lens, 64), _paged(few, table, lens, 64)):
        assert (np.abs(a - b) <= rel * np.abs(b)).all()


def test_more_sequences_than_a_launch_takes():
    """300 sequences: what the calls give does not depend on how they are launched, nor on the other sequences."""
    hq, hkv, hd, batch = 8, 2, 64, 300
    lens = [(37 * b) % 90 for b in range(batch)]
    g = torch.Generator().manual_seed(8)
    t = sum(lens) + batch
    k = _rnd(g, t, hkv, hd).cuda()
    cache, table = _cache([n + 1 for n in lens], hkv, hd, 16)
    cache.append(k, k, _ints([0] * batch), table, cu_tokens=_cu([n + 1 for n in lens]))
    q = _rnd(g, batch, hq, hd).cuda()
    chain = torch.ones(batch, 1, dtype=torch.int32, device="cuda")  # each row sees itself
    out, lse = cache.attention(q, _ints(lens), table, return_lse=True)
    out2, lse2 = cache.attention(q, _ints(lens), table, return_lse=True, tree_mask=chain)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for most in (1, 8):  # the kernels for few and for many rows
        whole, parts = cache.new_mass(), cache.new_mass()
        cache.attention_mass(q, lse, _ints(lens), table, whole, max_tokens=most)
        for b in (slice(0, 7), slice(7, 290), slice(290, 300)):
            cache.attention_mass(q[b], lse[b], _ints(lens[b]), table[b].contiguous(), parts, max_tokens=most)
        assert torch.equal(whole, parts)
    kept, count = cache.heaviest(whole, _ints(lens), table, 20, recent=3)
    for b, w in enumerate(_paged(whole, table, lens, 16)):
        assert np.array_equal(kept[b].cpu().numpy(), _heaviest_want(w, lens[b], 20, 0, 3))
    cache.check()
