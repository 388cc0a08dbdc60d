"""The paged 4-bit KV cache on the GPU (append, gather, attention) against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import kvq_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _cache(lens, hkv, hd, page, seed=0, spare=3):
    """A cache whose pages are handed out in random order to sequences of `lens` positions."""
    from latency_moe_decode_gb300 import ops
    g = np.random.default_rng(seed)
    need = [(n + page - 1) // page for n in lens]
    cache = ops.KvqCache(sum(need) + spare, hkv, hd, page_tokens=page)
    cache.pages.random_(0, 256)  # pages start with anything
    perm = g.permutation(cache.n_pages)
    table = np.full((len(lens), max(1, max(need))), -7, np.int32)  # entries past a sequence are never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return cache, torch.from_numpy(table).cuda()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(new, first=0):
    return _ints(np.concatenate([[first], first + np.cumsum(new)]))


def _np(t):
    return t.detach().double().cpu().numpy()


def _rnd(g, *s, dtype=BF, scale=1.0):
    return (torch.randn(*s, generator=g) * scale).to(dtype)


APPEND = [
    # hd, hq, hkv, page, dtype, norm, rot, interleaved, new tokens, lengths
    (128, 32, 8, 64, BF, True, 128, False, [1], [1000]),
    (128, 8, 2, 16, F32, False, 128, False, [1, 1, 1], [0, 15, 4000]),
    (128, 4, 4, 32, BF, True, 64, True, [5, 1, 33, 16], [0, 31, 17, 100]),
    (128, 3, 1, 128, F32, True, 16, False, [130], [127]),
    (64, 4, 2, 16, BF, True, 64, False, [7, 2, 40], [3, 14, 0]),
    (64, 6, 3, 256, F32, True, 32, True, [1, 300], [255, 1]),
    (64, 2, 1, 64, BF, False, 0, False, [65, 1], [0, 63]),
    (64, 8, 8, 16, BF, False, 16, False, [3], [9]),
]


@pytest.mark.parametrize("hd,hq,hkv,page,dtype,norm,rot,inter,new,lens", APPEND)
def test_append_and_gather(hd, hq, hkv, page, dtype, norm, rot, inter, new, lens):
    from latency_moe_decode_gb300 import ops
    g = torch.Generator().manual_seed(hd + hq + page)
    n = sum(new)
    q, k, v = (_rnd(g, n, h, hd, dtype=dtype) for h in (hq, hkv, hkv))
    k[0, 0, :16] = 0            # an empty run
    v[-1, -1, -16:] *= 1e-4     # scales at the bottom
    qn, kn = ((1 + 0.2 * torch.randn(hd, generator=g)).to(BF) for _ in range(2)) if norm else (None, None)
    pos = np.concatenate([np.arange(l, l + m) for l, m in zip(lens, new)])
    rope = ops.rope_table(int(pos.max()) + 1, rot, 1e4) if rot else None
    cache, table = _cache([a + b for a, b in zip(new, lens)], hkv, hd, page)
    before = cache.pages.clone()
    cu, ln = _cu(new), _ints(lens)
    dev = lambda t: None if t is None else t.cuda()
    qo = cache.append(dev(k), dev(v), ln, table, cu_tokens=cu, q=dev(q), q_norm=dev(qn), k_norm=dev(kn), rope=rope,
                      interleaved=inter)
    gk, gv = (_np(t) for t in cache.gather(ln, table, n, cu_tokens=cu))
    cache.check()
    # values go in as they are: codes and scales are decided exactly
    assert np.array_equal(gv, ref.store(_np(v))[0])
    tab = None if rope is None else _np(rope)
    # norm: the sum of hd squares in fp32 and three more roundings; rotation: two products and a sum
    for x, w, got, bits in ((q, qn, _np(qo), 2.0 ** -8), (k, kn, gk, None)):
        want = ref.norm_rotate(_np(x), None if w is None else _np(w), 1e-6, tab, pos, inter)
        size = np.abs(ref.norm_rotate(_np(x), None if w is None else _np(w), 1e-6, None, pos, inter))
        size = np.maximum(np.abs(want), np.broadcast_to(size.max(-1, keepdims=True), size.shape))
        eps = size * (2.0 ** -24 * (16 if w is not None else 4))
        if bits:
            assert (np.abs(got - want) <= bits * np.abs(want) + eps).all()
        else:
            held, s = ref.store(want)
            same = held == got
            # a value whose fp32 form falls on the other side of a border is held one step away
            assert same.mean() > 0.999 or (~same).sum() <= 2
            assert (np.abs(got - want) <= np.where(s > 2.0 ** -11, 0.5 * s * 1.125, 2.0 ** -11) + eps).all()
    # nothing but the appended positions has changed
    cache.gather(ln, table, n, cu_tokens=cu)
    changed = (before != cache.pages).nonzero().numel()
    assert changed <= n * hkv * 2 * (hd // 2 + hd // 16)


@pytest.mark.parametrize("hd,dtype,norm,rot,inter", [(128, BF, True, 128, False), (128, F32, True, 64, True),
                                                     (64, BF, False, 64, False), (64, F32, False, 0, False)])
def test_codes_are_those_of_the_formula(hd, dtype, norm, rot, inter):
    """Millions of values, so that some fall within fp32's error of the border between two codes or scales: every
    one is held as the formula in 64 bits says. (An empty row and one with a NaN among them.)"""
    from latency_moe_decode_gb300 import ops
    n, hkv = 2 ** 18 // hd, 8
    g = torch.Generator().manual_seed(hd)
    k, v = (_rnd(g, n, hkv, hd, dtype=dtype, scale=2.0) for _ in range(2))
    k[3, 1], v[5, 2, 20] = 0, float("nan")
    k[7, 3, 1] *= 1e4
    kn = (1 + 0.2 * torch.randn(hd, generator=g)).to(BF) if norm else None
    rope = ops.rope_table(n, rot, 1e6) if rot else None
    cache, table = _cache([n], hkv, hd, 64)
    cache.append(k.cuda(), v.cuda(), _ints([0]), table, cu_tokens=_cu([n]), k_norm=None if kn is None else kn.cuda(),
                 rope=rope, interleaved=inter)
    gk, gv = (_np(t) for t in cache.gather(_ints([0]), table, n, cu_tokens=_cu([n])))
    cache.check()
    want = ref.norm_rotate(_np(k), None if kn is None else _np(kn), 1e-6, None if rope is None else _np(rope), np.arange(n),
                           inter)
    for got, x in ((gk, want), (gv, _np(v))):
        held = ref.store(x)[0]
        wrong = ~((got == held) | (np.isnan(got) & np.isnan(held)))
        assert not wrong.any(), (wrong.sum(), got[wrong][:4], held[wrong][:4])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_on_the_border_between_codes(hd, dtype):
    """Keys (rotated by nothing: cos 1, sin 0) and values with runs on a middle between two codes, or between two
    scales, and just beside it, next to runs of zeros, tiny ones, NaNs and infinities."""
    n, hkv = 64, 40
    x = torch.zeros(n, hkv, hd)
    x[..., :16] = (torch.arange(16) - 7.5).clamp(-6.5, 6.5)
    x[..., 15] = 7
    x[:, ::2, 5] = 7 * 17 / 16              # between scales 1 and 1.125
    x[:, ::3, 16 + 3] = float("nan")
    x[:, 1::3, 32:48] = 2.0 ** -15 * torch.arange(16)
    x[:, 2::5, -1] = float("inf")
    x[:, 1::5, -2] = -1e5
    if dtype == F32:
        step = torch.arange(n)[:, None, None] - n // 2
        x[..., :16] *= 1 + 2.0 ** -23 * step
    x = x.to(dtype)
    rope = torch.tensor([1.0, 0.0]).repeat(n, hd // 2, 1).cuda()
    cache, table = _cache([n], hkv, hd, 16)
    cache.append(x.cuda(), x.cuda(), _ints([0]), table, cu_tokens=_cu([n]), rope=rope)
    with np.errstate(invalid="ignore"):  # (0 times what is not finite)
        turned = ref.norm_rotate(_np(x), None, 0.0, _np(rope), np.arange(n), False)
    for got, want in zip(cache.gather(_ints([0]), table, n, cu_tokens=_cu([n])), (turned, _np(x))):
        assert np.array_equal(_np(got), ref.store(want)[0], equal_nan=True)
    cache.check()


def test_append_takes_strides_and_leaves_other_rows():
    """q, k, v as slices of one projection, q_out a slice of a wider buffer, rows before the first and
    behind the last sequence, an empty sequence between two."""
    hd, hq, hkv, page = 128, 8, 2, 16
    g = torch.Generator().manual_seed(5)
    new, lens, first, n = [3, 0, 4], [14, 9, 0], 2, 12
    qkv = _rnd(g, n, hq + 2 * hkv, hd).cuda()
    qkv[0], qkv[-1] = float("nan"), float("inf")  # rows of no sequence
    cache, table = _cache([20, 20, 20], hkv, hd, page)
    before = cache.pages.clone()
    wide = torch.full((n, hq + 2, hd), 7.0, dtype=BF, device="cuda")
    args = (qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], _ints(lens), table)
    out = cache.append(*args, cu_tokens=_cu(new, first), q=qkv[:, :hq], q_out=wide[:, 1:-1])
    assert out.data_ptr() == wide[:, 1:-1].data_ptr()
    cache.check()
    live = slice(first, first + sum(new))
    assert torch.equal(wide[live, 1:-1], qkv[live, :hq])
    rest = torch.ones(n, dtype=torch.bool)
    rest[live] = False
    assert (wide[rest.cuda()] == 7).all() and (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()
    k, v = (torch.full((n, hkv, hd), -3.0, dtype=BF, device="cuda") for _ in range(2))
    cache.gather(_ints(lens), table, n, cu_tokens=_cu(new, first), out=(k, v))
    assert (k[rest.cuda()] == -3).all() and (v[rest.cuda()] == -3).all()
    assert np.array_equal(_np(k)[live], ref.store(_np(qkv[live, hq:hq + hkv]))[0])
    assert np.array_equal(_np(v)[live], ref.store(_np(qkv[live, hq + hkv:]))[0])
    assert (before != cache.pages).sum() <= 7 * hkv * 2 * (hd // 2 + hd // 16)
    # the same through a q that is its own output, and head-major keys
    k2 = qkv[:, hq:hq + hkv].transpose(0, 1).contiguous().transpose(0, 1)
    q2 = qkv[:, :hq].clone()
    pages = cache.pages.clone()
    cache.append(k2, args[1], _ints(lens), table, cu_tokens=_cu(new, first), q=q2, q_out=q2)
    assert torch.equal(pages, cache.pages) and torch.equal(q2[live], qkv[live, :hq])


def test_runs_that_are_not_finite_or_out_of_range():
    hd = 64
    x = torch.zeros(5, 1, hd)
    x[0, 0, 3] = float("nan")
    x[1, 0, 20] = float("-inf")
    x[2, 0, 40] = 1e6          # above the largest scale: held as the largest value there is
    x[3, 0, :16] = 2.0 ** -15  # below half the smallest scale times 7
    x[4, 0] = torch.linspace(-3360, 3360, hd)
    cache, table = _cache([5], 1, hd, 16)
    ln, cu = _ints([0]), _cu([5])
    cache.append(x.cuda(), x.cuda(), ln, table, cu_tokens=cu)
    for got in cache.gather(ln, table, 5, cu_tokens=cu):
        got = _np(got)
        want = ref.store(_np(x))[0]
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))
        assert np.isnan(got[0, 0, :16]).all() and (got[0, 0, 16:] == 0).all() and got[2, 0, 40] == 7 * 480


ATTN = [
    # hd, hq, hkv, page, causal, new tokens, lengths
    (128, 4, 1, 64, True, [1], [0]),
    (128, 32, 8, 64, True, [1], [1023]),
    (128, 8, 2, 16, True, [1, 1, 1, 1], [15, 16, 63, 300]),
    (128, 8, 8, 32, True, [1, 1], [5000, 2]),
    (128, 16, 2, 128, True, [8, 3, 1], [700, 0, 64]),
    (128, 12, 4, 64, False, [1, 2, 1], [0, 129, 1]),
    (128, 8, 2, 64, True, [40, 17], [33, 200]),
    (128, 64, 2, 16, True, [3], [50]),
    (64, 4, 2, 16, True, [1, 1], [0, 77]),
    (64, 4, 2, 64, False, [5, 1, 4], [0, 1, 301]),
    (64, 8, 1, 256, True, [9], [250]),
    (64, 3, 3, 32, True, [70], [0]),
    # more query rows than a stretch of the kernel for prompts, parts of tiles, several CTAs a unit
    (128, 8, 2, 16, True, [200, 1, 33], [700, 0, 2000]),
    (128, 4, 1, 64, True, [16], [127]),
    (128, 4, 4, 32, True, [129, 64], [0, 128]),
    (64, 8, 2, 64, False, [64, 40, 3], [0, 500, 129]),
    (64, 2, 1, 16, True, [300], [40]),
    (128, 16, 1, 256, False, [9, 2], [1, 1000]),
    # rows about which another kernel takes the call
    (128, 8, 2, 64, True, [2, 1], [30, 7]),
    (128, 8, 2, 64, True, [3, 2], [200, 31]),
    (128, 8, 2, 32, True, [4, 1], [127, 600]),
    (128, 8, 2, 32, True, [5, 1, 0, 2], [127, 600, 3, 0]),
    (64, 8, 2, 64, True, [8, 3], [500, 1]),
    (64, 8, 2, 64, True, [9, 3], [500, 1]),
    # prompts whose sequences see nothing
    (128, 4, 1, 16, False, [30, 20, 10], [0, 0, 0]),
    (64, 4, 1, 16, False, [30, 1, 10], [0, 9, 0]),
]


def _filled(lens, hkv, hd, page, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    cache, table = _cache(lens, hkv, hd, page, seed)
    k, v = (_rnd(g, max(1, sum(lens)), hkv, hd, scale=s) for s in (spread, 1.0))
    if sum(lens):
        cache.append(k.cuda(), v.cuda(), _ints([0] * len(lens)), table, cu_tokens=_cu(lens))
    return cache, table, ref.store(_np(k))[0], ref.store(_np(v))[0], g


def _check(out, lse, q, k, v, new, lens, causal, scale, hd, first=0):
    """Every row of out and lse against the 64-bit form over the values the cache holds."""
    at, row = 0, first
    for m, l in zip(new, lens):
        held = l + m if causal else l
        for j in range(m):
            seen = l + j + 1 if causal else l
            # (the kernel for prompts, from this many query rows on, keeps probabilities down to 2^-21)
            kept = 2.0 ** (-21 if max(new) * q.shape[1] // k.shape[1] > (16 if hd == 128 else 32) else -29)
            o, s, mass, big = ref.attend(q[row], k[at:at + held], v[at:at + held], scale, seen, kept)
            ob, lb = ref.out_bounds(o, s, mass, big, hd, max(seen, 1))
            assert (np.abs(out[row] - o) <= ob).all(), (row, np.max(np.abs(out[row] - o) / ob))
            if seen <= 0:
                assert (lse[row] == -np.inf).all() and (out[row] == 0).all()
            else:
                assert (np.abs(lse[row] - s) <= lb).all(), (row, np.max(np.abs(lse[row] - s) / lb))
            row += 1
        at += held


@pytest.mark.parametrize("hd,hq,hkv,page,causal,new,lens", ATTN)
@pytest.mark.parametrize("spread", [1.0, 12.0], ids=["flat", "peaked"])
def test_attention(hd, hq, hkv, page, causal, new, lens, spread):
    held = [l + m if causal else l for l, m in zip(lens, new)]
    cache, table, k, v, g = _filled(held, hkv, hd, page, hq + page, spread)
    q = _rnd(g, sum(new), hq, hd)
    out, lse = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(new), max_tokens=max(new), causal=causal,
                               return_lse=True)
    cache.check()
    _check(_np(out), _np(lse), _np(q), k, v, new, lens, causal, hd ** -0.5, hd)


def test_attention_one_row_per_sequence_without_cu():
    lens = [0, 1, 40, 129, 1000]
    cache, table, k, v, g = _filled([l + 1 for l in lens], 2, 128, 64, 3)
    q = _rnd(g, 5, 8, 128)
    out, lse = cache.attention(q.cuda(), _ints(lens), table, scale=0.05, return_lse=True)
    cache.check()
    _check(_np(out), _np(lse), _np(q), k, v, [1] * 5, lens, True, 0.05, 128)


def test_attention_leaves_rows_of_no_sequence_and_takes_strides():
    new, lens, first, n = [2, 0, 3], [30, 8, 100], 1, 9
    cache, table, k, v, g = _filled([l + m for l, m in zip(lens, new)], 2, 64, 16, 4)
    q = _rnd(g, n, 8, 64).cuda()
    q[0], q[-1] = float("nan"), float("nan")
    wide = torch.full((n, 12, 64), 5.0, dtype=BF, device="cuda")
    wide[:, 2:10] = q
    out = torch.full((n, 10, 64), 5.0, dtype=BF, device="cuda")
    got = cache.attention(wide[:, 2:10], _ints(lens), table, cu_tokens=_cu(new, first), max_tokens=3, out=out[:, 1:9])
    cache.check()
    at, row = 0, first
    for m, l in zip(new, lens):
        for j in range(m):
            o, s, mass, big = ref.attend(_np(q[row]), k[at:at + l + m], v[at:at + l + m], 0.125, l + j + 1)
            assert (np.abs(_np(got[row]) - o) <= ref.out_bounds(o, s, mass, big, 64, l + j + 1)[0]).all()
            row += 1
        at += l + m
    assert (out[0] == 5).all() and (out[row:] == 5).all() and (out[:, 0] == 5).all() and (out[:, 9] == 5).all()


def test_attention_ignores_what_lies_behind_a_sequence():
    """Positions behind the last one, in the same group and page, hold NaN scales and any codes."""
    for hd, hkv, page, ln in ((128, 2, 64, 17), (64, 1, 16, 5), (128, 1, 256, 200)):
        cache, table, k, v, g = _filled([ln + 1], hkv, hd, page, 11)
        bad = torch.full((10, hkv, hd), float("nan"), dtype=BF, device="cuda")
        room = min(10, table.shape[1] * page - ln - 1)
        cache.append(bad[:room], bad[:room], _ints([ln + 1]), table, cu_tokens=_cu([room]))
        q = _rnd(g, 1, 4 * hkv, hd)
        out, lse = cache.attention(q.cuda(), _ints([ln]), table, return_lse=True)
        cache.check()
        _check(_np(out), _np(lse), _np(q), k, v, [1], [ln], True, hd ** -0.5, hd)


def test_a_nan_reaches_only_its_own_heads():
    cache, table, k, v, g = _filled([100], 2, 128, 64, 12)
    q = _rnd(g, 1, 8, 128).cuda()
    good = cache.attention(q, _ints([99]), table)
    q2 = q.clone()
    q2[0, 1, 5] = float("nan")
    out = cache.attention(q2, _ints([99]), table)
    assert torch.isnan(out[0, 1]).all()
    keep = [h for h in range(8) if h != 1]
    assert torch.equal(out[0, keep], good[0, keep])
    bad = torch.zeros(1, 2, 128, dtype=BF, device="cuda")
    bad[0, 0, 3] = float("inf")
    cache.append(bad, bad, _ints([50]), table)
    out = cache.attention(q, _ints([99]), table)
    assert torch.isnan(out[0, :4]).any(-1).all() and torch.equal(torch.isnan(out[0, 4:]).any(), torch.tensor(False, device="cuda"))


@pytest.mark.parametrize("hd,hq,m", [(128, 8, 4), (64, 4, 8), (128, 4, 20)])
def test_a_nan_value_reaches_only_rows_that_see_it(hd, hq, m):
    """Token 2's key and value hold a NaN: the rows of tokens 0 and 1 are as if it were not there, and
    later rows get it where their own formula puts it."""
    cache, table, k, v, g = _filled([21 + m], 1, hd, 16, 13)
    q = _rnd(g, m, hq, hd).cuda()
    ln, cu = _ints([20]), _cu([m])
    good = cache.attention(q, ln, table, cu_tokens=cu, max_tokens=m)
    gk, gv = cache.gather(_ints([22]), table, 1)
    bad = gv.clone()
    bad[0, 0, 17] = float("nan")
    cache.append(gk, bad, _ints([22]), table)
    out = cache.attention(q, ln, table, cu_tokens=cu, max_tokens=m)
    assert torch.equal(out[:2], good[:2])
    nan = torch.isnan(out[2:])
    assert nan[..., 16:32].all() and not nan[..., :16].any() and not nan[..., 32:].any()  # the value's run
    bad = gk.clone()
    bad[0, 0, 0] = float("nan")
    cache.append(bad, gv, _ints([22]), table)
    out = cache.attention(q, ln, table, cu_tokens=cu, max_tokens=m)
    assert torch.equal(out[:2], good[:2]) and torch.isnan(out[2:]).all()


def test_attention_over_many_sequences():
    """More sequences than one launch lists, most of them empty or short."""
    b = 4500
    lens = [(i * 7) % 5 for i in range(b)]
    lens[2047], lens[2048], lens[4499] = 70, 130, 33
    cache, table, k, v, g = _filled([l + 1 for l in lens], 1, 64, 16, 14)
    q = _rnd(g, b, 2, 64)
    out, lse = cache.attention(q.cuda(), _ints(lens), table, return_lse=True)
    two = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu([1] * b), max_tokens=1)
    cache.check()
    assert torch.equal(out, two)
    _check(_np(out), _np(lse), _np(q), k, v, [1] * b, lens, True, 0.125, 64)


def test_append_then_attend_as_a_model_does():
    """Prompt, then single tokens, then a verify step of three, each appended with norm and rotation
    and attended to; the reference keeps the rows in 64 bits and stores them the same way."""
    from latency_moe_decode_gb300 import ops
    hd, hq, hkv, page = 128, 8, 2, 16
    g = torch.Generator().manual_seed(21)
    cache, table = _cache([80, 80], hkv, hd, page)
    rope = ops.rope_table(80, hd, 1e6)
    qn, kn = ((1 + 0.1 * torch.randn(hd, generator=g)).to(BF) for _ in range(2))
    hist = [[np.zeros((0, hkv, hd))] * 2, [np.zeros((0, hkv, hd))] * 2]
    lens = [0, 0]
    for new in ([33, 7], [1, 1], [1, 1], [3, 3]):
        n = sum(new)
        q, k, v = (_rnd(g, n, h, hd) for h in (hq, hkv, hkv))
        ln, cu = _ints(lens), _cu(new)
        qo = cache.append(k.cuda(), v.cuda(), ln, table, cu_tokens=cu, q=q.cuda(), q_norm=qn.cuda(), k_norm=kn.cuda(),
                          rope=rope)
        out, lse = cache.attention(qo, ln, table, cu_tokens=cu, max_tokens=max(new), return_lse=True)
        gk, gv = (_np(t) for t in cache.gather(ln, table, n, cu_tokens=cu))
        at = 0
        for b, m in enumerate(new):  # the values held are checked above: attention sees them as they are
            hist[b] = [np.concatenate([hist[b][0], gk[at:at + m]]), np.concatenate([hist[b][1], gv[at:at + m]])]
            at += m
        _check(_np(out), _np(lse), _np(qo), np.concatenate([h[0] for h in hist]), np.concatenate([h[1] for h in hist]),
               new, lens, True, hd ** -0.5, hd)
        lens = [l + m for l, m in zip(lens, new)]
    cache.check()


def test_captured_and_replayed_on_another_stream():
    lens = [70, 5]
    cache, table, k, v, g = _filled([80, 80], 2, 128, 16, 31)
    q = _rnd(g, 2, 8, 128).cuda()
    kv = _rnd(g, 2, 2, 128).cuda()
    ln = _ints(lens)
    cache.append(kv, kv, ln, table)
    want = cache.attention(q, ln, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cache.append(kv, kv, ln, table)
        out = cache.attention(q, ln, table)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    ln += 1  # the graph reads lengths from the device
    kv.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    moved = out.clone()
    cache.append(kv, kv, ln, table)
    assert torch.equal(moved, cache.attention(q, ln, table))
    with torch.cuda.stream(s):
        other = cache.attention(q, ln, table)
    named = cache.attention(q, ln, table, stream=s)
    raw = cache.attention(q, ln, table, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(other, moved) and torch.equal(named, moved) and torch.equal(raw, moved)


def test_two_streams_at_once_and_repeats_agree():
    cache, table, k, v, g = _filled([3000, 20], 2, 128, 64, 41)
    q = _rnd(g, 2, 8, 128).cuda()
    ln = _ints([2999, 19])
    want = cache.attention(q, ln, table, return_lse=True)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        for s in (a, b):
            with torch.cuda.stream(s):
                got.append(cache.attention(q, ln, table, return_lse=True))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in got)


@pytest.mark.parametrize("m", [1, 3, 30])
def test_pages_beyond_four_gigabytes(m):
    """Pages at the end of a pool of 5.9 GB hold and give what pages at the start of a small one do."""
    from latency_moe_decode_gb300 import ops
    g = torch.Generator().manual_seed(71)
    hkv, hq, hd, page, lens = 8, 32, 128, 256, [700, 3]
    far = ops.KvqCache(20000, hkv, hd, page)
    near = ops.KvqCache(6, hkv, hd, page)
    tables = _ints([[19999, 14570, 19998], [19997, 14569, 14568]]), _ints([[0, 1, 2], [3, 4, 5]])
    k, v = (_rnd(g, sum(lens), hkv, hd).cuda() for _ in range(2))
    kn, vn = (_rnd(g, 2 * m, hkv, hd).cuda() for _ in range(2))
    q = _rnd(g, 2 * m, hq, hd).cuda()
    got = []
    for cache, table in zip((far, near), tables):
        cache.append(k, v, _ints([0, 0]), table, cu_tokens=_cu(lens))
        cache.append(kn, vn, _ints(lens), table, cu_tokens=_cu([m, m]))
        got.append((*cache.attention(q, _ints(lens), table, cu_tokens=_cu([m, m]), max_tokens=m, return_lse=True),
                    *cache.gather(_ints([0, 0]), table, sum(lens), cu_tokens=_cu(lens))))
        cache.check()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][0].abs().sum() > 0


def _prompts(m, hd=128, hq=8, hkv=2, seed=61):
    """Three sequences of m, 1 and 2 m new tokens, which each of the kernels takes for some m."""
    new, lens = [m, 1, 2 * m], [300, 20, 0]
    cache, table, k, v, g = _filled([l + n for l, n in zip(lens, new)], hkv, hd, 16, seed)
    q = _rnd(g, sum(new), hq, hd).cuda()
    return cache, table, q, dict(lengths=_ints(lens), table=table, cu_tokens=_cu(new), max_tokens=2 * m)


@pytest.mark.parametrize("m", [1, 2, 25])
def test_streams_graphs_and_outputs_over_the_queries_agree(m):
    cache, table, q, kw = _prompts(m)
    want = cache.attention(q, return_lse=True, **kw)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(8):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(cache.attention(q, return_lse=True, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in got)
    graph, held = torch.cuda.CUDAGraph(), q.clone()
    with torch.cuda.graph(graph):
        cache.attention(held, out=held, **kw)  # (capture does not run it)
        twice = cache.attention(q, **kw)
    for _ in range(3):
        held.copy_(q)
        graph.replay()
        assert torch.equal(held, want[0]) and torch.equal(twice, want[0])
    cache.check()


@pytest.mark.parametrize("m", [2, 4, 25])
def test_rows_beyond_max_tokens_are_left(m):
    cache, table, q, kw = _prompts(m)
    want = cache.attention(q, **kw)
    out = torch.full_like(q, 3.0)
    cache.attention(q, out=out, **{**kw, "max_tokens": m})
    assert (out[2 * m + 1:] == 3.0).all()
    # (another bound may choose another kernel. Values up to 4.5; probabilities to 2^-11 of themselves and
    # their sum, outputs to 2^-8: 2 (2 4.5 2^-11 + 4.5 2^-8) = 0.044)
    assert (out[:2 * m + 1].float() - want[:2 * m + 1].float()).abs().max() < 0.05
    cache.check()


def test_prompts_of_many_sequences():
    """More sequences than one launch of the kernel for prompts lists, some without rows."""
    b = 300
    new, lens = [(i * 5) % 7 for i in range(b)], [(i * 11) % 40 for i in range(b)]
    cache, table, k, v, g = _filled([l + n for l, n in zip(lens, new)], 1, 128, 16, 62)
    q = _rnd(g, sum(new), 4, 128)
    out, lse = cache.attention(q.cuda(), _ints(lens), table, cu_tokens=_cu(new), max_tokens=6, return_lse=True)
    cache.check()
    _check(_np(out), _np(lse), _np(q), k, v, new, lens, True, 128 ** -0.5, 128)


def test_bad_pages_of_a_prompt_are_reported():
    from latency_moe_decode_gb300.capi import DecError
    cache, table, q, kw = _prompts(25)
    want = cache.attention(q, **kw)
    wrong = table.clone()
    wrong[0, 3], wrong[0, 7] = cache.n_pages, -5
    for bad, code in ((dict(table=wrong), -1), (dict(lengths=_ints([300, 20, 2 ** 31 - 60])), -8),
                      (dict(lengths=_ints([-3, 20, 0])), -1), (dict(table=table[:, :2]), -8)):
        out = cache.attention(q, **{**kw, **bad})
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == code
        if "table" in bad and bad["table"] is wrong:
            assert torch.equal(out[25:], want[25:])  # the other sequences'
    assert torch.equal(cache.attention(q, **kw), want)
    cache.check()


def test_bad_device_data_is_reported_and_touches_nothing():
    from latency_moe_decode_gb300.capi import DecError
    cache, table, k, v, g = _filled([100, 40], 2, 128, 16, 51)
    q, kv = _rnd(g, 2, 8, 128).cuda(), _rnd(g, 2, 2, 128).cuda()
    pages = cache.pages.clone()
    wrong = table.clone()
    wrong[0, 6] = cache.n_pages
    wrong[1, 2] = -1

    def fails(code, f):
        f()
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == code
        cache.check()  # reported once

    fails(-1, lambda: cache.append(kv, kv, _ints([100, 40]), wrong))
    fails(-1, lambda: cache.gather(_ints([100, 40]), wrong, 2))
    fails(-1, lambda: cache.attention(q, _ints([100, 40]), wrong))
    fails(-8, lambda: cache.append(kv, kv, _ints([table.shape[1] * 16, 2 ** 31 - 1]), table))
    fails(-8, lambda: cache.attention(q, _ints([table.shape[1] * 16 + 5, 2 ** 31 - 1]), table))
    fails(-1, lambda: cache.append(kv, kv, _ints([-1, -5]), table))
    fails(-1, lambda: cache.attention(q, _ints([-1, -5]), table))
    from latency_moe_decode_gb300 import ops
    short = ops.rope_table(10, 128, 1e4)
    fails(-8, lambda: cache.append(kv[:0].new_zeros(2, 2, 128), kv, _ints([10, 11]), table, rope=short, q=q))
    assert (cache.pages != pages).sum() <= 2 * 2 * 2 * 72 + 144  # (values, which are not rotated, may be written)


def test_refusals():
    from latency_moe_decode_gb300 import ops
    from latency_moe_decode_gb300.capi import DecError
    cache, table = _cache([10], 2, 128, 16)
    ln = _ints([0])
    kv, q = torch.zeros(1, 2, 128, dtype=BF, device="cuda"), torch.zeros(1, 8, 128, dtype=BF, device="cuda")
    for bad in (dict(k=kv.half(), v=kv.half()), dict(v=kv.float()), dict(k=kv[:, :1]), dict(k=kv[..., :64]),
                dict(k=kv.cpu()), dict(lengths=ln.long()), dict(lengths=ln.cpu()), dict(table=table.long()),
                dict(table=table[0]), dict(cu_tokens=_ints([0])), dict(q=q, q_norm=torch.ones(128, device="cuda")),
                dict(q=q, q_out=torch.zeros(1, 8, 128, device="cuda")), dict(rope=torch.zeros(4, 64, device="cuda")),
                dict(k=kv.repeat(2, 1, 1), v=kv.repeat(2, 1, 1))):
        with pytest.raises((ValueError, DecError)):
            cache.append(**{**dict(k=kv, v=kv, lengths=ln, table=table), **bad})
    with pytest.raises(DecError):
        cache.append(kv, kv, ln, table, rope=torch.zeros(4, 12, 2, device="cuda"))  # rotary_dim 24
    with pytest.raises(DecError):
        cache.attention(q[:, :3], ln, table)
    for bad in (dict(q=q.float()), dict(q=q, scale=-1.0), dict(q=q, out=q[:, :4])):
        with pytest.raises((ValueError, DecError)):
            cache.attention(lengths=ln, table=table, **bad)
    with pytest.raises(DecError):
        ops.KvqCache(4, 2, 96)
    with pytest.raises(DecError):
        ops.KvqCache(4, 2, 128, page_tokens=48)
    with pytest.raises(ValueError):
        ops.KvqCache(4, 2, 128, pages=torch.empty(10, dtype=torch.uint8, device="cuda"))
    # nothing to do is no error
    none = torch.zeros(0, 2, 128, dtype=BF, device="cuda")
    cache.append(none, none, _ints([]), table[:0])
    assert cache.attention(none, _ints([]), table[:0]).shape == (0, 2, 128)
    cache.check()
