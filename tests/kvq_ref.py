"""Plain 64-bit forms of the paged 4-bit cache's arithmetic, for the tests. numpy, one row at a time
where that is the plainest; shares nothing with the kernels."""
import numpy as np

# the scales there are: 8 * (mantissa of 3 bits) * 2^e, steps of 2^-14 at the bottom
SCALES = np.array([8.0 * (m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 15) for e in range(21) for m in range(8)])


def scale_of(amax):
    """Nearest scale to amax / 7, ties to the even mantissa."""
    want = np.asarray(amax, np.float64) / 7
    hi = np.clip(np.searchsorted(SCALES, want), 1, len(SCALES) - 1)
    lo = hi - 1
    a, b = want - SCALES[lo], SCALES[hi] - want
    return SCALES[np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)]


def store(x):
    """(values held, scale of every value) for rows x [..., hd]."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 16)
    amax = np.abs(b).max(-1)
    fine = np.isfinite(amax)
    s = np.broadcast_to(scale_of(np.where(fine, amax, 0))[..., None], b.shape)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.clip(np.rint(b / s), -8, 7), 0.0)
    c = np.where(fine[..., None], c * s, np.nan)
    return c.reshape(x.shape), s.reshape(x.shape)


def norm_rotate(x, w, eps, table, pos, interleaved):
    """x [n, heads, hd] float64; table [positions, rot / 2, 2] or None."""
    x = np.array(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    if table is not None:
        half = table.shape[1]
        c, s = (np.asarray(table[pos], np.float64)[..., i][:, None] for i in (0, 1))
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = xa * c - xb * s, xa * s + xb * c
    return x


def attend(q, k, v, scale, seen, kept=2.0 ** -29):
    """q [hq, hd], k, v [positions, hkv, hd]: out, lse, and per (head, d) what sizes the error bounds:
    sum_p p |v| + kept sum_p |v| / sum_p e^(s - max) (out_bounds takes 2^-11 of it) and max over the
    seen positions of scale * sum_d |q k|."""
    hq, hd = q.shape
    out, lse = np.zeros((hq, hd)), np.full(hq, -np.inf)
    mass, big = np.zeros((hq, hd)), np.zeros(hq)
    if seen <= 0:
        return out, lse, mass, big
    group = hq // k.shape[1]
    for h in range(hq):
        kk, vv = k[:seen, h // group], v[:seen, h // group]
        s = kk @ q[h] * scale
        m = s.max()
        e = np.exp(s - m)
        p = e / e.sum()
        out[h], lse[h] = p @ vv, m + np.log(e.sum())
        mass[h] = p @ np.abs(vv) + kept * np.abs(vv).sum(0) / e.sum()
        big[h] = (np.abs(kk) @ np.abs(q[h])).max() * scale
    return out, lse, mass, big


def out_bounds(out, lse, mass, big, hd, seen):
    """Bounds of the kernel's error. A score is a sum of hd exact products in fp32: off by at most
    d = hd 2^-23 big (an fp32 accumulator may truncate: a whole step, 2^-23, per addition) plus the
    queries' 2^-25 of the row's largest |q| (below big 2^-14 / hd), plus the exponent's own rounding,
    2^-22 big. Every probability is then off by a factor e^(2 d'), rounds to 11 bits and sums in fp32
    over `seen` terms; the output rounds to bf16. Rounding to 11 bits is 2^-11 of a term as long as f16
    has them: terms e^(s - max) are kept times 2^15, and f16's subnormal step is 2^-24, so a term is off
    by half a step, 2^-25 / 2^15 = 2^-40 (of the largest term, 1, before the division by the sum), at
    least; times |v| and summed that is 2^-11 of `mass`'s second part, 2^-29 sum |v| / sum e^(s - max).
    The kernel for prompts (calls of many query rows) keeps terms times 2^7 and lets the maximum lead its
    reference by 2^8, so the largest term is kept as 2^7 at least: 2^-25 / 2^7 = 2^-32, kept = 2^-21."""
    d = hd * 2.0 ** -23 * big + 2.0 ** -14 / hd * big * 2.0 ** -9 + 2.0 ** -21 * (big + 1)
    n = 2.0 ** -23 * (np.sqrt(seen) * 8 + 32)
    ob = 2.0 ** -8 * np.abs(out) + mass * (2.0 ** -11 + 2 * d[:, None] + n) + 1e-30
    lb = d + n + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0) + 1e-30
    return ob, lb
