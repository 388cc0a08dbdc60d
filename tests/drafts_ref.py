"""Plain 64-bit forms of draft trees and their verification, for the tests. numpy, one row at a time; shares nothing
with the kernels."""
import numpy as np


def random_parents(g, n, width):
    """Row 0 a root, every other row's parent one of the `width` rows before it."""
    return [-1] + [int(g.integers(max(0, j - width), j)) for j in range(1, n)]


def paths(parents):
    """Of every row: itself and what is above it, ascending. A parent that is no earlier row begins a path."""
    out = []
    for j, p in enumerate(parents):
        out.append((out[p] if 0 <= p < j else []) + [j])
    return out


def words(rows, n):
    """Mask words of lists of rows, n words each, as int32."""
    m = np.zeros((len(rows), n), np.uint32)
    for j, a in enumerate(rows):
        for i in a:
            m[j, i // 32] |= np.uint32(1 << (i % 32))
    return m.view(np.int32)


def softmax(x, t):
    """Row x's distribution, or None where it has none."""
    x = np.asarray(x, np.float64)
    m = x.max()
    if not np.isfinite(m) or np.isnan(x).any():
        return None
    if not t > 0:
        return np.eye(len(x))[int(np.argmax(x))]
    with np.errstate(over="ignore"):  # (a tiny temperature)
        e = np.exp((x - m) / t)
    return e / e.sum()


def verify(logits, tokens, uniforms, parents, t, probs=None):
    """(path, next token, how near the nearest decision was to the other one: relative to what was compared)."""
    n, vocab = logits.shape
    node, path, near = 0, [0], np.inf
    p = softmax(logits[0], t)
    j = 1
    while p is not None and j < n:
        if parents[j] != node or not 0 <= tokens[j] < vocab:
            j += 1
            continue
        d = tokens[j]
        q = np.eye(vocab)[d] if probs is None or not t > 0 else np.asarray(probs[node], np.float64)
        a, b = float(uniforms[j]) * q[d], p[d]
        if t > 0:
            near = min(near, abs(a - b) / max(a, b, 1e-300))
        if a < b:
            node = j
            path.append(j)
            p = softmax(logits[node], t)
        else:
            rest = np.maximum(p - q, 0.0)
            if rest.sum() > 0:
                p = rest / rest.sum()
        j += 1
    if p is None:
        return path, -1, near
    c = np.cumsum(p)
    want = float(uniforms[0]) * c[-1]
    if t > 0:
        near = min(near, np.abs(c[p > 0] - want).min())
    above = np.nonzero((c > want) & (p > 0))[0]
    return path, int(above[0]) if len(above) else int(np.nonzero(p > 0)[0][-1]), near
