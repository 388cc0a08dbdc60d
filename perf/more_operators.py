"""The operators of speculative decoding and of a bounded cache, as they are measured.

Five operators over the paged 4-bit cache and the target's logits, each in a plain form of elementary
torch operations and, with `own` set, as the calls a user makes of latency_moe_decode_gb300.ops:

* tree: who sees whom in each sequence's tree of drafted tokens, and attention of the drafted tokens
  over the cache: every stored position, and those of the tree that lie on the token's own path;
* verify: which path of a tree (or chain) of drafted tokens the target's probabilities accept, from
  given random numbers, and the token that follows it;
* commit: appending a tree's keys and values (rotated by depth), and moving the accepted path's to
  where a sequence without a tree would have them;
* mass: the attention weight that every cached position receives from a call's queries, accumulated;
* evict: the positions that a bounded cache keeps (the first ones, the last ones, and between them the
  heaviest), and their keys, values and weights moved together into fresh pages.

The cache holds each 16 consecutive values x of a row as codes c in -8 .. 7 and one scale s:
s = max|x| / 7 rounded to 3 mantissa bits (5 exponent bits, at most 480), c = x / s rounded to
even, value c * s.
"""
import math
import random

import torch

own = False

BLOCK = 16


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one user, a tree of 16 drafted tokens on 1k of context: latency
        dict(name="tree_b1_1k", op="tree", batch=1, new_lo=16, new_hi=16, len_lo=1024, len_hi=1024, hq=32, hkv=8, hd=128,
             bush=4, page=64, layout=1),
        # 32 users with trees of up to 64 tokens on contexts of up to 4k: the largest verify step
        dict(name="tree_b32_4k", op="tree", batch=32, new_lo=24, new_hi=64, len_lo=500, len_hi=4096, hq=32, hkv=8, hd=128,
             bush=8, page=64, layout=2),
        # heads of 64, a few odd tokens each on short histories (one empty), small pages
        dict(name="tree_odd_hd64", op="tree", batch=7, new_lo=1, new_hi=13, len_lo=0, len_hi=301, hq=4, hkv=2, hd=64,
             bush=3, page=16, layout=3),
        # one user's chain of seven drafts drawn from a draft model, the 8-layer stack's vocabulary: latency
        dict(name="verify_chain_b1", op="verify", batch=1, new_lo=8, new_hi=8, vocab=32000, dtype="f32", probs=True, bush=1,
             layout=4),
        # trees whose drafts are the draft model's likeliest tokens (no probabilities), bf16 logits
        dict(name="verify_tree_b16", op="verify", batch=16, new_lo=9, new_hi=64, vocab=32000, dtype="bf16", probs=False,
             bush=6, layout=5),
        # 64 users' chains with their draft model's probabilities: the most that is read
        dict(name="verify_chain_b64", op="verify", batch=64, new_lo=5, new_hi=8, vocab=32000, dtype="f32", probs=True, bush=1,
             layout=6),
        # one user's tree of 16 enters the cache and its path stays: latency
        dict(name="commit_b1", op="commit", batch=1, new_lo=16, new_hi=16, len_lo=1000, len_hi=1000, hkv=8, hd=128, bush=4,
             page=64, dtype="f32", layout=7),
        # 64 users' trees of odd sizes in small pages
        dict(name="commit_b64", op="commit", batch=64, new_lo=3, new_hi=61, len_lo=0, len_hi=2047, hkv=8, hd=128, bush=6,
             page=16, dtype="f32", layout=8),
        # a decode step of 16 users of 8k to 32k adds its attention weight to what the positions have
        dict(name="mass_step_b16_32k", op="mass", batch=16, new_lo=1, new_hi=1, len_lo=8000, len_hi=32768, hq=32, hkv=8,
             hd=128, causal=True, decay=1.0, page=64, layout=9),
        # two prompts' last 64 tokens weigh the 4k to 8k before them, from nothing
        dict(name="mass_window_64", op="mass", batch=2, new_lo=64, new_hi=64, len_lo=4000, len_hi=8192, hq=32, hkv=8, hd=128,
             causal=True, decay=0.0, page=64, layout=10),
        # one user's 32k brought down to 8k
        dict(name="evict_b1_32k", op="evict", batch=1, len_lo=32768, len_hi=32768, hkv=8, hd=128, budget=8192, sinks=4,
             recent=256, page=64, layout=11),
        # 24 users of odd lengths, some of them within the budget already, small pages, heads of 64
        dict(name="evict_b24_odd", op="evict", batch=24, len_lo=90, len_hi=4100, hkv=2, hd=64, budget=1001, sinks=1,
             recent=33, page=16, layout=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "verify", "commit", "mass", "evict"])
    layout = rng.randrange(13, 1 << 30)
    bush = rng.choice([1, 2, 4, 8])
    if op == "verify":
        vocab = _log(rng, 300, 160000)
        new = _log(rng, 1, 64)
        batch = _log(rng, 1, max(1, min(64, 14000000 // (new * vocab))))
        return dict(op=op, batch=batch, new_lo=max(1, new // 2), new_hi=new, vocab=vocab, dtype=rng.choice(["bf16", "f32"]),
                    probs=rng.random() < 0.5, bush=bush, layout=layout)
    hd = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        new = _log(rng, 1, 64)
        length = _log(rng, 1, 8192)
        batch = _log(rng, 1, max(1, min(32, 120000 // (length + new))))
        return dict(op=op, batch=batch, new_lo=max(1, new // 3), new_hi=new, len_lo=length // 4, len_hi=length, hq=hq, hkv=hkv,
                    hd=hd, bush=bush, page=page, layout=layout)
    if op == "commit":
        new = _log(rng, 1, 64)
        return dict(op=op, batch=_log(rng, 1, 64), new_lo=max(1, new // 3), new_hi=new, len_lo=0, len_hi=_log(rng, 1, 4000),
                    hkv=hkv, hd=hd, bush=bush, page=page, dtype=rng.choice(["bf16", "f32"]), layout=layout)
    if op == "mass":
        new = rng.choice([1, 1, _log(rng, 2, 128)])
        length = _log(rng, 1, 32768 if new == 1 else 8192)
        batch = _log(rng, 1, max(1, min(32, (300000 if new == 1 else 1500000 // new) // (length + new))))
        return dict(op=op, batch=batch, new_lo=max(1, new // 2), new_hi=new, len_lo=length // 4, len_hi=length, hq=hq, hkv=hkv,
                    hd=hd, causal=rng.random() < 0.7, decay=rng.choice([0.0, 0.9, 1.0]), page=page, layout=layout)
    length = _log(rng, 16, 32768)
    budget = max(8, int(length * rng.uniform(0.1, 0.9)))
    return dict(op=op, batch=_log(rng, 1, max(1, min(32, 60000 // length))), len_lo=length // 5, len_hi=length, hkv=hkv, hd=hd,
                budget=budget, sinks=rng.choice([0, 1, 4]), recent=rng.randrange(0, budget // 2), page=page, layout=layout)


def _sizes(case):
    """New tokens and stored lengths of each sequence (the case's, not the seed's)."""
    r = random.Random(case["layout"])
    new = [r.randint(case.get("new_lo", 0), case.get("new_hi", 0)) for _ in range(case["batch"])]
    lens = [r.randint(case.get("len_lo", 0), case.get("len_hi", 0)) for _ in range(case["batch"])]
    if case["batch"] > 2:
        new[0], lens[0] = case.get("new_hi", 0), case.get("len_hi", 0)
        new[1], lens[1] = case.get("new_lo", 0), case.get("len_lo", 0)
    return new, lens


def _parents(case):
    """Each sequence's tree: row 0 is its last known token, every other row's parent an earlier row (bush 1: a chain)."""
    r = random.Random(case["layout"] + 1)
    return [[-1] + [r.randrange(max(0, j - case["bush"]), j) for j in range(1, n)] for n in _sizes(case)[0]]


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _paths(case, seed=0):
    """A path through each tree, as verification might leave it: from the root to some node."""
    r = random.Random(case["layout"] + 2)
    out = []
    for p in _parents(case):
        j, path = r.randrange(len(p)), []
        while j >= 0:
            path.insert(0, j)
            j = p[j]
        out.append(path)
    return out


def work(case):
    op = case["op"]
    new, lens = _sizes(case)
    if op == "verify":
        n = sum(new) * case["vocab"]
        # every row of logits, the draft's row where a chain ends
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + (case["batch"] * case["vocab"] * 4 if case["probs"] else 0) +
                sum(new) * 20, "flops": 5 * n}
    hkv, hd = case["hkv"], case["hd"]
    row = 2 * hkv * (hd // 2 + hd // BLOCK)  # one position's keys and values in the cache
    if op == "commit":
        n = sum(new)
        moved = sum(i != j for p in _paths(case) for i, j in enumerate(p))
        # keys and values in, codes written and read back, bf16 out, the path's codes read and written
        return {"bytes": n * (2 * hkv * hd * (2 if case["dtype"] == "bf16" else 4) + 2 * row + 4 * hkv * hd + hd * 4) + 2 * moved * row,
                "flops": n * 2 * hkv * hd * 8}
    if op == "evict":
        kept = sum(min(l, case["budget"]) for l in lens)
        # the weights read, the kept positions' codes and weights read and written, codes read back, bf16 out
        return {"bytes": sum(lens) * hkv * 4 + kept * (3 * row + hkv * (4 + 8) + 4 * hkv * hd), "flops": 2 * sum(lens) * hkv}
    hq = case["hq"]
    if op == "tree":
        pairs = sum(n * l + sum(d + 1 for d in _depths(p)) for n, l, p in zip(new, lens, _parents(case)))
        return {"bytes": (sum(new) + sum(lens)) * row + sum(new) * hq * (4 * hd + 4), "flops": 4 * pairs * hq * hd}
    causal = case["causal"]
    seen = sum(l + n if causal else l for n, l in zip(new, lens))
    pairs = sum(n * l + (n * (n + 1) // 2 if causal else 0) for n, l in zip(new, lens))
    return {"bytes": seen * (row // 2 + hkv * (8 if case["decay"] else 4)) + sum(new) * hq * (2 * hd + 4),
            "flops": 2 * pairs * hq * hd}


# ---------------------------------------------------------------------------------------------
# inputs

def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bounds(n):
    return _ints([0] + [sum(n[:b + 1]) for b in range(len(n))])


def _inputs(case, seed):
    """The raw inputs of a case, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    op = case["op"]
    dt = torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
    uni = lambda *s: torch.rand(*s, generator=g, device=dev)
    new, lens = _sizes(case)
    n = sum(new)
    s = dict(cu=_bounds(new), n_tokens=n, max_tokens=max(new))
    if op in ("tree", "verify", "commit"):
        s["parents"] = _ints([p for ps in _parents(case) for p in ps])
    if op == "verify":
        vocab = case["vocab"]
        x = 2.5 * rnd(n, vocab)
        peak = torch.randint(0, vocab, (n, 3), generator=g, device=dev)
        x.scatter_add_(1, peak, 9.0 + 2.0 * rnd(n, 3))
        s["logits"] = x.to(dt)
        r = random.Random(case["layout"] + 3)
        # a few users decode greedily, the others at temperatures around 1
        t = torch.tensor([r.choice([0.0, 0.6, 0.8, 1.0, 1.0, 1.2]) for _ in new], device=dev)
        s["temperature"] = t if case["batch"] > 1 else torch.ones(1, device=dev)
        per_row = torch.repeat_interleave(s["temperature"], torch.tensor(new, device=dev))[:, None]
        draft = (x + 0.8 * rnd(n, vocab)) / torch.where(per_row > 0, per_row, torch.ones_like(per_row))
        if case["probs"]:
            s["draft_probs"] = torch.softmax(draft, 1)
        first = torch.repeat_interleave(s["cu"][:-1].long(), torch.tensor(new, device=dev))
        up = (first + s["parents"].long()).clamp(min=0)
        # each draft drawn from its parent's row
        noise = -torch.log(-torch.log(uni(n, vocab).clamp(1e-20, 1 - 1e-7)))
        s["tokens"] = (draft[up] + noise).argmax(1).to(torch.int32)
        s["uniforms"] = uni(n)
        return s
    hkv, hd, page = case["hkv"], case["hd"], case["page"]
    total = [a + b for a, b in zip(new, lens)]
    pages = [(t + page - 1) // page for t in total]
    fresh = [(min(l, case["budget"]) + page - 1) // page for l in lens] if op == "evict" else []
    n_pages = sum(pages) + sum(fresh) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    at = 0
    for name, each in (("table", pages), ("to", fresh)):
        t = torch.full((case["batch"], max(each, default=0)), 0, dtype=torch.int32, device=dev)
        for b, p in enumerate(each):
            t[b, :p] = perm[at:at + p]
            at += p
        s[name] = t
    s.update(n_pages=n_pages, page=page, lengths=_ints(lens))
    chan = 1.0 + 5.0 * (uni(hkv, hd) < 0.03)  # channels of large keys
    if op == "commit":
        s.update(k=(rnd(n, hkv, hd) * chan).to(dt), v=(0.7 * rnd(n, hkv, hd)).to(dt))
        inv = 1e6 ** (-torch.arange(0, hd, 2, dtype=torch.float64, device=dev) / hd)
        a = torch.arange(max(total), dtype=torch.float64, device=dev)[:, None] * inv
        s["rope"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()  # the table a server keeps
        paths = _paths(case)
        s["path"] = _ints([p + [-1] * (s["max_tokens"] - len(p)) for p in paths])
        s["count"] = _ints([len(p) for p in paths])
        return s
    # the stored rows of every sequence, one after another (history, and the new tokens')
    held = lens if op == "evict" or not case.get("causal", True) else total
    t = max(1, sum(held))
    s.update(held=held, k=(rnd(t, hkv, hd) * chan).to(torch.bfloat16), v=rnd(t, hkv, hd).to(torch.bfloat16))
    if op != "tree":
        # weights as positions collect them: a few heavy, most light, some none at all
        s["mass"] = torch.exp(2.0 * rnd(n_pages, hkv, page) - 4.0) * (uni(n_pages, hkv, page) > 0.1)
    if op != "evict":
        hq = case["hq"]
        q = rnd(n, hkv, hq // hkv, hd)
        pick = torch.randint(0, t, (n,), generator=g, device=dev)
        q = 0.7 * q + 0.25 * s["k"][pick].float()[:, :, None, :]  # each query leans on one stored key
        s["q"] = q.reshape(n, hq, hd).to(torch.bfloat16)
    if op == "mass":  # what the step's attention left beside its output
        k, lse, at, row = _held(s["k"]), [], 0, 0
        for a, l, h in zip(new, lens, held):
            x = torch.einsum("jhgd,phd->jhgp", s["q"][row:row + a].float().view(a, hkv, -1, hd), k[at:at + h]) / math.sqrt(hd)
            if case["causal"]:
                x.masked_fill_((torch.arange(h, device=dev) > l + torch.arange(a, device=dev)[:, None])[:, None, None], -math.inf)
            lse.append(torch.logsumexp(x.double(), -1).flatten(1) if h else torch.full((a, case["hq"]), -math.inf, device=dev))
            at, row = at + h, row + a
        s["lse"] = torch.cat([x.float() for x in lse])
    return s


def _quantise(x):
    """Codes and scales of rows x [..., hd] in float64."""
    b = x.double().unflatten(-1, (-1, BLOCK))
    _, e = torch.frexp(b.abs().amax(-1) / 7)  # in [2^(e - 1), 2^e): steps of 2^(e - 4), of 2^-14 below 2^-11
    e = e.clamp(min=-10)
    step = ((e.long() + (1023 - 4)) << 52).view(torch.float64)  # 2^(e - 4), exactly: codes meet ties
    s = ((b.abs().amax(-1) / 7 / step).round() * step).clamp(max=480.0)
    c = torch.where(s[..., None] > 0, (b / s[..., None]).round().clamp(-8, 7), 0.0)
    return c.flatten(-2).to(torch.int8), s.float()


def _held(x):
    c, s = _quantise(x)
    return c * s.repeat_interleave(BLOCK, -1)


def _where(cu, table, page, start, rows):
    """(page, offset in the page) of `rows` consecutive rows that cu divides among the sequences."""
    seq = torch.searchsorted(cu[1:], torch.arange(rows, dtype=torch.int32, device="cuda"), right=True)
    pos = start[seq] + torch.arange(rows, device="cuda") - cu[seq]
    return seq, pos, table[seq, pos // page].long(), pos % page


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "verify":
        return s
    hkv, hd, page = case["hkv"], case["hd"], case["page"]
    if own:
        from latency_moe_decode_gb300 import ops
        s["cache"] = ops.KvqCache(s["n_pages"], hkv, hd, page_tokens=page)
    else:
        s["codes"] = torch.zeros(2, s["n_pages"], hkv, page, hd, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(2, s["n_pages"], hkv, page, hd // BLOCK, device="cuda")
    if op == "mass":
        s["sums"] = torch.zeros_like(s["mass"])
    s["zero"] = torch.zeros_like(s["lengths"])
    if op == "evict":
        s["kept_cu"] = _bounds([min(l, case["budget"]) for l in _sizes(case)[1]])
        s["n_kept"] = sum(min(l, case["budget"]) for l in _sizes(case)[1])
    if op != "commit":
        held = s.pop("held")
        if sum(held):
            cu = _bounds(held)
            if own:
                s["cache"].append(s["k"], s["v"], s["zero"], s["table"], cu_tokens=cu)
            else:
                _, _, at, off = _where(cu, s["table"], page, s["zero"], s["k"].shape[0])
                for i, x in enumerate((s["k"], s["v"])):
                    s["codes"][i][at, :, off], s["scales"][i][at, :, off] = _quantise(x)
        del s["k"], s["v"]
    return s


# ---------------------------------------------------------------------------------------------
# the operators

def _rows(s):
    """The sequence of every row and its index there."""
    seq = torch.searchsorted(s["cu"][1:], torch.arange(s["n_tokens"], dtype=torch.int32, device="cuda"), right=True)
    return seq, torch.arange(s["n_tokens"], device="cuda") - s["cu"][seq]


def _tree_sees(s):
    """[n, max_tokens]: row by row, which rows of its sequence lie on its path (itself included); depths."""
    seq, j = _rows(s)
    most = s["max_tokens"]
    sees = torch.zeros(s["n_tokens"], most, dtype=torch.bool, device="cuda")
    at = j.long()
    for _ in range(most):  # one step up at a time
        live = at >= 0
        sees |= torch.nn.functional.one_hot(at.clamp(min=0), most).bool() & live[:, None]
        at = torch.where(live, s["parents"][(s["cu"][seq] + at.clamp(min=0)).long()].long(), at)
    return seq, j, sees, sees.sum(-1) - 1


def _dense(s, kind):
    """Keys (0) or values (1) as their sequences have them: [batch, hkv, positions, hd]."""
    t = s["table"].long()
    return (s["codes"][kind][t].float() * s["scales"][kind][t].repeat_interleave(BLOCK, -1)).transpose(1, 2).flatten(2, 3)


def _scores(s, seq, j):
    c = s["case"]
    q = torch.zeros(c["batch"], s["max_tokens"], c["hkv"], c["hq"] // c["hkv"], c["hd"], device="cuda")
    q[seq, j] = s["q"].float().view(s["n_tokens"], c["hkv"], -1, c["hd"])
    return torch.einsum("bjhgd,bhpd->bhgjp", q, _dense(s, 0)) / math.sqrt(c["hd"])


def _tree(s):
    seq, j, sees, depth = _tree_sees(s)
    most, c = s["max_tokens"], s["case"]
    x = _scores(s, seq, j)
    p = torch.arange(x.shape[-1], device="cuda")
    dense = torch.zeros(c["batch"], most, most, dtype=torch.bool, device="cuda")
    dense[seq, j] = sees
    i = p - s["lengths"][:, None]  # [batch, positions]: the tree's row that stands there
    on = dense.gather(2, i.clamp(0, most - 1).long()[:, None].expand(-1, most, -1)) & (i < most)[:, None]
    see = torch.where((i < 0)[:, None], True, on)  # [batch, most, positions]
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m.clamp(min=-1e30))
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgjp,bhpd->bjhgd", e / total.clamp(min=1e-30), _dense(s, 1))
    lse = (m + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    words = (most + 31) // 32
    bits = torch.nn.functional.pad(sees, (0, 32 * words - most)).view(-1, words, 32).long() << torch.arange(32, device="cuda")
    mask = bits.sum(-1)
    return {"mask": torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32),
            "positions": (s["lengths"][seq] + depth).to(torch.int32),
            "out": o[seq, j].flatten(1, 2).to(torch.bfloat16), "lse": lse[seq, j].flatten(1)}


def _verify(s):
    """All sequences at once, in 64 bits (a sum's border decides a token), one row of every tree at a time."""
    batch, most, vocab = s["case"]["batch"], s["max_tokens"], s["case"]["vocab"]
    first, n = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    t = s["temperature"].double()[:, None]
    greedy = t <= 0
    one = torch.arange(batch, device="cuda")

    def target(rows):
        x = s["logits"][rows].double()
        e = torch.exp((x - x.amax(1, keepdim=True)) / torch.where(greedy, 1.0, t))
        best = torch.zeros_like(x)
        best[one, x.argmax(1)] = 1.0
        return torch.where(greedy, best, e / e.sum(1, keepdim=True))

    node = torch.zeros(batch, dtype=torch.long, device="cuda")
    p = target(first)
    path = torch.full((batch, most), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    count = torch.ones(batch, dtype=torch.long, device="cuda")
    for j in range(1, most):
        row = (first + j).clamp(max=s["n_tokens"] - 1)
        child = (j < n) & (s["parents"][row] == node)
        d = s["tokens"][row].long()
        q = torch.nn.functional.one_hot(d, vocab).double()
        if "draft_probs" in s:
            q = torch.where(greedy, q, s["draft_probs"][first + node].double())
        take = child & (s["uniforms"][row].double() * q[one, d] < p[one, d])
        left = (p - q).clamp(min=0.0)
        rest = left.sum(1, keepdim=True)
        left = torch.where(rest > 0, left / rest.clamp(min=1e-300), p)
        node = torch.where(take, j, node)
        p = torch.where((child & ~take)[:, None], left, p)
        p = torch.where(take[:, None], target(first + node), p)
        path[one, torch.where(take, count, most - 1)] = torch.where(take, j, path[one, most - 1])
        count = count + take
    c = p.cumsum(1)
    past = c > s["uniforms"][first].double()[:, None] * c[:, -1:]
    last = vocab - 1 - (p > 0).int().flip(1).argmax(1)
    return {"path": path.to(torch.int32), "count": count.to(torch.int32),
            "next": torch.where(past.any(1), past.int().argmax(1), last).to(torch.int32)}


def _rotate(x, table, pos):
    half = x.shape[-1] // 2
    c, d = table[pos.long()].double().unbind(-1)
    c, d = c[:, None], d[:, None]
    a, b = x[..., :half].double(), x[..., half:].double()
    return torch.cat([a * c - b * d, a * d + b * c], -1)


def _commit(s):
    seq, j, _, depth = _tree_sees(s)
    _, _, at, off = _where(s["cu"], s["table"], s["page"], s["lengths"], s["n_tokens"])
    source = j.long()
    kept = j < s["count"][seq]
    source[kept] = s["path"][seq[kept], j[kept].long()].long()
    row = s["cu"][seq] + source
    got = []
    for i, x in enumerate((_rotate(s["k"], s["rope"], s["lengths"][seq] + depth), s["v"])):
        codes, scales = _quantise(x)
        s["codes"][i][at, :, off], s["scales"][i][at, :, off] = codes[row], scales[row]
        got.append((s["codes"][i][at, :, off] * s["scales"][i][at, :, off].repeat_interleave(BLOCK, -1)).to(torch.bfloat16))
    return {"k": got[0], "v": got[1]}


def _mass(s):
    c = s["case"]
    seq, j = _rows(s)
    most = s["max_tokens"]
    x = _scores(s, seq, j)
    lse = torch.full((c["batch"], most, c["hq"]), math.inf, device="cuda")  # (rows that are not there weigh nothing)
    lse[seq, j] = torch.where(s["lse"] > -math.inf, s["lse"], math.inf)
    p = torch.arange(x.shape[-1], device="cuda")
    n = s["cu"][1:] - s["cu"][:-1]
    last = s["lengths"][:, None] + (torch.arange(1, most + 1, device="cuda") if c["causal"] else torch.zeros(most, device="cuda"))
    see = (p < last[..., None])[:, None, None]
    e = torch.exp(x - lse.view(c["batch"], most, c["hkv"], -1).permute(0, 2, 3, 1)[..., None])
    sums = torch.where(see, e, 0.0).sum((2, 3))  # [batch, hkv, positions]
    there = p < (s["lengths"] + n if c["causal"] else s["lengths"])[:, None]
    old = p < s["lengths"][:, None]
    b, pos = there.nonzero(as_tuple=True)
    at, off = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    before = torch.where(old[b, pos][:, None], s["mass"][at, :, off], 0.0)
    s["sums"][at, :, off] = sums[b, :, pos] + (c["decay"] * before if c["decay"] else 0.0)
    return {"mass": s["sums"]}


def _evict(s):
    c = s["case"]
    page, budget = s["page"], c["budget"]
    t = s["table"].long()
    w = s["mass"][t].transpose(1, 2).flatten(2)  # [batch, hkv, positions]
    p, n = torch.arange(w.shape[-1], device="cuda"), s["lengths"][:, None, None]
    w = torch.where((p < c["sinks"]) | (p >= n - c["recent"]), math.inf, w)
    w = torch.where(p < n, w, -math.inf)
    w = torch.nn.functional.pad(w, (0, max(0, budget - w.shape[-1])), value=-math.inf)
    kept = torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :budget]
    kept = torch.where(kept < n, kept, 1 << 30).sort(-1)[0]
    count = s["lengths"].clamp(max=budget)
    kept = torch.where(kept < 1 << 30, kept, -1)
    seq, i, at, off = _where(s["kept_cu"], s["to"], page, s["zero"], s["n_kept"])
    src = kept[seq, :, i.long()]  # [rows, hkv]
    h = torch.arange(c["hkv"], device="cuda")
    sp, so = t[seq[:, None], src // page], src % page
    got = []
    for kind in (0, 1):
        codes, scales = s["codes"][kind], s["scales"][kind]
        codes[at[:, None], h, off[:, None]], scales[at[:, None], h, off[:, None]] = codes[sp, h, so], scales[sp, h, so]
        got.append((codes[at, :, off] * scales[at, :, off].repeat_interleave(BLOCK, -1)).to(torch.bfloat16))
    s["mass"][at[:, None], h, off[:, None]] = s["mass"][sp, h, so]
    return {"kept": kept.to(torch.int32), "count": count.to(torch.int32), "k": got[0], "v": got[1], "mass": s["mass"]}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"tree": _tree, "verify": _verify, "commit": _commit, "mass": _mass, "evict": _evict}[op](s)
    from latency_moe_decode_gb300 import ops
    if op == "verify":
        r = ops.verify_drafts(s["logits"], s["tokens"], s["uniforms"], s["cu"], parents=s["parents"],
                              draft_probs=s.get("draft_probs"), temperature=s["temperature"], max_tokens=s["max_tokens"])
        return {"path": r.path, "count": r.count, "next": r.next_tokens}
    cache = s["cache"]
    if op == "tree":
        tree = ops.draft_tree(s["parents"], s["lengths"], s["cu"], max_tokens=s["max_tokens"])
        out, lse = cache.attention(s["q"], s["lengths"], s["table"], cu_tokens=s["cu"], max_tokens=s["max_tokens"],
                                   tree_mask=tree.mask, return_lse=True)
        return {"mask": tree.mask, "positions": tree.positions, "out": out, "lse": lse}
    if op == "commit":
        tree = ops.draft_tree(s["parents"], s["lengths"], s["cu"], max_tokens=s["max_tokens"])
        cache.append(s["k"], s["v"], s["lengths"], s["table"], cu_tokens=s["cu"], rope=s["rope"], positions=tree.positions)
        cache.move(s["path"], s["count"], s["table"], start=s["lengths"])
        k, v = cache.gather(s["lengths"], s["table"], s["n_tokens"], cu_tokens=s["cu"])
        return {"k": k, "v": v}
    if op == "mass":
        cache.attention_mass(s["q"], s["lse"], s["lengths"], s["table"], s["mass"], cu_tokens=s["cu"],
                             max_tokens=s["max_tokens"], causal=c["causal"], decay=c["decay"], out=s["sums"])
        return {"mass": s["sums"]}
    kept, count = cache.heaviest(s["mass"], s["lengths"], s["table"], c["budget"], sinks=c["sinks"], recent=c["recent"])
    cache.move(kept, count, s["table"], to=s["to"], mass=s["mass"])
    k, v = cache.gather(s["zero"], s["to"], s["n_kept"], cu_tokens=s["kept_cu"])
    return {"kept": kept, "count": count, "k": k, "v": v, "mass": s["mass"]}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _stored(x):
    """The values the cache holds for rows x, from the definition: each scale is the nearest of
    all the scales there are, ties to the even one."""
    grid = torch.tensor([8.0 * ((8 + m if e else m) / 8.0) * 2.0 ** (max(e, 1) - 15) for e in range(21) for m in range(8)][:168],
                        dtype=torch.float64, device=x.device)
    b = x.double().reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    want = b.abs().max(-1).values / 7.0
    hi = torch.searchsorted(grid, want.contiguous()).clamp(1, 167)
    lo = hi - 1
    a, z = want - grid[lo], grid[hi] - want
    s = grid[torch.where((a < z) | ((a == z) & (lo % 2 == 0)), lo, hi)][..., None]
    c = torch.where(s > 0, torch.clamp(torch.round(b / torch.where(s > 0, s, 1.0)), -8.0, 7.0), 0.0)
    return (c * s).reshape(x.shape)


def _ancestors(parents):
    out = []
    for j, p in enumerate(parents):
        out.append(([] if p < 0 else out[p]) + [j])
    return out


def _exact_verify(case, s):
    paths, nexts, row = [], [], 0
    for parents, t in zip(_parents(case), s["temperature"].tolist()):
        n = len(parents)
        x, u, d = s["logits"][row:row + n].double(), s["uniforms"][row:row + n].tolist(), s["tokens"][row:row + n].tolist()

        def probabilities(j):
            if t <= 0:
                return torch.nn.functional.one_hot(x[j].argmax(), case["vocab"]).double()
            return torch.softmax(x[j] / t, 0)

        path, p = [0], probabilities(0)
        while True:
            for c in [c for c in range(path[-1] + 1, n) if parents[c] == path[-1]]:
                if "draft_probs" in s and t > 0:
                    q = s["draft_probs"][row + path[-1]].double()
                else:
                    q = torch.zeros_like(p)
                    q[d[c]] = 1.0
                if u[c] * float(q[d[c]]) < float(p[d[c]]):
                    break
                rest = torch.relu(p - q)
                p = rest / rest.sum() if float(rest.sum()) > 0 else p
            else:
                break
            path.append(c)
            p = probabilities(c)
        up = torch.cumsum(p, 0)
        above = torch.nonzero(up > u[0] * up[-1])
        nexts.append(int(above[0]) if len(above) else int(torch.nonzero(p > 0)[-1]))
        paths.append(path)
        row += n
    most = s["max_tokens"]
    return {"path": _ints([p + [-1] * (most - len(p)) for p in paths]), "count": _ints([len(p) for p in paths]), "next": _ints(nexts)}


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(case, s)
    new, lens = _sizes(case)
    hkv, hd, page = case["hkv"], case["hd"], case["page"]
    if op == "commit":
        ks, vs, row = [], [], 0
        for parents, path, l in zip(_parents(case), _paths(case), lens):
            n = len(parents)
            source = path + list(range(len(path), n))
            turn = s["rope"][_ints([l + len(a) - 1 for a in _ancestors(parents)]).long()].double()
            z = torch.complex(turn[..., 0], turn[..., 1])[:, None]
            k = s["k"][row:row + n].double()
            y = torch.complex(k[..., :hd // 2], k[..., hd // 2:]) * z
            ks.append(_stored(torch.cat([y.real, y.imag], -1))[source])
            vs.append(_stored(s["v"][row:row + n])[source])
            row += n
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    if op == "evict":
        kept = torch.full((case["batch"], hkv, case["budget"]), -1, dtype=torch.int32)
        k, v, ks, vs, at = _stored(s["k"]), _stored(s["v"]), [], [], 0
        mass = s["mass"].double()
        table, to = s["table"].tolist(), s["to"].tolist()
        for b, l in enumerate(lens):
            p = torch.arange(l, device="cuda")
            src = torch.tensor(table[b], device="cuda")[p // page]
            m = min(l, case["budget"])
            dst = torch.tensor(to[b], device="cuda")[p[:m] // page]
            safe = [i for i in range(l) if i < case["sinks"] or i >= l - case["recent"]]
            kk, vv = [], []
            for h in range(hkv):
                w = s["mass"][src, h, p % page].double()
                rest = torch.argsort(w, descending=True, stable=True).tolist()
                chosen, have = set(safe) if l > m else set(range(l)), None
                for i in rest:
                    if len(chosen) >= m:
                        break
                    chosen.add(i)
                have = torch.tensor(sorted(chosen), device="cuda")
                kept[b, h, :m] = have.int().cpu()
                kk.append(k[at + have, h])
                vv.append(v[at + have, h])
                mass[dst, h, p[:m] % page] = w[have]
            ks.append(torch.stack(kk, 1))
            vs.append(torch.stack(vv, 1))
            at += l
        return {"kept": kept.cuda(), "count": _ints([min(l, case["budget"]) for l in lens]), "k": torch.cat(ks),
                "v": torch.cat(vs), "mass": mass}
    hq = case["hq"]
    k, v, q = _stored(s["k"]), _stored(s["v"]), s["q"].double()
    if op == "mass":
        out = torch.zeros_like(s["mass"], dtype=torch.float64)
        at = row = 0
        for b, (n, l, held) in enumerate(zip(new, lens, s["held"])):
            total = torch.zeros(hkv, held, dtype=torch.float64, device="cuda")
            kk = k[at:at + held].permute(1, 2, 0)  # [hkv, hd, held]
            for j0 in range(0, n if held else 0, 16):
                j = torch.arange(j0, min(n, j0 + 16), device="cuda")
                x = torch.matmul(q[row + j].view(len(j), hkv, hq // hkv, hd).transpose(0, 1).flatten(1, 2), kk) * hd ** -0.5
                x = (x.view(hkv, len(j), -1, held) - s["lse"][row + j].double().view(len(j), hkv, -1).transpose(0, 1)[..., None]).exp()
                if case["causal"]:
                    x = x * (torch.arange(held, device="cuda")[None] <= l + j[:, None])[:, None]
                total += x.sum((1, 2))
            p = torch.arange(held, device="cuda")
            pg = s["table"][b, p // page].long()
            was = torch.where((p < l)[:, None], s["mass"][pg, :, p % page].double(), 0.0)
            out[pg, :, p % page] = total.T + case["decay"] * was
            at, row = at + held, row + n
        return {"mass": out}
    outs, lses, masks, positions = [], [], [], []
    words = (max(new) + 31) // 32
    at = row = 0
    for n, l, held, parents in zip(new, lens, s["held"], _parents(case)):
        paths = _ancestors(parents)
        kk = k[at:at + held].repeat_interleave(hq // hkv, 1).permute(1, 2, 0)
        vv = v[at:at + held].repeat_interleave(hq // hkv, 1).transpose(0, 1)
        x = torch.matmul(q[row:row + n].transpose(0, 1), kk) * hd ** -0.5
        hide = torch.ones(n, held, dtype=torch.bool)
        hide[:, :l] = False
        for j, a in enumerate(paths):
            hide[j, [l + i for i in a]] = False
            positions.append(l + len(a) - 1)
            bits = sum(1 << i for i in a)
            each = [(bits >> (32 * w)) & 0xFFFFFFFF for w in range(words)]
            masks.append([w - (1 << 32) if w >> 31 else w for w in each])
        x = x.masked_fill(hide.cuda(), -math.inf)
        lses.append(torch.logsumexp(x, -1).T)
        outs.append(torch.matmul(torch.softmax(x, -1), vv).transpose(0, 1))
        at += held
        row += n
    return {"mask": _ints(masks), "positions": _ints(positions), "out": torch.cat(outs), "lse": torch.cat(lses)}
