"""The serving operators beside the decode engine, as they are measured.

Three operators, each in a plain form of elementary torch operations and, with `own` set, as the
calls a user makes of latency_moe_decode_gb300.ops:

* append: RMSNorm of every query and key head, position rotation, and appending the keys and
  values to a paged cache of 4-bit codes, then reading the appended positions back;
* attention: attention over such a cache, for decode steps, verify steps and prompt chunks;
* logprobs: log probabilities of given tokens, with entropy, rank and the top alternatives.

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
        # one user's next token, a layer of the 8-layer stack with query / key norms: latency
        dict(name="append_step_b1", op="append", batch=1, new_lo=1, new_hi=1, len_lo=1000, len_hi=1000, hq=32, hkv=8,
             hd=128, rot=128, inter=False, norm=True, dtype="bf16", page=64, layout=1),
        # 64 sequences decoding together, fp32 projections as the engine's GEMVs leave them
        dict(name="append_step_b64", op="append", batch=64, new_lo=1, new_hi=1, len_lo=0, len_hi=2047, hq=32, hkv=8,
             hd=128, rot=128, inter=False, norm=False, dtype="f32", page=64, layout=2),
        # prompts of odd lengths entering small pages, half of each head rotated in adjacent pairs
        dict(name="append_prompts", op="append", batch=6, new_lo=17, new_hi=2500, len_lo=0, len_hi=700, hq=32, hkv=8,
             hd=128, rot=64, inter=True, norm=True, dtype="bf16", page=16, layout=3),
        # one user at 1k of context: latency
        dict(name="attn_step_b1_1k", op="attn", batch=1, new_lo=1, new_hi=1, len_lo=1023, len_hi=1023, hq=32, hkv=8,
             hd=128, causal=True, page=64, layout=4),
        # the largest decode batch, contexts from one token to 2k
        dict(name="attn_step_b64_2k", op="attn", batch=64, new_lo=1, new_hi=1, len_lo=0, len_hi=2047, hq=32, hkv=8,
             hd=128, causal=True, page=64, layout=5),
        # one user with a long document
        dict(name="attn_step_b1_64k", op="attn", batch=1, new_lo=1, new_hi=1, len_lo=65535, len_hi=65535, hq=32, hkv=8,
             hd=128, causal=True, page=64, layout=6),
        # a verify step of 8 positions at 8k
        dict(name="attn_verify8_8k", op="attn", batch=1, new_lo=8, new_hi=8, len_lo=8192, len_hi=8192, hq=32, hkv=8,
             hd=128, causal=True, page=32, layout=7),
        # many long contexts: the largest cache read
        dict(name="attn_step_b16_32k", op="attn", batch=16, new_lo=1, new_hi=1, len_lo=8000, len_hi=32768, hq=32, hkv=8,
             hd=128, causal=True, page=64, layout=8),
        # heads of 64, a few odd tokens each against stored prefixes (some empty), small pages
        dict(name="attn_prefix_hd64", op="attn", batch=7, new_lo=1, new_hi=5, len_lo=0, len_hi=301, hq=4, hkv=2,
             hd=64, causal=False, page=16, layout=9),
        # two prompts taking their next 256 tokens against 4k of history
        dict(name="attn_chunk_256", op="attn", batch=2, new_lo=256, new_hi=256, len_lo=3500, len_hi=4096, hq=32, hkv=8,
             hd=128, causal=True, page=64, layout=10),
        # one user's token with five alternatives, the 8-layer stack's vocabulary: latency
        dict(name="logprobs_step", op="logprobs", rows=1, vocab=32000, dtype="f32", top=5, masked=False),
        # a scored prompt, bf16 logits (many ties), some tokens masked
        dict(name="logprobs_prompt", op="logprobs", rows=2048, vocab=32000, dtype="bf16", top=20, masked=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "logprobs"])
    layout = rng.randrange(11, 1 << 30)
    hd = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        new = _log(rng, 1, 2500)
        batch = _log(rng, 1, max(1, min(64, 7000 // new)))
        return dict(op=op, batch=batch, new_lo=max(1, new // 3), new_hi=new, len_lo=0, len_hi=_log(rng, 1, 4000), hq=hq,
                    hkv=hkv, hd=hd, rot=rng.choice([0, 16, hd // 2, hd]), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]), page=page, layout=layout)
    if op == "attn":
        new = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 2, 256)])
        length = _log(rng, 1, 65536 if new == 1 else 8192)
        room = 320000 // length if new <= 8 else 1000 // new
        batch = _log(rng, 1, max(1, min(64, room)))
        if new > 8:
            length = min(length, 4096)
        return dict(op=op, batch=batch, new_lo=max(1, new // 2), new_hi=new, len_lo=length // 4, len_hi=length, hq=hq,
                    hkv=hkv, hd=hd, causal=rng.random() < 0.7, page=page, layout=layout)
    vocab = _log(rng, 1000, 160000)
    return dict(op=op, rows=_log(rng, 1, max(1, min(2048, 60000000 // vocab))), vocab=vocab,
                dtype=rng.choice(["bf16", "f32"]), top=rng.choice([0, 1, 5, 20, 32]), masked=rng.random() < 0.5)


def _sizes(case):
    """New tokens and stored lengths of each sequence (the case's, not the seed's)."""
    r = random.Random(case["layout"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["batch"])]
    if case["batch"] > 2:
        new[0], lens[0] = case["new_hi"], case["len_hi"]
        new[1], lens[1] = case["new_lo"], case["len_lo"]
    return new, lens


def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * (16 + 8 * case["top"]), "flops": 5 * n}
    new, lens = _sizes(case)
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    row = 2 * hkv * (hd // 2 + hd // BLOCK)  # one position's keys and values in the cache
    if case["op"] == "append":
        n = sum(new)
        e = 2 if case["dtype"] == "bf16" else 4
        # inputs, bf16 queries out, codes written, codes read back, bf16 keys and values out
        return {"bytes": n * ((hq + 2 * hkv) * hd * e + hq * hd * 2 + 2 * row + 2 * hkv * hd * 2 + case["rot"] * 4),
                "flops": n * (hq + 2 * hkv) * hd * 12}
    seen = sum(l + n if case["causal"] else l for n, l in zip(new, lens))
    pairs = sum(n * l + (n * (n + 1) // 2 if case["causal"] else 0) for n, l in zip(new, lens))
    return {"bytes": seen * row + sum(new) * hq * (4 * hd + 4), "flops": 4 * pairs * hq * hd}


# ---------------------------------------------------------------------------------------------
# inputs

def _inputs(case, seed):
    """The raw inputs of a case, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = torch.device("cuda")
    dt = torch.bfloat16 if case.get("dtype", "bf16") == "bf16" else torch.float32
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)
    if case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        x = 2.5 * rnd(rows, vocab)
        peak = torch.randint(0, vocab, (rows, 3), generator=g, device=dev)
        x.scatter_add_(1, peak, 9.0 + 2.0 * rnd(rows, 3))
        if case["masked"]:
            x.masked_fill_(torch.rand(rows, vocab, generator=g, device=dev) < 0.3, -math.inf)
        alt = torch.randint(0, vocab, (rows,), generator=g, device=dev)
        targets = torch.where(torch.rand(rows, generator=g, device=dev) < 0.7, peak[:, 0], alt).to(torch.int32)
        return dict(logits=x.to(dt), targets=targets)
    new, lens = _sizes(case)
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    pages = [(n + l + page - 1) // page for n, l in zip(new, lens)]
    n_pages = sum(pages) + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((case["batch"], max(pages)), 0, dtype=torch.int32, device=dev)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p]
        at += p
    cu = torch.tensor([0] + [sum(new[:b + 1]) for b in range(len(new))], dtype=torch.int32, device=dev)
    s = dict(table=table, n_pages=n_pages, cu=cu, lengths=torch.tensor(lens, dtype=torch.int32, device=dev),
             n_tokens=sum(new), max_tokens=max(new))
    chan = 1.0 + 5.0 * (torch.rand(hkv, hd, generator=g, device=dev) < 0.03)  # channels of large keys
    if case["op"] == "append":
        n = s["n_tokens"]
        s.update(q=(1.5 * rnd(n, hq, hd)).to(dt), k=(rnd(n, hkv, hd) * chan).to(dt), v=(0.7 * rnd(n, hkv, hd)).to(dt))
        if case["norm"]:
            s.update(q_norm=(1 + 0.1 * rnd(hd)).to(torch.bfloat16), k_norm=(1 + 0.1 * rnd(hd)).to(torch.bfloat16))
        if case["rot"]:
            far = max(n_ + l for n_, l in zip(new, lens))
            inv = 1e6 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
            a = torch.arange(far, dtype=torch.float64, device=dev)[:, None] * inv
            s["rope"] = torch.stack([a.cos(), a.sin()], -1).float().contiguous()  # the table a server keeps
        return s
    # the stored rows of every sequence, one after another (history, and under a causal mask the new tokens')
    held = [l + n if case["causal"] else l for n, l in zip(new, lens)]
    t = max(1, sum(held))
    s.update(held=held, k=(rnd(t, hkv, hd) * chan).to(torch.bfloat16), v=rnd(t, hkv, hd).to(torch.bfloat16))
    q = rnd(s["n_tokens"], hkv, hq // hkv, hd)
    # each query leans on one stored key
    pick = torch.randint(0, t, (s["n_tokens"],), generator=g, device=dev)
    q = 0.7 * q + 0.25 * s["k"][pick].float()[:, :, None, :]
    s["q"] = q.reshape(s["n_tokens"], hq, hd).to(torch.bfloat16)
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


def _where(state, lens, rows):
    """(page, offset in the page) of `rows` consecutive rows that cu divides among the sequences."""
    seq = torch.searchsorted(state["cu"][1:], torch.arange(rows, dtype=torch.int32, device="cuda"), right=True)
    pos = lens[seq] + torch.arange(rows, device="cuda") - state["cu"][seq]
    return seq, pos, state["table"][seq, pos // state["page"]].long(), pos % state["page"]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "logprobs":
        return s
    hkv, hd, page = case["hkv"], case["hd"], case["page"]
    s["page"] = page
    s["eps"] = 1e-6
    if own:
        from latency_moe_decode_gb300 import ops
        s["cache"] = ops.KvqCache(s["n_pages"], hkv, hd, page_tokens=page)
    else:
        s["codes"] = torch.zeros(2, s["n_pages"], hkv, page, hd, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(2, s["n_pages"], hkv, page, hd // BLOCK, device="cuda")
    if case["op"] == "attn" and sum(s["held"]):
        cu = torch.tensor([0] + [sum(s["held"][:b + 1]) for b in range(len(s["held"]))], dtype=torch.int32, device="cuda")
        zero = torch.zeros_like(s["lengths"])
        if own:
            s["cache"].append(s["k"], s["v"], zero, s["table"], cu_tokens=cu)
        else:
            _, _, at, off = _where({"cu": cu, "table": s["table"], "page": page}, zero, s["k"].shape[0])
            for i, x in enumerate((s["k"], s["v"])):
                s["codes"][i][at, :, off], s["scales"][i][at, :, off] = _quantise(x)
    for k in ("k", "v", "held") if case["op"] == "attn" else ():
        del s[k]
    return s


# ---------------------------------------------------------------------------------------------
# the operators

def _norm_rotate(x, w, s, pos, rot, inter):
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * w.double()
    if rot:
        c, d = s["rope"][pos].double().unbind(-1)
        c, d = c[:, None], d[:, None]
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
        y = torch.stack([a * c - b * d, a * d + b * c], -1 if inter else -2).flatten(-2)
        x = torch.cat([y, x[..., rot:]], -1)
    return x


def _append(s):
    c = s["case"]
    _, pos, at, off = _where(s, s["lengths"], s["n_tokens"])
    q = _norm_rotate(s["q"], s.get("q_norm"), s, pos, c["rot"], c["inter"])
    k = _norm_rotate(s["k"], s.get("k_norm"), s, pos, c["rot"], c["inter"])
    got = []
    for i, x in enumerate((k, s["v"])):
        s["codes"][i][at, :, off], s["scales"][i][at, :, off] = _quantise(x)
        got.append((s["codes"][i][at, :, off] * s["scales"][i][at, :, off].repeat_interleave(BLOCK, -1)).to(torch.bfloat16))
    return {"q": q.to(torch.bfloat16), "k": got[0], "v": got[1]}


def _attention(s):
    c = s["case"]
    hkv, hd, group = c["hkv"], c["hd"], c["hq"] // c["hkv"]
    n, most = s["n_tokens"], s["max_tokens"]
    held = [(s["codes"][i][s["table"].long()].float() * s["scales"][i][s["table"].long()].repeat_interleave(BLOCK, -1))
            .transpose(1, 2).flatten(2, 3) for i in (0, 1)]  # [batch, hkv, positions, hd]
    seq = torch.searchsorted(s["cu"][1:], torch.arange(n, dtype=torch.int32, device="cuda"), right=True)
    j = torch.arange(n, device="cuda") - s["cu"][seq]
    q = torch.zeros(c["batch"], most, hkv, group, hd, device="cuda")
    q[seq, j] = s["q"].float().view(n, hkv, group, hd)
    x = torch.einsum("bjhgd,bhpd->bhgjp", q, held[0]) / math.sqrt(hd)
    last = s["lengths"][:, None] + (torch.arange(1, most + 1, device="cuda") if c["causal"] else torch.zeros(most, device="cuda"))
    hide = torch.arange(x.shape[-1], device="cuda") >= last[..., None]  # [batch, most, positions]
    x = x.masked_fill(hide[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgjp,bhpd->bjhgd", p / total.clamp(min=1e-30), held[1])
    lse = (m + total.log()).squeeze(-1).permute(0, 3, 1, 2)
    return {"out": o[seq, j].flatten(1, 2).to(torch.bfloat16), "lse": lse[seq, j].flatten(1)}


def _logprobs(s):
    x = s["logits"].float()
    top = s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    lse = m + total.log()
    t = s["targets"].long()[:, None]
    xt = x.gather(1, t)
    ahead = (x > xt) | ((x == xt) & (torch.arange(x.shape[1], device="cuda") < t))
    out = {"logprob": (xt - lse).squeeze(1), "rank": ahead.sum(-1).to(torch.int32),
           "entropy": (lse - (e * x.masked_fill(e == 0, 0.0)).sum(-1, keepdim=True) / total).squeeze(1)}
    if top:
        v, i = torch.sort(x, dim=1, descending=True, stable=True)
        out.update(top_ids=i[:, :top].to(torch.int32), top_logprobs=v[:, :top] - lse)
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _append, "attn": _attention, "logprobs": _logprobs}[c["op"]](s)
    if c["op"] == "append":
        q = s["cache"].append(s["k"], s["v"], s["lengths"], s["table"], cu_tokens=s["cu"], q=s["q"],
                              q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=s["eps"], rope=s.get("rope"),
                              interleaved=c["inter"])
        k, v = s["cache"].gather(s["lengths"], s["table"], s["n_tokens"], cu_tokens=s["cu"])
        return {"q": q, "k": k, "v": v}
    if c["op"] == "attn":
        out, lse = s["cache"].attention(s["q"], s["lengths"], s["table"], cu_tokens=s["cu"], max_tokens=s["max_tokens"],
                                        causal=c["causal"], return_lse=True)
        return {"out": out, "lse": lse}
    from latency_moe_decode_gb300 import ops
    r = ops.logprobs(s["logits"], s["targets"], top_n=c["top"])
    out = {"logprob": r.logprob, "rank": r.rank, "entropy": r.entropy}
    if c["top"]:
        out.update(top_ids=r.top_ids, top_logprobs=r.top_logprobs)
    return out


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


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "logprobs":
        rows = {"logprob": [], "rank": [], "entropy": [], "top_ids": [], "top_logprobs": []}
        for x, t in zip(s["logits"].double().split(64), s["targets"].long().split(64)):
            lp = x - torch.logsumexp(x, 1, keepdim=True)
            order = torch.argsort(x, dim=1, descending=True, stable=True)
            rows["logprob"].append(lp.gather(1, t[:, None])[:, 0])
            rows["rank"].append((order == t[:, None]).int().argmax(1).to(torch.int32))
            rows["entropy"].append(-torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(1))
            rows["top_ids"].append(order[:, :case["top"]].to(torch.int32))
            rows["top_logprobs"].append(lp.gather(1, order[:, :case["top"]]))
        out = {k: torch.cat(v) for k, v in rows.items()}
        return out if case["top"] else {k: out[k] for k in ("logprob", "rank", "entropy")}
    new, lens = _sizes(case)
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    if case["op"] == "append":
        rot = case["rot"]
        pos = torch.cat([torch.arange(l, l + n, device="cuda") for n, l in zip(new, lens)])

        def turned(x, w):
            x = x.double()
            if w is not None:
                x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / hd + 1e-6) * w.double()
            x = x.clone()
            if rot:
                ang = s["rope"][pos].double()  # the table is an input
                z = torch.complex(ang[..., 0], ang[..., 1])[:, None]
                i = torch.arange(rot // 2, device="cuda")
                a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
                y = torch.complex(x[..., a], x[..., b]) * z
                x[..., a], x[..., b] = y.real, y.imag
            return x

        return {"q": turned(s["q"], s.get("q_norm")), "k": _stored(turned(s["k"], s.get("k_norm"))), "v": _stored(s["v"])}
    outs, lses = [], []
    k, v, q = _stored(s["k"]), _stored(s["v"]), s["q"].double()
    at = row = 0
    for n, l, held in zip(new, lens, s["held"]):
        kk = k[at:at + held].repeat_interleave(hq // hkv, 1).permute(1, 2, 0)
        vv = v[at:at + held].repeat_interleave(hq // hkv, 1).transpose(0, 1)
        for j0 in range(0, n, 64):
            j = torch.arange(j0, min(n, j0 + 64), device="cuda")
            x = torch.matmul(q[row + j].transpose(0, 1), kk) * hd ** -0.5
            if case["causal"]:
                x = torch.where(torch.arange(held, device="cuda")[None] <= l + j[:, None], x, -math.inf)
            lses.append(torch.logsumexp(x, -1).T if held else torch.full((len(j), hq), -math.inf, dtype=torch.float64, device="cuda"))
            outs.append(torch.matmul(torch.softmax(x, -1), vv).transpose(0, 1))
        at += held
        row += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
