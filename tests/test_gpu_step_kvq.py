"""The engine over paged 4-bit caches (dec_step_kvq, dec_kvq_store, dec_kvq_load) against the 64-bit
restatement of a decode step whose cache holds every key and value as the 4-bit cache does, and
dec_score against the logits of the engine's own steps."""
import numpy as np
import pytest
import torch

import kvq_ref as ref
from latency_moe_decode_gb300 import synth
from tests.parity import HIDDEN_REL_L2, LOGIT_MAX_ABS, ROUTER_LOGIT_ABS, bf16_to_f64, oracle_logits, rel_l2, t_bits, topk_of
from tests.test_gpu_parity import MOE_SMALL, _engine, _models
from tests.test_oracle_layer_composition import Restated, bf16, bfv

pytestmark = pytest.mark.gpu

MOE = MOE_SMALL.replace(max_batch=20, max_ctx=160)
DENSE = synth.TINY.replace(max_batch=24, max_ctx=96)


class RestatedHeld(Restated):
    """The restated step over a cache that holds the rotated keys and the values in 4 bits, rounded
    once, from what the projections give (the bf16 cache's rounding does not come between). held(l)
    gives the rows that the engine's cache holds at this position: they have to be a right rounding
    of this step's own, and the attention then sees them as they are. (Both sides decide codes from
    their own sums; a layer's input that rounds the other way in a few elements moves a few codes,
    which at a context of one or two positions would be most of what is compared.)"""

    @staticmethod
    def check_held(got, want):
        """Half a step of the run's scale (a neighbouring scale's, one eighth larger), and what the
        layer's input may be off by: HIDDEN_REL_L2 of the row's norm, spread over its elements."""
        s = ref.store(want)[1] * 1.125
        off = HIDDEN_REL_L2 * np.linalg.norm(want, axis=-1, keepdims=True)
        assert (np.abs(got - want) <= s / 2 + off).all()

    def step(self, kv, pos, token, held):
        c = self.c
        hd, hq, hkv = c.head_dim, c.n_heads, c.n_kv_heads
        x = self.embed[token].copy()
        routes = []
        for l, W in enumerate(self.L):
            xn = self.rmsnorm(x, W["attn_norm"])
            q = bf16(self.rope((W["wq"] @ xn).reshape(hq, hd), pos))
            kv["k"][l, :, pos], kv["v"][l, :, pos] = held(l)
            self.check_held(kv["k"][l, :, pos], self.rope((W["wk"] @ xn).reshape(hkv, hd), pos))
            self.check_held(kv["v"][l, :, pos], (W["wv"] @ xn).reshape(hkv, hd))
            o = ref.attend(q, kv["k"][l].transpose(1, 0, 2), kv["v"][l].transpose(1, 0, 2), hd ** -0.5, pos + 1)[0]
            x = bf16(x + W["wo"] @ bf16(o.reshape(-1)))
            xn = self.rmsnorm(x, W["ffn_norm"])
            if c.dense_ffn:
                y = self.swiglu(W["ffn"], xn)
            else:
                sc = 1.0 / (1.0 + np.exp(-(W["router"] @ xn)))
                idx = np.argsort(-sc, kind="stable")[: c.top_k]
                routes.append((idx, sc))
                y = sum(g * self.swiglu(W["experts"][e], xn) for g, e in zip(sc[idx] / sc[idx].sum(), idx))
                y = y + sum(self.swiglu(e, xn) for e in W["shared"])
            x = bf16(x + y)
        return x, self.lm @ self.rmsnorm(x, self.final_norm), routes


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(lens, page, spare, seed):
    """Pages in random order for sequences of up to `lens` positions."""
    need = [(n + page - 1) // page for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare)
    t = np.zeros((len(lens), max(need)), np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t).cuda(), sum(need) + spare


def _setup(cfg, batch, seed, page):
    """Histories in the engine's slots, stored to pages; the restated caches hold what the pages do."""
    m_cpu, m_gpu = _models(cfg, seed)
    eng = _engine(m_gpu)
    lens = [(11 + 23 * b) % (cfg.max_ctx - 8) for b in range(batch)]
    lens[0] = 0
    table, n_pages = _tables([l + 4 for l in lens], page, 3, seed)
    caches = eng.kvq_caches(n_pages, page)
    kvs = []
    for b in range(batch):
        k, v = synth.gen_kv(cfg, max(1, lens[b]), seed=900 + b)
        kv = {n: np.zeros((cfg.n_layers, cfg.n_kv_heads, cfg.max_ctx, cfg.head_dim)) for n in ("k", "v")}
        if lens[b]:
            eng.prefill_import(k.cuda(), v.cuda(), seq=b)
            kv["k"][:, :, :lens[b]], kv["v"][:, :, :lens[b]] = ref.store(bfv(k))[0], ref.store(bfv(v))[0]
        eng.kvq_store(b, caches, table[b].contiguous())
        kvs.append(kv)
    caches[0].check()
    return m_cpu, eng, caches, table, lens, kvs


def _same_route(gpu_idx, gpu_logits, idx, scores, k, layer):
    """Whether the engine selected the reference's experts; if not, they have to score alike. Layer 0's
    router sees matched inputs: ROUTER_LOGIT_ABS. A later layer's input may be off by HIDDEN_REL_L2, that
    is 1e-2 sqrt(512) = 0.23 in norm after its RMSNorm, against router rows of N(0, 0.02): 4.5e-3 a
    logit, and 2e-2 is 4.4 of them."""
    off = ROUTER_LOGIT_ABS if layer == 0 else 2e-2
    want = oracle_logits(scores)
    assert list(topk_of(gpu_logits, k)) == [int(x) for x in gpu_idx[:k]]
    assert np.abs(gpu_logits - want).max() <= off
    if set(gpu_idx[:k].tolist()) == set(int(x) for x in idx):
        return True
    order = np.sort(want)[::-1]
    assert order[k - 1] - order[k] <= 2 * off
    return False


def _step(eng, caches, lens, table, toks, **kw):
    c = eng.cfg
    n = len(toks)
    logits = torch.empty(n, c.vocab, device="cuda")
    nxt = torch.empty(n, dtype=torch.int32, device="cuda")
    hid = torch.empty(n, c.hidden, dtype=torch.bfloat16, device="cuda")
    eng.step_kvq(caches, _ints(lens), table, tokens=_ints(toks), logits=logits, next_tokens=nxt, hidden_out=hid, **kw)
    eng.sync()
    caches[0].check()
    return logits.double().cpu().numpy(), nxt.cpu().numpy(), bf16_to_f64(t_bits(hid))


@pytest.mark.parametrize("cfg,batch,page", [(DENSE, 24, 16), (DENSE, 1, 64), (MOE, 1, 32), (MOE, 5, 64), (MOE, 20, 16)],
                         ids=["dense24", "dense1", "moe1", "moe5", "moe20"])
def test_steps_match_the_restatement(cfg, batch, page):
    m_cpu, eng, caches, table, lens, kvs = _setup(cfg, batch, 3, page)
    rs = RestatedHeld(m_cpu)
    toks = synth.gen_tokens(batch, cfg.vocab, seed=60 + batch).tolist()
    before = eng.info()["launches"]
    routed = flipped = 0
    for i in range(2):
        lg, nx, hid = _step(eng, caches, lens, table, toks)
        routes = [(eng.routing(l)[0], eng.router_logits(l)) for l in range(cfg.n_layers)] if cfg.n_experts else []
        for b in range(batch):
            held = lambda l: [t.double().cpu().numpy()[0] for t in caches[l].gather(_ints([lens[b]]), table[b:b + 1], 1)]
            x, logits, want = rs.step(kvs[b], lens[b], toks[b], held)
            # (a selection between experts that score alike is right either way; what follows is not compared)
            same = [_same_route(routes[l][0][b], routes[l][1][b], idx, sc, cfg.top_k, l) for l, (idx, sc) in enumerate(want)]
            routed += len(same)
            flipped += len(same) - sum(same)
            if not all(same):
                continue
            assert rel_l2(hid[b], x) <= HIDDEN_REL_L2, (i, b, rel_l2(hid[b], x))
            off = np.abs(lg[b] - logits).max()
            assert off <= LOGIT_MAX_ABS
            # the greedy token is the first largest of the step's own logits, each within `off`: no other
            # token can lead it by more than twice that
            assert nx[b] == np.argmax(lg[b]) and logits.max() - logits[nx[b]] <= 2 * off
        toks = nx.tolist()
        lens = [l + 1 for l in lens]
    assert flipped <= 0.05 * routed
    assert eng.info()["launches"] - before == 2 * (cfg.n_layers + 1)
    assert all(eng.get_length(b) == lens[b] - 2 for b in range(batch))  # the engine's own slots are untouched


def test_callers_rotation_table_small_engine_and_reruns():
    """An engine of one position per slot decodes far positions with its caller's table, bit for bit as
    the engine whose own table reaches them; a repeated step gives the same bits."""
    from latency_moe_decode_gb300 import ops
    cfg = DENSE
    m_cpu, m_gpu = _models(cfg, 3)
    _, eng, caches, table, lens, _ = _setup(cfg, 6, 3, 16)
    toks = synth.gen_tokens(6, cfg.vocab, seed=8).tolist()
    a = _step(eng, caches, lens, table, toks)
    again = _step(eng, caches, lens, table, toks)
    small = _engine(m_gpu, max_ctx=1, max_batch=6)
    rope = ops.rope_table(cfg.max_ctx, cfg.head_dim, cfg.rope_theta)
    b = _step(small, caches, lens, table, toks, rope=rope)
    for x, y, z in zip(a, b, again):
        assert np.array_equal(x, z)
        # (the two tables are computed by different libraries: cos and sin may differ in the last place)
        assert rel_l2(x, y) <= 2.0 ** -8


def test_store_and_load():
    cfg = DENSE
    m_cpu, eng, caches, table, lens, kvs = _setup(cfg, 7, 5, 32)
    for b in (1, 3, 6):
        eng.kvq_load(10 + b, caches, table[b].contiguous(), lens[b])
        caches[0].check()
        assert eng.get_length(10 + b) == lens[b]
        for l in range(cfg.n_layers):
            k, v = eng.export_kv(10 + b, l, 0, lens[b])
            assert np.array_equal(k.double().cpu().numpy(), kvs[b]["k"][l, :, :lens[b]])
            assert np.array_equal(v.double().cpu().numpy(), kvs[b]["v"][l, :, :lens[b]])


def test_captured_steps_chain_on_the_device():
    """Greedy decoding from a captured graph: the step reads its tokens and lengths from the device."""
    cfg = DENSE
    _, eng, caches, table, lens, _ = _setup(cfg, 5, 7, 16)
    toks = synth.gen_tokens(5, cfg.vocab, seed=9).tolist()
    want, t, ln = [], toks, list(lens)
    for _ in range(3):
        _, nx, _ = _step(eng, caches, ln, table, t)
        want.append(nx)
        t, ln = nx.tolist(), [x + 1 for x in ln]
    s = torch.cuda.Stream()
    tok, dl, nxt = _ints(toks), _ints(lens), torch.empty(5, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        eng.step_kvq(caches, dl, table, tokens=tok, next_tokens=nxt, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        eng.step_kvq(caches, dl, table, tokens=tok, next_tokens=nxt, stream=s)
        tok.copy_(nxt)
        dl += 1
    for w in want:
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(nxt.cpu().numpy(), w)
    eng.sync()
    caches[0].check()


def test_refusals_of_steps_over_caches():
    from latency_moe_decode_gb300 import ops
    from latency_moe_decode_gb300.capi import DecError
    _, eng, caches, table, lens, _ = _setup(DENSE, 5, 7, 16)
    tok = _ints([1, 2, 3, 4, 5])
    other = [ops.KvqCache(8, DENSE.n_kv_heads, 128, 16)] * DENSE.n_layers
    for bad in (lambda: eng.step_kvq(caches[:1], _ints(lens), table, tokens=tok),
                lambda: eng.step_kvq(other, _ints(lens), table, tokens=tok),
                lambda: eng.step_kvq(caches, _ints(lens), table),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=tok[:4]),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=tok.long()),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=tok, next_tokens=tok[:3]),
                lambda: eng.step_kvq(caches, _ints(lens * 6), table.repeat(6, 1), tokens=tok.repeat(6)),
                lambda: eng.step_kvq(caches, _ints(lens), table, tokens=tok, rope=torch.zeros(4, 8, 2, device="cuda")),
                lambda: eng.kvq_store(99, caches, table[0].contiguous()),
                lambda: eng.kvq_load(0, caches, table[0, :1].contiguous(), 60),
                lambda: eng.kvq_load(0, caches, table[0].contiguous(), 10000)):
        with pytest.raises((DecError, ValueError)):
            bad()
    # a bad cache of the last layer is refused before anything is queued
    import ctypes as C
    from latency_moe_decode_gb300.capi import DecKvqCache, DecStepKvqArgs
    pages = [k.pages.clone() for k in caches]
    for field, value in (("pages", None), ("pages", caches[0].c.pages + 8), ("n_pages", 0), ("page_tokens", 24)):
        arr = (DecKvqCache * len(caches))(*[k.c for k in caches])
        setattr(arr[len(caches) - 1], field, value)
        a = DecStepKvqArgs(tok.data_ptr(), None, 5, arr, C.pointer(caches[0]._seqs(_ints(lens), table, None, 5)), None, 0, None,
                           None, None, None)
        assert eng.lib.dec_step_kvq(eng.h, C.byref(a)) == -1
    torch.cuda.synchronize()
    assert all(torch.equal(k.pages, p) for k, p in zip(caches, pages))
    small = _engine(_models(DENSE, 3)[1], max_ctx=16, max_batch=1)  # no wide kernels
    with pytest.raises(DecError) as e:
        small.step_kvq(caches, _ints([0]), table[:1], tokens=_ints([1]))
    assert e.value.status == -5
    eng.step_kvq(caches, _ints([]), table[:0], tokens=_ints([]))
    # a length beyond the table: recorded in the caches, nothing written
    eng.step_kvq(caches, _ints([100000] * 5), table, tokens=tok, rope=ops.rope_table(64, 64, 1e4))
    eng.sync()
    with pytest.raises(DecError):
        caches[0].check()


@pytest.mark.parametrize("n,top_n", [(1, 0), (8, 5), (21, 32)])
def test_score(n, top_n):
    """The log-probabilities of a text, in one call, against the logits of the same positions."""
    cfg = synth.TINY
    _, m_gpu = _models(cfg, 0)
    eng, plain = _engine(m_gpu), _engine(m_gpu)
    text = synth.gen_tokens(n, cfg.vocab, seed=4).cuda()
    r = eng.score(text, top_n=top_n)
    logits = torch.empty(n, cfg.vocab, device="cuda")
    for i in range(0, n, 8):
        m = min(8, n - i)
        plain.step_positions(text[i:i + m], logits=logits[i:i + m])
    plain.sync()
    eng.sync()
    assert eng.get_length(0) == n
    lp = torch.log_softmax(logits.double(), -1)
    nxt = text[1:].long()
    # (as dec_logprobs' own tests: rounded exponentials and sums of a row of 1024)
    tol = 2.0 ** -24 * (16 + 8 * 16 + 32)
    assert (r.logprob[:-1].double() - lp[:-1].gather(1, nxt[:, None])[:, 0]).abs().max().item() <= tol if n > 1 else True
    assert torch.isnan(r.logprob[-1]) and r.rank[-1] == -1
    assert (r.entropy.double() + (lp.exp() * lp).sum(-1)).abs().max().item() <= tol * 8
    if top_n:
        order = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :top_n]
        assert torch.equal(r.top_ids.long(), order)
        assert (r.top_logprobs.double() - lp.gather(1, order)).abs().max().item() <= tol
    want = torch.tensor([3] * n, dtype=torch.int32, device="cuda")
    eng.set_length(0, 0)
    r2 = eng.score(text, targets=want)
    eng.sync()
    assert (r2.logprob.double() - lp[:, 3]).abs().max().item() <= tol
    from latency_moe_decode_gb300.capi import DecError
    with pytest.raises(DecError):
        eng.score(torch.zeros(cfg.max_ctx, dtype=torch.int32, device="cuda"))  # sequence full
    with pytest.raises(DecError):
        eng.score(text, top_n=33)
