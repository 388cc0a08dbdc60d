"""Moving slots to pages and back (Engine.kvq_store, kvq_load) beside work that is still queued on the
caller's stream: the pages' appends and reads, and the page table itself."""
import numpy as np
import pytest
import torch

import kvq_ref as ref
from latency_moe_decode_gb300 import synth
from tests.test_gpu_parity import _engine, _models
from tests.test_oracle_layer_composition import bfv

pytestmark = pytest.mark.gpu

CFG = synth.TINY.replace(max_batch=4, max_ctx=96)
N, PAGE = 75, 16
BUSY = 200_000_000  # cycles, a tenth of a second: what follows is still queued when the call is made


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _setup():
    eng = _engine(_models(CFG, 2)[1])
    need = (N + PAGE - 1) // PAGE
    caches = eng.kvq_caches(need + 2, PAGE)
    for c in caches:
        c.pages.zero_()
    return eng, caches, [need + 1 - i for i in range(need)]


def _held(eng, slot):
    return [[t.double().cpu().numpy() for t in eng.export_kv(slot, l, 0, N)] for l in range(CFG.n_layers)]


@pytest.mark.parametrize("own_stream", [False, True], ids=["current", "named"])
def test_load_follows_the_appends_and_the_table(own_stream):
    eng, caches, pages = _setup()
    g = torch.Generator().manual_seed(5)
    kv = [[torch.randn(N, CFG.n_kv_heads, CFG.head_dim, generator=g).to(torch.bfloat16) for _ in range(2)] for _ in caches]
    dev = [[t.cuda() for t in p] for p in kv]
    late, zero, cu, table = _ints(pages), _ints([0]), _ints([0, N]), torch.zeros(len(pages), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s if own_stream else torch.cuda.current_stream()):
        torch.cuda._sleep(BUSY)
        table.copy_(late)
        for c, (k, v) in zip(caches, dev):
            c.append(k, v, zero, table[None], cu_tokens=cu)
        if not own_stream:
            eng.kvq_load(1, caches, table, N)
    if own_stream:
        eng.kvq_load(1, caches, table, N, stream=s)
    assert eng.get_length(1) == N
    for (k, v), want in zip(_held(eng, 1), kv):
        for got, x in zip((k, v), want):
            assert np.array_equal(got, ref.store(bfv(x))[0].transpose(1, 0, 2))
    caches[0].check()


@pytest.mark.parametrize("raw", [False, True])
def test_store_follows_the_reads_and_the_table(raw):
    eng, caches, pages = _setup()
    g = torch.Generator().manual_seed(6)
    k0, v0 = (torch.randn(N, CFG.n_kv_heads, CFG.head_dim, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    late, zero, cu = _ints(pages), _ints([0]), _ints([0, N])
    for c in caches:
        c.append(k0, v0, zero, late[None], cu_tokens=cu)
    before = [c.gather(zero, late[None], N, cu_tokens=cu) for c in caches]
    k, v = synth.gen_kv(CFG, N, seed=31)
    eng.prefill_import(k.cuda(), v.cuda(), seq=2)
    table = torch.zeros(len(pages), dtype=torch.int32, device="cuda")
    outs = [tuple(torch.empty_like(t) for t in p) for p in before]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
        table.copy_(late)
        for c, o in zip(caches, outs):
            c.gather(zero, table[None], N, cu_tokens=cu, out=o)
        eng.kvq_store(2, caches, table, **(dict(stream=s.cuda_stream) if raw else {}))
    assert all(torch.equal(a, b) for p, q in zip(before, outs) for a, b in zip(p, q))  # read before they were written over
    for l, c in enumerate(caches):
        for got, x in zip(c.gather(zero, late[None], N, cu_tokens=cu), (k, v)):
            assert np.array_equal(got.double().cpu().numpy(), ref.store(bfv(x[l]))[0].transpose(1, 0, 2))
        assert not c.pages[:c.page_bytes].any()  # page 0, which the table held before it was written
    caches[0].check()


def test_slots_filled_and_read_beside_queued_work():
    """Keys, values and ids that are still being written when a slot is filled from them; a slot read into memory
    that queued work has used."""
    eng, plain = (_engine(_models(CFG, 2)[1]) for _ in range(2))
    k, v = (t.cuda() for t in synth.gen_kv(CFG, N, seed=8))
    ids = synth.gen_tokens(9, CFG.vocab, seed=3).cuda().to(torch.int32)
    plain.prefill_import(k, v, seq=1)
    plain.prefill_tokens(ids, seq=2)
    plain.prefill_tokens_noalloc(ids, seq=3)
    late = [torch.zeros_like(t) for t in (k, v, ids)]
    torch.cuda.synchronize()

    def fill():
        for t in late:
            t.zero_()
        torch.cuda._sleep(BUSY)
        for t, x in zip(late, (k, v, ids)):
            t.copy_(x)

    fill()
    eng.prefill_import(late[0], late[1], seq=1)
    fill()
    eng.prefill_tokens(late[2], seq=2)
    fill()
    eng.prefill_tokens_noalloc(late[2], seq=3)
    for seq, n in ((1, N), (2, 9), (3, 9)):
        for l in range(CFG.n_layers):
            torch.cuda._sleep(BUSY // 10)
            used = torch.empty(2, CFG.n_kv_heads, n, CFG.head_dim, dtype=torch.bfloat16, device="cuda")
            used.fill_(7.0)  # queued; its memory goes to the next outputs
            del used
            got = eng.export_kv(seq, l, 0, n)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, plain.export_kv(seq, l, 0, n)))
