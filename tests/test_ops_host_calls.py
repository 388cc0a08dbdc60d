"""What the Python bindings hand to the library, without a GPU."""
import os
import subprocess
import sys
import types

import pytest
import torch

from latency_moe_decode_gb300 import build, capi, ops
from latency_moe_decode_gb300.engine import Engine


def _engine(lib):
    e = object.__new__(Engine)
    e.lib, e.h, e.cfg = lib, None, types.SimpleNamespace(n_layers=1)
    return e


def _cache():
    c = object.__new__(ops.KvqCache)
    c.c, c.device = ops.DecKvqCache(), torch.device("cpu")
    return c


def test_moving_slots_is_queued_on_the_callers_stream():
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, a)) or 0

    eng, table = _engine(Lib()), torch.zeros(3, dtype=torch.int32)
    eng.kvq_store(2, [_cache()], table, stream=4096)
    eng.kvq_load(2, [_cache()], table, 33, stream=0)  # (torch's default stream: not the engine's own)
    assert [c[0] for c in calls] == ["dec_kvq_store_ex", "dec_kvq_load_ex"]
    assert calls[0][1][-1] == 4096 and calls[1][1][-2:] == (33, 1)


def test_appending_nothing_with_queries_of_no_address():
    """An empty tensor has no address: rows of nothing are no error, with queries or without."""
    build.build()
    lib = capi.lib()
    cache = capi.DecKvqCache(4096, 4, 64, 2, 128, None)
    none = dict(dtype=0, k=None, v=None, eps=1e-6)
    for batch, cu in ((0, None), (2, 4096)):
        seqs = capi.DecKvqSeqs(batch, 0, cu, 4096, 4096, 4, 4)
        for heads in (0, 8):
            assert lib.dec_kvq_append(cache, seqs, capi.DecKvqAppendArgs(n_heads=heads, **none), None) == 0
        assert lib.dec_kvq_append(cache, seqs, capi.DecKvqAppendArgs(n_heads=-1, **none), None) == -1
    # with rows, queries still have to be there
    one = capi.DecKvqSeqs(1, 1, None, 4096, 4096, 4, 4)
    assert lib.dec_kvq_append(cache, one, capi.DecKvqAppendArgs(n_heads=8, dtype=0, k=4096, v=4096, eps=1e-6), None) == -1
    assert b"n_heads goes with q" in lib.dec_op_error()


def test_imports_with_a_torch_without_cuda():
    """A torch built without CUDA lacks the short cut to a stream's handle; importing asks for none of it."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "from latency_moe_decode_gb300 import engine, ops\n"
            "torch.cuda.current_stream = lambda i: type('S', (), {'cuda_stream': 40 + i})\n"
            "print(ops._raw_stream(2))\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["42"]


def test_streams_belong_to_the_tensors_device(monkeypatch):
    """With another device than the tensors' current, a raw handle is a stream of the tensors' device; a torch
    stream of another device is refused (the call would run unordered with it)."""
    class Stream:
        def __init__(self, handle, device=None):
            self.handle, self.device = handle, torch.device("cuda:0") if device is None else device

    used = []
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", used.append)
    one = torch.device("cuda:1")
    ops._on_stream(4096, one)
    ops._on_stream(Stream(5, one), one)
    assert [(s.handle, s.device) for s in used] == [(4096, one), (5, one)]
    with pytest.raises(ValueError):
        ops._on_stream(Stream(5), one)
    assert len(used) == 2


def test_attention_passes_on_the_likely_rows(monkeypatch):
    """Without max_tokens the bound is all rows, and the kernel goes by the mean; given, it is what counts."""
    build.build()
    calls = []
    monkeypatch.setattr(ops, "_call", lambda f, index, c, s, a: calls.append((s.batch, a.max_tokens, a.likely_tokens)) or 0)
    monkeypatch.setattr(ops.KvqCache, "_seqs", lambda self, lengths, table, cu, n: capi.DecKvqSeqs(lengths.numel(), n))
    cache = object.__new__(ops.KvqCache)
    cache._index, cache.head_dim, cache.n_kv_heads, cache.device, cache.c = -1, 64, 2, torch.device("cpu"), None
    cache._ws = {(4, m): 16 for m in (1, 9, 2, 0)}
    lib = capi.lib()
    cache.lib = lib
    cu, lengths = torch.zeros(5, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(9, 4, 64, dtype=torch.bfloat16)
    cache.attention(q, lengths, None, cu_tokens=cu)
    cache.attention(q, lengths, None, cu_tokens=cu, max_tokens=2)
    cache.attention(q[:4], lengths, None)
    cache.attention(q[:0], lengths[:0], None, cu_tokens=cu[:1])
    assert [c[1:] for c in calls] == [(9, 3), (2, 0), (1, 1), (0, 0)]
    a = capi.DecKvqAttentionArgs(n_heads=8, q=4096, q_token_stride=1024, q_head_stride=128, out=4096, out_token_stride=1024,
                                 out_head_stride=128, max_tokens=1, likely_tokens=-1)
    seqs, c = capi.DecKvqSeqs(1, 1, None, 4096, 4096, 4, 4), capi.DecKvqCache(4096, 4, 64, 2, 128, None)
    assert lib.dec_kvq_attention(c, seqs, a, None) == -1 and b"likely_tokens" in lib.dec_op_error()


def test_rows_whose_ids_would_pass_32_bits_are_refused():
    build.build()
    lib = capi.lib()
    for vocab, refused in ((2 ** 31 - 1, True), (2 ** 31 - 1024, True), (2 ** 31 - 1025, False)):
        a = capi.DecLogprobsArgs(logits=4096, dtype=0, rows=1, vocab=vocab, row_stride=vocab, entropy=4096)
        assert (lib.dec_logprobs(a, None) == -5) == refused


def test_batches_whose_sequences_would_pass_32_bits_are_refused():
    build.build()
    lib = capi.lib()
    cache = capi.DecKvqCache(4096, 4, 64, 2, 128, None)
    rows = capi.DecRows(4096, 256, 128)
    append = capi.DecKvqAppendArgs(dtype=0, k=4096, k_token_stride=256, k_head_stride=128, v=4096, v_token_stride=256,
                                   v_head_stride=128, eps=1e-6)
    attend = capi.DecKvqAttentionArgs(n_heads=2, q=4096, q_token_stride=256, q_head_stride=128, out=4096,
                                      out_token_stride=256, out_head_stride=128, max_tokens=1)
    for batch, refused in ((2 ** 31 - 1, True), (2 ** 31 - 1024, True), (2 ** 31 - 1025, False)):
        seqs = capi.DecKvqSeqs(batch, 1, 4096, 4096, 4096, 4, 4)
        got = [lib.dec_kvq_append(cache, seqs, append, None), lib.dec_kvq_gather(cache, seqs, rows, rows, None)]
        assert [st == -5 for st in got] == [refused] * 2
        assert lib.dec_kvq_attention(cache, seqs, attend, None) == (-5 if refused else -1)  # (no workspace)


def test_calls_on_the_engines_own_stream_wait_for_torchs(monkeypatch):
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(synchronize=lambda: calls.append("wait")))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: empty(*a, dtype=kw["dtype"]))
    eng = _engine(Lib())
    eng.cfg.n_kv_heads, eng.cfg.head_dim = 2, 64
    t = torch.zeros(5, dtype=torch.int32)
    kv = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    eng.prefill_tokens(t)
    eng.prefill_tokens_noalloc(t)
    eng.prefill_import(kv, kv)
    eng.export_kv(0, 0, 0, 3)
    assert calls == ["wait", "dec_prefill_kv", "wait", "dec_prefill_kv_noalloc", "wait", "dec_prefill_kv", "wait", "dec_export_kv"]
