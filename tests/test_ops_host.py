"""Host-side checks of the operators' C entry points (no GPU needed): what they refuse before they
touch a device, with its reason, and the sizes they report."""
import ctypes as C

import pytest

from latency_moe_decode_gb300 import build, capi
from latency_moe_decode_gb300.capi import (DecKvqAppendArgs, DecKvqAttentionArgs, DecKvqCache, DecKvqSeqs,
                                           DecLogprobsArgs, DecRows)

ARG, UNSUPPORTED = -1, -5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


def _cache(**kw):
    d = dict(pages=4096, n_pages=4, page_tokens=64, n_kv_heads=2, head_dim=128, status=None)
    d.update(kw)
    return DecKvqCache(**d)


def _seqs(**kw):
    d = dict(batch=1, n_tokens=1, cu_tokens=None, lengths=4096, table=4096, max_pages=4, table_stride=4)
    d.update(kw)
    return DecKvqSeqs(**d)


def _r(**kw):
    d = dict(p=4096, token_stride=1024, head_stride=128)
    d.update(kw)
    return DecRows(**d)


def _flat(d):
    """dec_rows members as the structures' own fields."""
    return {k2: v2 for k, v in d.items() for k2, v2 in (
        [(k, v.p), (k + "_token_stride", v.token_stride), (k + "_head_stride", v.head_stride)]
        if isinstance(v, DecRows) else [(k, v)])}


def _append(**kw):
    d = dict(dtype=0, n_heads=8, q=_r(), k=_r(), v=_r(), q_out=_r(), eps=1e-6)
    d.update(kw)
    return DecKvqAppendArgs(**_flat(d))


def _attn(**kw):
    d = dict(n_heads=8, q=_r(), out=_r(), max_tokens=1, causal=1)
    d.update(kw)
    return DecKvqAttentionArgs(**_flat(d))


def test_page_bytes(lib):
    f = lib.dec_kvq_page_bytes
    assert f(64, 8, 128) == 64 * 8 * 2 * (64 + 8)
    assert f(16, 1, 64) == 16 * 2 * (32 + 4)
    for bad in ((48, 8, 128), (8, 8, 128), (512, 8, 128), (64, 0, 128), (64, 1025, 128), (64, 8, 96), (-64, 8, 128)):
        assert f(*bad) == 0


@pytest.mark.parametrize("cache,status", [
    (None, ARG), (dict(pages=None), ARG), (dict(n_pages=0), ARG), (dict(head_dim=96), UNSUPPORTED),
    (dict(page_tokens=24), UNSUPPORTED), (dict(n_kv_heads=0), ARG), (dict(n_kv_heads=2000), UNSUPPORTED),
    (dict(pages=4100), ARG)])
def test_caches_are_checked(lib, cache, status):
    c = None if cache is None else _cache(**cache)
    assert lib.dec_kvq_append(c, _seqs(), _append(), None) == status
    assert lib.dec_op_error()
    assert lib.dec_kvq_attention(c, _seqs(), _attn(), None) == status
    assert lib.dec_kvq_gather(c, _seqs(), _r(), _r(), None) == status


@pytest.mark.parametrize("seqs", [None, dict(batch=-1), dict(n_tokens=-1), dict(n_tokens=2), dict(lengths=None),
                                  dict(table=None), dict(max_pages=0), dict(max_pages=-1), dict(table_stride=-4)])
def test_sequences_are_checked(lib, seqs):
    s = None if seqs is None else _seqs(**seqs)
    assert lib.dec_kvq_append(_cache(), s, _append(), None) == ARG
    assert lib.dec_kvq_attention(_cache(), s, _attn(), None) == ARG
    assert lib.dec_kvq_gather(_cache(), s, _r(), _r(), None) == ARG
    assert b"sequences" in lib.dec_op_error()


def test_page_tables_beyond_32_bits_are_refused(lib):
    assert lib.dec_kvq_attention(_cache(), _seqs(max_pages=1 << 26), _attn(), None) == UNSUPPORTED


@pytest.mark.parametrize("args", [
    None, dict(dtype=2), dict(n_heads=0), dict(q=_r(p=None)), dict(k=_r(p=None)), dict(v=_r(p=4098)),
    dict(k=_r(token_stride=130)), dict(q=_r(head_stride=4)), dict(q_out=_r(p=None)), dict(rotary_dim=24, rope=4096),
    dict(rotary_dim=256, rope=4096), dict(rotary_dim=64), dict(rope=4096), dict(rotary_dim=64, rope=4100),
    dict(eps=-1.0), dict(eps=float("nan")), dict(q_norm=4098), dict(k_norm=4104)])
def test_append_arguments_are_checked(lib, args):
    assert lib.dec_kvq_append(_cache(), _seqs(), None if args is None else _append(**args), None) == ARG


@pytest.mark.parametrize("args", [
    None, dict(n_heads=0), dict(n_heads=7), dict(max_tokens=-1), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(q=_r(p=None)), dict(out=_r(token_stride=12)), dict(q=_r(p=4104))])
def test_attention_arguments_are_checked(lib, args):
    assert lib.dec_kvq_attention(_cache(), _seqs(), None if args is None else _attn(**args), None) == ARG


def test_nothing_to_do(lib):
    s = _seqs(batch=0, n_tokens=0, lengths=None, table=None)
    assert lib.dec_kvq_append(_cache(), s, _append(), None) == 0
    assert lib.dec_kvq_attention(_cache(), s, _attn(), None) == 0
    assert lib.dec_kvq_gather(_cache(), s, _r(), _r(), None) == 0
    assert lib.dec_op_error() == b""


def test_readable_copies_odd_strides():
    import torch
    from latency_moe_decode_gb300 import ops
    b = torch.arange(5000).to(torch.bfloat16)
    for t in (torch.as_strided(b, (1, 8, 128), (1027, 128, 1)), torch.as_strided(b, (2, 8, 128), (1027, 128, 1)),
              b[1:1025].view(1, 8, 128), torch.as_strided(b, (2, 4, 128), (1024, 256, 2))):
        r = ops._readable(t)
        assert torch.equal(r, t) and all(x % 8 == 0 for x in r.stride()[:2]) and r.stride(2) == 1 and r.data_ptr() % 16 == 0
    t = b[:2048].view(2, 8, 128)
    assert ops._readable(t) is t


def test_workspace_sizes(lib):
    w = lib.dec_kvq_attention_workspace
    for bad in (dict(head_dim=96), dict(page_tokens=3), dict(n_kv_heads=0)):
        assert w(_cache(**bad), 8, 1, 1) == -1
    assert w(_cache(), 7, 1, 1) == -1 and w(_cache(), 8, -1, 1) == -1 and w(None, 8, 1, 1) == -1


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(rows=-1), dict(vocab=0), dict(row_stride=-1), dict(top_n=-1),
                                dict(top_n=33), dict(top_n=11, vocab=10), dict(logprob=4096), dict(rank=4096),
                                dict(logits=None)])
def test_logprobs_arguments_are_checked(lib, kw):
    d = dict(logits=4096, dtype=1, rows=1, vocab=100, row_stride=100, entropy=4096)
    d.update(kw)
    assert lib.dec_logprobs(DecLogprobsArgs(**d), None) == ARG
    assert b"logprobs" in lib.dec_op_error()


def test_logprobs_of_no_rows(lib):
    assert lib.dec_logprobs(None, None) == ARG
    assert lib.dec_logprobs(DecLogprobsArgs(dtype=1, rows=0, vocab=10), None) == 0


def test_struct_sizes_match_the_header(lib, tmp_path):
    """The binding's structures have the C compiler's sizes."""
    import os
    import subprocess
    names = {"dec_kvq_cache": DecKvqCache, "dec_kvq_seqs": DecKvqSeqs, "dec_rows": DecRows,
             "dec_kvq_append_args": DecKvqAppendArgs, "dec_kvq_attention_args": DecKvqAttentionArgs,
             "dec_logprobs_args": DecLogprobsArgs, "dec_step_kvq_args": capi.DecStepKvqArgs,
             "dec_score_args": capi.DecScoreArgs}
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "dec.h"\nint main(void) {' +
                   "".join(f'printf("%d\\n", (int)sizeof({n}));' for n in names) + "return 0; }")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-o", str(tmp_path / "s"), str(src)], check=True)
    got = subprocess.run([str(tmp_path / "s")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == [C.sizeof(t) for t in names.values()]


def test_engine_entry_points_reject_null(lib):
    assert lib.dec_step_kvq(None, None) == ARG
    assert lib.dec_kvq_store(None, 0, None, None, 0) == ARG
    assert lib.dec_kvq_load(None, 0, None, None, 0, 0) == ARG
    assert lib.dec_score(None, None) == ARG
