"""Calls at the edges of what the paged 4-bit cache's operators are given."""
import numpy as np
import pytest
import torch

import kvq_ref as ref
from tests.test_gpu_kvq import _cache, _cu, _filled, _ints, _np, _rnd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("batch", [0, 2])
def test_no_rows(batch):
    cache, table = _cache([20, 20], 2, 128, 16)
    pages = cache.pages.clone()
    kv, q = (torch.zeros(0, h, 128, dtype=BF, device="cuda") for h in (2, 8))
    ln, t = _ints([3, 5][:batch]), table[:batch]
    cu = _cu([0] * batch) if batch else None
    for kw in (dict(), dict(q=q), dict(q=q, q_out=torch.empty_like(q))):
        out = cache.append(kv, kv, ln, t, cu_tokens=cu, **kw)
        assert out is None if not kw else out.shape == (0, 8, 128) and out.dtype == BF
    k, v = cache.gather(ln, t, 0, cu_tokens=cu)
    out, lse = cache.attention(q, ln, t, cu_tokens=cu, return_lse=True)
    assert k.shape == v.shape == (0, 2, 128) and out.shape == (0, 8, 128) and lse.shape == (0, 8)
    cache.check()
    assert torch.equal(pages, cache.pages)


@pytest.mark.parametrize("dtype,hd,rot", [(BF, 128, 128), (F32, 64, 32)])
@pytest.mark.parametrize("status", [True, False])
def test_rows_beyond_the_rotation_table_are_not_appended_by_half(dtype, hd, rot, status):
    """Rows inside the page table and beyond the rotation table leave the page and their queries' place as they
    were, values included; rows before it are appended as ever. Also where no status word is kept."""
    from latency_moe_decode_gb300 import ops
    from latency_moe_decode_gb300.capi import DecError
    g = torch.Generator().manual_seed(hd)
    n, hkv, hq, reach = 30, 2, 4, 21
    cache, table = _cache([n], hkv, hd, 16)
    q, k, v = (_rnd(g, n, h, hd, dtype=dtype).cuda() for h in (hq, hkv, hkv))
    ln, rope = _ints([0]), ops.rope_table(n, rot, 1e4)
    cache.append(k, v, ln, table, cu_tokens=_cu([n]), rope=rope)
    k2, v2 = (torch.randn(n, hkv, hd, generator=g).to(dtype).cuda() for _ in range(2))
    if not status:
        cache.c.status = None
    pages = cache.pages.clone()
    out = torch.full((n, hq, hd), 9.0, dtype=BF, device="cuda")
    cache.append(k2[reach:], v2[reach:], _ints([reach]), table, cu_tokens=_cu([n - reach]), q=q[reach:], q_out=out[reach:],
                 rope=rope[:reach])
    assert torch.equal(pages, cache.pages) and (out == 9).all()
    cache.append(k2, v2, ln, table, cu_tokens=_cu([n]), q=q, q_out=out, rope=rope[:reach])
    want = _cache([n], hkv, hd, 16)
    want[0].append(k, v, ln, want[1], cu_tokens=_cu([n]), rope=rope)
    qo = want[0].append(k2[:reach], v2[:reach], ln, want[1], cu_tokens=_cu([reach]), q=q[:reach], rope=rope)
    assert torch.equal(out[:reach], qo) and (out[reach:] == 9).all()
    for a, b in zip(cache.gather(ln, table, n, cu_tokens=_cu([n])), want[0].gather(ln, want[1], n, cu_tokens=_cu([n]))):
        assert torch.equal(a, b)
    if status:
        with pytest.raises(DecError) as e:
            cache.check()
        assert e.value.status == -8
