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
