"""Per-layer times of steps over paged 4-bit caches."""
import numpy as np
import pytest
import torch

from latency_moe_decode_gb300 import synth
from tests.test_gpu_parity import MOE_SMALL, _engine, _models

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cfg", [synth.TINY.replace(max_batch=16, max_ctx=64), MOE_SMALL.replace(max_batch=16, max_ctx=64)],
                         ids=["dense", "moe"])
def test_layer_times_are_of_the_latest_step(cfg):
    eng = _engine(_models(cfg, 1)[1])
    caches = eng.kvq_caches(8, 16)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    tok, table, nxt = ints([1, 2, 3]), ints([[0, 1], [2, 3], [4, 5]]), ints([0, 0, 0])
    seen = [np.zeros(1, np.uint64)]
    for i in range(4):
        if i == 2:  # another kind of step between
            eng.step(tokens=tok, next_tokens=nxt)
        else:
            eng.step_kvq(caches, ints([i, i, i]), table, tokens=tok, next_tokens=nxt)
        t = np.asarray(eng.layer_times(), np.uint64)
        assert len(t) == cfg.n_layers + 2
        assert (np.diff(t.astype(np.int64)) > 0).all() and t[0] > seen[-1][-1], (i, t, seen[-1])
        seen.append(t)
    caches[0].check()
