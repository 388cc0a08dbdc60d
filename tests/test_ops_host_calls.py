"""What the Python bindings hand to the library, without a GPU."""
import types

import torch

from latency_moe_decode_gb300 import ops
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
