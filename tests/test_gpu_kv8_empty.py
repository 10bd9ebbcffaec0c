"""Batches without sequences, pools without pages."""
import pytest

from kv8_ref import torch

pytestmark = pytest.mark.gpu


def test_a_batch_without_sequences():
    """Nothing to do is no error, for the store as for the attention."""
    import persistent_runtime_b200 as prb
    t = torch()
    cache = prb.KV8Cache.empty(4, 1, 2, 64, 32, 16)
    table = t.zeros(0, 3, dtype=t.int32, device="cuda")
    lens = t.zeros(0, dtype=t.int32, device="cuda")
    start = t.zeros(1, dtype=t.int32, device="cuda")
    q = t.zeros(0, 4, 64, dtype=t.bfloat16, device="cuda")
    side = t.cuda.Stream()
    for kw in ({}, {"row_start": start}, {"stream": side}):
        cache.store(0, q[:, :2], q[:, :2], table, lens, **kw)
        if "row_start" in kw:
            kw["max_rows"] = 3
        out, lse = cache.attention(0, q, table, lens, return_lse=True, **kw)
        assert out.shape == (0, 4, 64) and out.dtype == t.bfloat16 and lse.shape == (0, 4)
    cache.check()
    # rows that no sequence could own are refused, as before
    some = t.zeros(2, 4, 64, dtype=t.bfloat16, device="cuda")
    with pytest.raises(prb.MkError):
        cache.attention(0, some, table, lens)
    with pytest.raises(prb.MkError):
        cache.attention(0, some, table, lens, row_start=start, max_rows=1)
    with pytest.raises(prb.MkError):
        cache.store(0, some[:, :2], some[:, :2], table, lens, row_start=start)


def test_pools_without_pages_are_refused():
    import persistent_runtime_b200 as prb
    t = torch()
    none, table = t.zeros(0, dtype=t.int32, device="cuda"), t.zeros(2, 2, dtype=t.int32, device="cuda")
    for pools in ([], [t.zeros(0, 4, device="cuda")]):
        with pytest.raises(prb.MkError):
            prb.PagePool(table, none, 16, pools)
    with pytest.raises(prb.MkError):
        prb.PagePool.empty(2, 2, 16, [])
    with pytest.raises(prb.MkError):
        prb.PagePool.empty(2, 2, 16, [t.zeros(0, 4, device="cuda")])
