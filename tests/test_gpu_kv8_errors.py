"""A refused call leaves nothing behind that a later call would report as its own failure."""
import ctypes

import numpy as np
import pytest

from kv8_ref import dev, torch

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("built_libs")]


def test_a_device_that_does_not_exist():
    import persistent_runtime_b200 as prb
    import synth
    from gpu_helpers import dev_weights
    L, ref, A, none = prb.lib(), ctypes.byref, 1 << 20, 1 << 12  # the address is never read
    w = synth.TINY.with_(name="tiny-b2", batch=2, kv_len=0, steps=1)
    weights = dev_weights(synth.make_weights(w, 8))
    cache = prb.Kv8Cache(none, prb.MK_KV8_INT8, 2, 2, 64, 64, 32, 10, A, A, A, A, None)
    batch, rows, size = prb.Batch(3, 3, 1, 100, None, A, A), prb.Rows(A, prb.MK_BF16, 128, 64), ctypes.c_int64()
    pages = prb.Pages(none, 10, 3, 4, 64, 0)
    pages.d_page_table = pages.d_ref = A
    calls = {"store": lambda: L.mk_kv8_store(ref(cache), 0, ref(rows), ref(rows), ref(batch), None),
             "attention": lambda: L.mk_kv8_attention(ref(cache), 0, ref(rows), 4, 1.0, A, None, ref(batch), A, 1 << 40, None),
             "free": lambda: L.mk_pages_free(ref(pages), 1, A, A, 1 << 40, None),
             "reserve": lambda: L.mk_pages_reserve(ref(pages), A, A, A, 1 << 40, None)}
    mk = prb.Megakernel(w, 64, 0)
    for name, call in calls.items():
        assert call() == prb.MK_ERR_CUDA, name
        assert "device" in L.mk_last_error(None).decode(), name
        mk.load_weights(weights)  # its launches ask for CUDA's last error
    # the size alone needs no device
    assert L.mk_kv8_attention_workspace(ref(cache), 4, prb.MK_BF16, ref(batch), ref(size)) == prb.MK_OK
    mk.load_weights(weights)
    t = torch()
    k, v = (t.zeros(w.n_layers, 2, w.n_kv_heads, 64, w.head_dim, dtype=t.int16, device="cuda") for _ in range(2))
    tok = dev(np.array([3, 4], np.int32))
    mk.decode_step(tok, tok, dev(np.zeros(2, np.int32)), k, v)
    assert mk.sync_status()[0] == 0
    mk.close()
