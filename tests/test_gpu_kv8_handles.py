"""The step over an 8-bit cache runs the same on every kind of handle, and on a given stream."""
import numpy as np
import pytest

import kv8_ref as ref
import synth
from gpu_helpers import dev_weights
from kv8_ref import dev, torch

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("built_libs")]


@pytest.mark.parametrize("batch", [1, 2, 12])
def test_kinds_of_handles(batch):
    import persistent_runtime_b200 as prb
    t = torch()
    w = synth.TINY.with_(name="tiny-kv8", batch=batch, kv_len=600, steps=4)
    weights = dev_weights(synth.make_weights(w, 6))
    table, n_pages = ref.make_table([700] * batch, 64, seed=6)
    host = ref.Cache(n_pages, w.n_layers, w.n_kv_heads, w.head_dim, 64, 64, "int8", 6)
    want = None
    kinds = [{}, dict(kv_page_size=64), dict(dispatch=1), dict(num_workers=37)] + [dict(attn_jit=1)] * (batch > 1)
    for kind in kinds:
        mk = prb.Megakernel(w, 700, 0, **kind)
        mk.load_weights(weights)
        cache, d_table = host.device(), dev(table)
        tok, lens = dev((np.arange(batch) + 3).astype(np.int32)), dev(np.full(batch, 600, np.int32))
        logits, side = t.zeros(batch, w.vocab, device="cuda"), t.cuda.Stream()
        for stream in (None, side, None):
            t.cuda.synchronize()
            mk.decode_step_kv8(tok, tok, lens, cache, d_table, logits, stream=stream)
        assert mk.sync_status()[0] == 0 and lens.tolist() == [603] * batch
        got = (tok, logits, *cache.pools())
        assert want is None or all(t.equal(a, b) for a, b in zip(got, want)), kind
        want = want or got
        mk.close()
