"""The decode step over an 8-bit paged cache (mk_decode_step_kv8), and the cache, the attention
and the page calls together as a server uses them, against a float64 restatement of the step
that quantises its K/V rows as the cache does."""
import numpy as np
import pytest

import kv8_ref as ref
import synth
from gpu_helpers import (HIDDEN_TOL, LOGIT_TOL, SEPARATION, _wrap_device_f32, dev_weights)
from kv8_ref import dev, torch

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("built_libs")]


class Host:
    """The step in float64 for the sequences of a batch, on a host copy of the cache."""

    def __init__(self, w, weights, cache):
        self.w, self.cache = w, cache
        f = lambda a: None if a is None else synth.bf16_to_f32(a).astype(np.float64)  # noqa: E731
        self.embed, self.final_norm = f(weights["embed"]), f(weights["final_norm"])
        self.head = self.embed if weights["lm_head"] is None else f(weights["lm_head"])
        self.layers = [{k: f(a) for k, a in lw.items()} for lw in weights["layers"]]

    def norm(self, x, g):
        return x * g / np.sqrt((x * x).mean(-1, keepdims=True) + self.w.rms_eps)

    def rope(self, x, pos):
        D = self.w.head_dim
        ang = pos * self.w.rope_theta ** (-2.0 * np.arange(D // 2) / D)
        c, s = np.cos(ang), np.sin(ang)
        a, b = x[..., :D // 2], x[..., D // 2:]
        return np.concatenate([a * c - b * s, b * c + a * s], -1)

    def step(self, tokens, table, lens):
        w, B, D = self.w, len(tokens), self.w.head_dim
        x = self.embed[tokens]
        start = np.arange(B + 1)
        for l, y in enumerate(self.layers):
            z = self.norm(x, y["attn_norm"])
            q = self.norm((z @ y["wq"].T).reshape(B, -1, D), y["q_norm"])
            k = self.norm((z @ y["wk"].T).reshape(B, -1, D), y["k_norm"])
            v = (z @ y["wv"].T).reshape(B, -1, D)
            q = np.stack([self.rope(q[b], lens[b]) for b in range(B)])
            k = np.stack([self.rope(k[b], lens[b]) for b in range(B)])
            self.cache.store(l, [k.astype(np.float32), v.astype(np.float32)], table, lens, start)
            o = self.cache.attention(l, q, table, lens, start, D ** -0.5, "float32")[0]
            x = x + o.reshape(B, -1) @ y["wo"].T
            z = self.norm(x, y["mlp_norm"])
            g = z @ y["w_gate"].T
            x = x + (g / (1 + np.exp(-g)) * (z @ y["w_up"].T)) @ y["w_down"].T
        return x, self.norm(x, self.final_norm) @ self.head.T


def compare(mk, w, want, logits, tokens):
    hidden = _wrap_device_f32(mk.final_hidden_ptr(), w.batch * w.hidden).view(w.batch, -1).cpu().numpy()
    x, z = want
    for b in range(w.batch):
        assert np.linalg.norm(hidden[b] - x[b]) <= HIDDEN_TOL * np.linalg.norm(x[b])
        size = np.abs(z[b]).max()
        assert np.abs(logits[b] - z[b]).max() <= LOGIT_TOL * size
        top = np.sort(z[b])[-2:]
        if top[1] - top[0] > SEPARATION * size:
            assert tokens[b] == int(z[b].argmax())


def codes_close(cache, host):
    """Codes of the device against the host's float64 step: rows that round the other way are
    off by one code, and are few (a projection's fp32 error moves a value by some 1e-6 of its
    row's largest, 1e-4 of a code: about one code in a thousand may round the other way)."""
    t = torch()
    for got, want in zip((cache.k, cache.v), host.codes):
        a = ref.decode(got.view(t.uint8).cpu().numpy(), host.fmt)
        b = ref.decode(want, host.fmt)
        differ = a != b
        assert differ.mean() < 1e-2
        step = 1.0 if host.fmt == "int8" else np.maximum(2.0 ** -3 * np.maximum(np.abs(a), np.abs(b)), 2.0 ** -9)
        assert np.all(np.abs(a - b) <= step)
    for got, want in zip((cache.k_scale, cache.v_scale), host.scales):
        np.testing.assert_allclose(got.cpu().numpy(), want, rtol=1e-4)


@pytest.mark.parametrize("batch,fmt,page,block,kv_page", [(1, "int8", 64, 64, 0), (1, "e4m3", 32, 16, 0),
                                                          (3, "int8", 64, 32, 0), (12, "e4m3", 128, 128, 0),
                                                          (2, "int8", 16, 16, 64)])
def test_steps_against_float64(batch, fmt, page, block, kv_page):
    import persistent_runtime_b200 as prb
    t = torch()
    w = synth.TINY.with_(name="tiny-kv8", batch=batch, kv_len=None, kv_len_range=(0, 150), steps=3)
    weights = synth.make_weights(w, 3)
    lens = w.kv_lens(3).astype(np.int64)
    cap = int(lens.max()) + 3
    table, n_pages = ref.make_table(lens + 3, page, seed=3)
    table = np.concatenate([table, np.full((batch, -(-cap // page)), -1, np.int32)], 1)
    host = ref.Cache(n_pages, w.n_layers, w.n_kv_heads, w.head_dim, page, block, fmt, 3)
    cache = host.device()
    model = Host(w, weights, host)
    mk = prb.Megakernel(w, cap, 0, **({"kv_page_size": kv_page} if kv_page else {}))
    mk.load_weights(dev_weights(weights))
    tok, d_len, d_table = dev(synth.make_tokens(w, 3)), dev(lens.astype(np.int32)), dev(table)
    logits = t.zeros(batch, w.vocab, device="cuda")
    tokens = tok.cpu().numpy()
    for s in range(3):
        mk.decode_step_kv8(tok, tok, d_len, cache, d_table, logits)
        assert mk.sync_status()[0] == 0
        want = model.step(tokens, table, (lens + s).tolist())
        tokens = tok.cpu().numpy()
        compare(mk, w, want, logits.cpu().numpy(), tokens)
        codes_close(cache, host)
    assert (d_len.cpu().numpy() == lens + 3).all()
    mk.close()


def test_a_bad_page_or_length_writes_nothing():
    import persistent_runtime_b200 as prb
    t = torch()
    w = synth.TINY.with_(name="tiny-kv8", batch=2, kv_len=40, steps=2)
    mk = prb.Megakernel(w, 64, 0)
    table, n_pages = ref.make_table([42, 42], 16)
    host = ref.Cache(n_pages, w.n_layers, w.n_kv_heads, w.head_dim, 16, 16, "int8", 4)
    cache = host.device()
    lens, tok = dev(np.array([40, 40], np.int32)), dev(np.array([1, 2], np.int32))
    out = t.full((2,), -7, dtype=t.int32, device="cuda")
    with pytest.raises(prb.MkError) as e:  # no weights yet
        mk.decode_step_kv8(tok, out, lens, cache, dev(table))
    assert e.value.status == prb.MK_ERR_NOT_LOADED
    mk.load_weights(dev_weights(synth.make_weights(w, 3)))
    bad = table.copy()
    bad[1, 1] = n_pages
    for tab, n in ((bad, [40, 40]), (table, [40, 64]), (table, [-1, 40])):
        d_len = dev(np.array(n, np.int32))
        before = [x.clone() for x in cache.pools()]
        mk.decode_step_kv8(tok, out, d_len, cache, dev(np.ascontiguousarray(tab)))
        rc, detail = mk.sync_status()
        assert rc == prb.MK_ERR_DEVICE
        for x, y in zip(cache.pools(), before):
            assert t.equal(x.view(t.uint8) if x.dtype == t.int8 else x, y.view(t.uint8) if y.dtype == t.int8 else y)
        assert (out == -7).all() and d_len.tolist() == n
        mk.reset()
    mk.decode_step_kv8(tok, out, lens, cache, dev(table))
    assert mk.sync_status()[0] == 0 and lens.tolist() == [41, 41]
    # refused on the host
    with pytest.raises(prb.MkError):  # the table covers fewer than kv_capacity positions
        mk.decode_step_kv8(tok, out, lens, cache, dev(np.ascontiguousarray(table[:, :3])))
    other = ref.Cache(n_pages, w.n_layers + 1, w.n_kv_heads, w.head_dim, 16, 16, "int8", 4).device()
    with pytest.raises(prb.MkError):
        mk.decode_step_kv8(tok, out, lens, other, dev(table))
    with pytest.raises(prb.MkError):
        mk.decode_step_kv8(tok, out, lens, cache, dev(table).long())
    mk.close()


def test_serving_with_shared_pages():
    """Prompts stored, decoded, forked, continued, freed and compacted: after every step all
    sequences agree with the restatement on a host cache without any sharing."""
    import persistent_runtime_b200 as prb
    t = torch()
    B, page, block = 6, 32, 16
    w = synth.TINY.with_(name="tiny-kv8", batch=B, kv_len=0, steps=1)
    weights = synth.make_weights(w, 5)
    n_pages, cap = 26, 6 * page
    dev_cache = prb.KV8Cache.empty(n_pages, w.n_layers, w.n_kv_heads, w.head_dim, page, block)
    for x in (dev_cache.k, dev_cache.v):
        x.zero_()
    pages = prb.PagePool.empty(B, cap // page, page, dev_cache.pools())
    # the host's sequences have pages of their own
    own = np.arange(B * cap // page, dtype=np.int32).reshape(B, -1)
    host = ref.Cache(own.size, w.n_layers, w.n_kv_heads, w.head_dim, page, block, "int8", 0)
    model = Host(w, weights, host)
    mk = prb.Megakernel(w, cap, 0)
    mk.load_weights(dev_weights(weights))
    rng = np.random.default_rng(0)
    # prompts of sequences 0 .. 2 (their K/V come from elsewhere); the others idle at length 0
    new = np.array([70, 33, 5, 0, 0, 0])
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    d_len = dev(np.zeros(B, np.int32))
    pages.reserve(d_len, dev(new.astype(np.int32)))
    for l in range(w.n_layers):
        x = rng.standard_normal((2, start[-1], w.n_kv_heads, w.head_dim)).astype(np.float32)
        dev_cache.store(l, dev(x[0]), dev(x[1]), pages.page_table, d_len, row_start=dev(start))
        host.store(l, x, own, [0] * B, start)
    lens = new.astype(np.int64)
    d_len = dev(lens.astype(np.int32))
    ones = dev(np.ones(B, np.int32))
    tok = dev(rng.integers(0, w.vocab, B).astype(np.int32))
    logits = t.zeros(B, w.vocab, device="cuda")

    def steps(n):
        nonlocal lens
        for _ in range(n):
            tokens = tok.cpu().numpy()
            pages.reserve(d_len, ones)
            mk.decode_step_kv8(tok, tok, d_len, dev_cache, pages.page_table, logits)
            assert mk.sync_status()[0] == 0
            want = model.step(tokens, own, lens.tolist())
            compare(mk, w, want, logits.cpu().numpy(), tok.cpu().numpy())
            lens = lens + 1
        pages.check()
        held = pages.page_table.cpu().numpy()
        np.testing.assert_array_equal(pages.ref_count.cpu().numpy(),
                                      np.bincount(held[held >= 0], minlength=n_pages))

    def clear(seqs):
        for s in seqs:
            lens[s], d_len[s], tok[s] = 0, 0, 1

    def fork(src, dst):
        pages.free(dev(np.array(dst, np.int32)))
        pages.fork(dev(np.array(src, np.int32)), dev(np.array(dst, np.int32)))
        for a, b in zip(src, dst):
            for c in host.codes + host.scales:
                c[own[b]] = c[own[a]]
            lens[b], d_len[b] = lens[a], d_len[a]
            tok[b] = (int(tok[a]) + 17 * b) % w.vocab

    steps(2)
    fork([0, 0, 1], [3, 4, 5])
    steps(4)
    pages.free(dev(np.array([0, 2], np.int32)))
    clear([0, 2])
    pages.compact()
    steps(3)
    fork([3], [0])
    pages.compact()
    steps(30)  # over the end of a page
    used = int((pages.ref_count > 0).sum())
    assert used < n_pages
    mk.close()


def test_the_step_in_a_graph():
    import persistent_runtime_b200 as prb
    t = torch()
    w = synth.TINY.with_(name="tiny-kv8", batch=2, kv_len=600, steps=4)
    mk = prb.Megakernel(w, 700, 0)
    mk.load_weights(dev_weights(synth.make_weights(w, 6)))
    table, n_pages = ref.make_table([700, 700], 64, seed=6)
    host = ref.Cache(n_pages, w.n_layers, w.n_kv_heads, w.head_dim, 64, 64, "int8", 6)
    d_table = dev(table)

    def state():
        return (host.device(), dev(np.array([3, 4], np.int32)), dev(np.array([600, 333], np.int32)),
                t.zeros(2, w.vocab, device="cuda"))

    cache, tok, d_len, logits = state()
    seen = []
    for _ in range(4):
        mk.decode_step_kv8(tok, tok, d_len, cache, d_table, logits)
        seen.append((tok.clone(), logits.clone()))
    assert mk.sync_status()[0] == 0
    cache2, tok, d_len, logits = state()
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        mk.decode_step_kv8(tok, tok, d_len, cache2, d_table, logits)
    for want_tok, want in seen:
        g.replay()
        t.cuda.synchronize()
        assert t.equal(tok, want_tok) and t.equal(logits, want)
    assert mk.sync_status()[0] == 0
    for x, y in zip(cache.pools(), cache2.pools()):
        assert t.equal(x, y)
    mk.close()


FIRST_CALLS = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np, torch
import kv8_ref as ref, persistent_runtime_b200 as prb
from kv8_ref import dev
table, n = ref.make_table([3000, 2500], 64)
cache = ref.Cache(n, 1, 8, 128, 64, 64, "int8", 1).device()
q = torch.randn(2, 32, 128, device="cuda", dtype=torch.bfloat16)
k = torch.randn(2, 8, 128, device="cuda")
lens, table = dev(np.array([2990, 2400], np.int32)), dev(table)
held = prb.PagePool.empty(4, 10, 64, cache.pools())
a, b, c = (dev(np.array([x], np.int32)) for x in (0, 1, 3))
six = c + 3
zero, one = dev(np.zeros(4, np.int32)), dev(np.array([1, 0, 1, 0], np.int32))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    held.reserve(zero, one)
    held.fork(a, b)
    held.free(a)
    held.compact()
    held.copy(c, six)
    cache.store(0, k, k, table, lens)
    out = cache.attention(0, q, table, lens)
g.replay()
cache.check()
held.check()
assert torch.equal(out, cache.attention(0, q, table, lens))
assert held.page_table[:, 0].tolist() == [-1, 0, 1, -1], held.page_table
print("ok")
"""


def test_first_calls_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALLS.format(root=os.path.dirname(tests), tests=tests)
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip() == "ok", done.stderr[-2000:]
