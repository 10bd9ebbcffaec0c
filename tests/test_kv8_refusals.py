"""What the calls on 8-bit caches and pages refuse on the host, before anything is launched
(no device is needed), and the layouts of their structures."""
import ctypes
import os
import subprocess

import pytest

import persistent_runtime_b200 as prb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # an aligned address; it is never read


def cache(**kw):
    c = prb.Kv8Cache(0, prb.MK_KV8_INT8, 2, 2, 64, 64, 32, 10, A, A, A, A, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def batch(**kw):
    b = prb.Batch(3, 3, 1, 4, None, A, A)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def rows(**kw):
    r = prb.Rows(A, prb.MK_BF16, 128, 64)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def pages(**kw):
    p = prb.Pages(0, 10, 3, 4, 64, 1)
    p.d_pool[0], p.page_bytes[0] = A, 64
    p.d_page_table = p.d_ref = A
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def refused(rc, word):
    text = prb.lib().mk_last_error(None).decode()
    assert rc == prb.MK_ERR_ARG and word in text, (rc, text)


BAD_CACHES = [(dict(format=2), "format"), (dict(head_dim=96), "head_dim"), (dict(block=8), "block"),
              (dict(block=48), "block"), (dict(page_size=40), "page_size"), (dict(page_size=16), "page_size"),
              (dict(n_pages=0), "empty"), (dict(n_kv_heads=0), "empty"), (dict(n_layers=0), "empty"),
              (dict(d_v=None), "null"), (dict(d_k_scale=None), "null"), (dict(d_k=A + 8), "aligned"),
              (dict(device=-1), "device")]
BAD_BATCHES = [(dict(n_seqs=0), "at least 1"), (dict(max_rows=0), "at least 1"), (dict(n_rows=-1), "at least 1"),
               (dict(max_pages=0), "at least 1"), (dict(d_kv_len=None), "null"), (dict(d_page_table=None), "null"),
               (dict(n_rows=4), "one row per sequence"), (dict(max_pages=1 << 26), "2^31")]
BAD_ROWS = [(dict(data=None), "null"), (dict(data=A + 2), "aligned"), (dict(dtype=3), "element type"),
            (dict(row_stride=100), "strides"), (dict(head_stride=68), "strides"),
            (dict(dtype=prb.MK_F32, row_stride=126), "strides")]


def test_store_and_attention_refuse():
    L = prb.lib()
    ref = ctypes.byref

    def store(c, layer, k, v, b):
        return L.mk_kv8_store(c, layer, k, v, b, None)

    def attend(c, layer, q, heads, b, out=A, ws=A, size=1 << 40):
        return L.mk_kv8_attention(c, layer, q, heads, 1.0, out, None, b, ws, size, None)

    ok = ref(rows())
    for bad, word in BAD_CACHES:
        refused(store(ref(cache(**bad)), 0, ok, ok, ref(batch())), word)
        refused(attend(ref(cache(**bad)), 0, ok, 4, ref(batch())), word)
    for bad, word in BAD_BATCHES:
        refused(store(ref(cache()), 0, ok, ok, ref(batch(**bad))), word)
        refused(attend(ref(cache()), 0, ok, 4, ref(batch(**bad))), word)
    for bad, word in BAD_ROWS:
        refused(store(ref(cache()), 1, ref(rows(**bad)), ok, ref(batch())), word)
        refused(store(ref(cache()), 1, ok, ref(rows(**bad)), ref(batch())), word)
        refused(attend(ref(cache()), 1, ref(rows(**bad)), 4, ref(batch())), word)
    refused(store(None, 0, ok, ok, ref(batch())), "null cache")
    refused(store(ref(cache()), 0, ok, ok, None), "null batch")
    refused(store(ref(cache()), 0, None, ok, ref(batch())), "null rows")
    refused(store(ref(cache()), 0, ok, ref(rows(dtype=prb.MK_F16)), ref(batch())), "differ")
    for layer in (-1, 2):
        refused(store(ref(cache()), layer, ok, ok, ref(batch())), "layer")
        refused(attend(ref(cache()), layer, ok, 4, ref(batch())), "layer")
    for heads in (0, 3, -2, 2 * 1025):
        refused(attend(ref(cache()), 0, ok, heads, ref(batch())), "query heads" if heads > 3 else "n_q_heads")
    refused(attend(ref(cache()), 0, ok, 4, ref(batch(max_rows=17, d_row_start=A))), "max_rows")
    refused(attend(ref(cache()), 0, ok, 4, ref(batch()), out=None), "output")
    refused(attend(ref(cache()), 0, ok, 4, ref(batch()), out=A + 4), "output")
    big = batch(max_pages=1000)
    refused(attend(ref(cache()), 0, ok, 4, ref(big), ws=None), "workspace")
    refused(attend(ref(cache()), 0, ok, 4, ref(big), ws=A + 8), "workspace")
    refused(attend(ref(cache()), 0, ok, 4, ref(big), size=16), "workspace of 16 bytes")
    size = ctypes.c_int64(-1)
    refused(L.mk_kv8_attention_workspace(ref(cache()), 4, 7, ref(big), ref(size)), "element type")
    refused(L.mk_kv8_attention_workspace(ref(cache()), 4, prb.MK_BF16, ref(big), None), "null")
    assert L.mk_kv8_attention_workspace(ref(cache()), 4, prb.MK_BF16, ref(big), ref(size)) == prb.MK_OK
    assert size.value > 0
    # nothing to do is no error, and needs no device
    empty = batch(n_rows=0, d_row_start=A)
    assert store(ref(cache()), 0, None, None, ref(empty)) == prb.MK_OK
    assert attend(ref(cache()), 0, ok, 4, ref(empty), out=None, ws=None, size=0) == prb.MK_OK


def test_page_calls_refuse():
    L = prb.lib()
    ref = ctypes.byref
    size = ctypes.c_int64(-1)
    assert L.mk_pages_workspace(ref(pages()), 3, ref(size)) == prb.MK_OK
    calls = {
        "fork": lambda p, n=1, a=A, b=A, ws=A, s=1 << 40: L.mk_pages_fork(p, n, a, b, ws, s, None),
        "copy": lambda p, n=1, a=A, b=A, ws=A, s=1 << 40: L.mk_pages_copy(p, n, a, b, ws, s, None),
        "free": lambda p, n=1, a=A, b=A, ws=A, s=1 << 40: L.mk_pages_free(p, n, a, ws, s, None),
        "reserve": lambda p, n=1, a=A, b=A, ws=A, s=1 << 40: L.mk_pages_reserve(p, a, b, ws, s, None),
        "compact": lambda p, n=1, a=A, b=A, ws=A, s=1 << 40: L.mk_pages_compact(p, ws, s, None)}
    odd = pages()
    odd.page_bytes[0] = 6
    unaligned = pages()
    unaligned.d_pool[0] = A + 2
    for name, call in calls.items():
        refused(call(None), "null pages")
        for bad, word in ((dict(n_pages=0), "at least 1"), (dict(n_seqs=0), "at least 1"),
                          (dict(max_pages=0), "at least 1"), (dict(page_size=0), "at least 1"),
                          (dict(n_pools=9), "n_pools"), (dict(n_pools=-1), "n_pools"), (dict(device=-1), "device"),
                          (dict(d_ref=None), "null"), (dict(d_page_table=None), "null"),
                          (dict(n_seqs=1 << 30), "2^31")):
            refused(call(ref(pages(**bad))), word)
        refused(call(ref(odd)), "page_bytes")
        refused(call(ref(unaligned)), "aligned")
        refused(call(ref(pages()), ws=None), "workspace")
        refused(call(ref(pages()), ws=A + 4), "workspace")
        refused(call(ref(pages()), s=8), "workspace of 8 bytes")
        if name in ("fork", "copy", "free"):
            refused(call(ref(pages()), n=-1), "negative")
            refused(call(ref(pages()), n=1 << 30), "too long")
            refused(call(ref(pages()), a=None), "null list")
            assert call(ref(pages()), n=0, a=None, ws=None, s=0) == prb.MK_OK
        if name in ("fork", "copy"):
            refused(call(ref(pages()), b=None), "null list")
        if name == "reserve":
            refused(call(ref(pages()), a=None), "null")
            refused(call(ref(pages()), b=None), "null")


def test_the_binding_wants_cuda_tensors():
    import torch
    k = torch.zeros(4, 1, 2, 32, 64, dtype=torch.int8)
    s = torch.ones(4, 1, 2, 1)
    with pytest.raises(prb.MkError, match="CUDA"):
        prb.KV8Cache(k, k, s, s)
    with pytest.raises(prb.MkError, match="CUDA"):
        prb.PagePool(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 32, [k])


STRUCTS = {"mk_kv8_cache": prb.Kv8Cache, "mk_rows": prb.Rows, "mk_batch": prb.Batch, "mk_pages": prb.Pages}


def test_binding_structures_match_the_header_layouts(tmp_path):
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "mk.h"', "int main(void) {"]
    for cname, py in STRUCTS.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        for field, _ in py._fields_:
            lines.append(f'  printf("{cname} {field} %zu\\n", offsetof({cname}, {field}));')
    for name in ("MK_KV8_INT8", "MK_KV8_E4M3", "MK_F32", "MK_BF16", "MK_F16", "MK_KV8_MAX_ROWS", "MK_MAX_POOLS"):
        lines.append(f'  printf("{name} value %d\\n", (int){name});')
    lines += ["  return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in subprocess.check_output([str(exe)]).decode().splitlines()}
    for cname, py in STRUCTS.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for field, _ in py._fields_:
            assert got[(cname, field)] == getattr(py, field).offset, (cname, field)
    for (name, kind), value in got.items():
        if kind == "value":
            assert getattr(prb, name) == value, name


def test_page_calls_refuse_more_pages_than_a_copy_counts():
    many = pages(n_pages=1 << 29, n_pools=4)
    for i in range(4):
        many.d_pool[i], many.page_bytes[i] = A, 4
    size = ctypes.c_int64()
    refused(prb.lib().mk_pages_workspace(ctypes.byref(many), 0, ctypes.byref(size)), "2^31 pages")
    refused(prb.lib().mk_pages_compact(ctypes.byref(many), A, 1 << 40, None), "2^31 pages")
    many.n_pages = 1 << 28
    assert prb.lib().mk_pages_workspace(ctypes.byref(many), 0, ctypes.byref(size)) == prb.MK_OK
