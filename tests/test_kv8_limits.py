"""Sizes so large that a product of them passes 64 bits are refused as the smaller ones above the
limits are (host only, nothing is launched)."""
import ctypes

import pytest

import persistent_runtime_b200 as prb
from test_kv8_refusals import A, cache, pages, refused, rows


# (positions / 32 + 16) x kv heads x row groups x sequences: 2^64 (0 in 64 bits), 2^63, and
# just above the limit of 2^30
@pytest.mark.parametrize("n_seqs,kv_heads,max_pages", [(1 << 24, 1 << 15, (1 << 21) - 1), (1 << 23, 1 << 15, (1 << 21) - 1),
                                                       (1 << 24, 1 << 11, (1 << 21) - 1), (4, 8, (1 << 21) + 1)])
def test_attention_refuses_products_beyond_64_bits(n_seqs, kv_heads, max_pages):
    L, ref, size = prb.lib(), ctypes.byref, ctypes.c_int64(-1)
    c = cache(n_kv_heads=kv_heads, page_size=512)
    b = prb.Batch(n_seqs, n_seqs, 1, max_pages, None, A, A)
    word = "positions"
    refused(L.mk_kv8_attention_workspace(ref(c), kv_heads, prb.MK_BF16, ref(b), ref(size)), word)
    refused(L.mk_kv8_attention(ref(c), 0, ref(rows()), kv_heads, 1.0, A, None, ref(b), A, 1 << 40, None), word)
    assert size.value == -1


def test_pages_refuse_sizes_beyond_64_bits():
    """The sum of the pools' page sizes, and a size rounded up to steps of the copy."""
    L, ref, size = prb.lib(), ctypes.byref, ctypes.c_int64(-1)
    for sizes in ([1 << 62] * 4, [(1 << 63) - 4], [1 << 40], [1 << 39, 1 << 39]):
        p = pages(n_pools=len(sizes))
        for i, n in enumerate(sizes):
            p.d_pool[i], p.page_bytes[i] = A, n
        refused(L.mk_pages_workspace(ref(p), 0, ref(size)), "page_bytes")
        refused(L.mk_pages_compact(ref(p), A, 1 << 40, None), "page_bytes")
    assert size.value == -1
