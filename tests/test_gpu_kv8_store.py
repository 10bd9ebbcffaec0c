"""mk_kv8_store against the block-by-block restatement: codes and scales bit for bit (every
operation of its definition is one IEEE fp32 operation), everything else untouched."""
import numpy as np
import pytest

import kv8_ref as ref
from kv8_ref import dev, make_table, torch

pytestmark = pytest.mark.gpu

CASES = [
    # heads, dim, page, block, format, dtype, cached, new rows
    (2, 64, 64, 16, "int8", "bfloat16", [0], [1]),
    (2, 64, 64, 64, "e4m3", "float32", [33], [1]),
    (1, 128, 128, 128, "int8", "float16", [127, 128, 129, 0], [1, 1, 1, 1]),
    (8, 128, 64, 32, "e4m3", "bfloat16", [0, 31, 64, 500], [3, 0, 65, 1]),
    (3, 64, 48, 16, "int8", "float32", [15, 16, 47, 48, 1], [1, 33, 2, 0, 130]),
    (8, 128, 256, 128, "int8", "bfloat16", [100, 0], [300, 129]),
    (4, 128, 16, 16, "e4m3", "float16", [5, 77], [40, 17]),
    (2, 128, 64, 64, "int8", "float32", [1000, 63], [200, 1]),
]


def run(case, seed, layers=2, layer=1, spread=1.0):
    H, D, P, T, fmt, dtype, cached, new = case
    t = torch()
    cached, new = np.array(cached), np.array(new)
    table, n_pages = make_table(cached + new, P, seed=seed)
    host = ref.Cache(n_pages, layers, H, D, P, T, fmt, seed)
    cache = host.device()
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rng = np.random.default_rng(seed + 1)
    kind = getattr(t, dtype)
    x = [t.from_numpy((rng.standard_normal((start[-1], H, D)) * spread).astype(np.float32)).to(kind)
         for _ in range(2)]
    single = (new == 1).all()
    cache.store(layer, x[0].cuda(), x[1].cuda(), dev(table), dev(cached.astype(np.int32)),
                row_start=None if single else dev(start))
    cache.check()
    host.store(layer, [a.float().numpy() for a in x], table, cached, start)
    return host, cache, x, table, cached, start


def same(host, cache):
    t = torch()
    for got, want in zip((cache.k, cache.v), host.codes):
        np.testing.assert_array_equal(got.view(t.uint8).cpu().numpy(), want)
    for got, want in zip((cache.k_scale, cache.v_scale), host.scales):
        np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("case", CASES, ids=[f"{c[4]}-{c[5]}-d{c[1]}-p{c[2]}-b{c[3]}" for c in CASES])
def test_codes_and_scales_bit_for_bit(case):
    for spread in (1.0, 0.01, 30.0):  # scales that grow, stay, and grow much
        host, cache, *_ = run(case, 5, spread=spread)
        same(host, cache)


def test_a_fresh_block_is_off_by_half_a_step():
    for fmt, half in (("int8", 0.5), ("e4m3", 2.0 ** -4)):
        host, cache, x, table, cached, start = run((2, 64, 64, 32, fmt, "float32", [0], [64]), 9)
        got = host.rows(0, 1, table[0][:1], 64)
        want = x[0].double().numpy()
        size = np.repeat(host.scales[0][table[0][0], 1], 32, axis=1).T[:, :, None].astype(np.float64)
        # int8: half a step of the scale; e4m3: half a step of the value, or of the smallest code
        # (2^-9); the fp32 reciprocal and product add 2 roundings of 2^-24 to the quotient
        bound = half * size if fmt == "int8" else np.maximum(half * np.abs(want), 2.0 ** -10 * size)
        assert np.all(np.abs(got - want) <= bound + 2.0 ** -22 * np.abs(want))


def test_token_by_token_keeps_the_scale_of_the_largest():
    t = torch()
    rng = np.random.default_rng(3)
    x = rng.standard_normal((70, 2, 64)).astype(np.float32)
    table, n_pages = make_table([70], 32)
    host = ref.Cache(n_pages, 1, 2, 64, 32, 32, "int8", 3)
    cache = host.device()
    d_table = dev(table)
    for p in range(70):
        row = dev(x[p:p + 1])
        cache.store(0, row, -row, d_table, dev(np.array([p], np.int32)))
        host.store(0, [x[p:p + 1], -x[p:p + 1]], table, [p], [0, 1])
    cache.check()
    same(host, cache)
    for b in range(3):
        rows = x[32 * b:32 * (b + 1)]
        want = np.abs(rows).max(axis=(0, 2)) * (np.float32(1) / np.float32(127))
        page, at = table[0][b], 0
        np.testing.assert_array_equal(cache.k_scale[page, 0, :, at].cpu().numpy(), want)
    del t


def test_special_values():
    t = torch()
    for fmt in ("int8", "e4m3"):
        table, n_pages = make_table([64], 64)
        host = ref.Cache(n_pages, 1, 4, 64, 64, 32, fmt, 3)
        cache = host.device()
        x = np.random.default_rng(0).standard_normal((40, 4, 64)).astype(np.float32)
        x[:, 0] = 0            # a block of zeros
        x[3, 1, 5] = np.inf    # infinity and NaN poison their block alone
        x[35, 2, 0] = np.nan
        x[:, 3] *= 1e-38       # the smallest scale
        cache.store(0, dev(x), dev(x), dev(table), dev(np.zeros(1, np.int32)),
                    row_start=dev(np.array([0, 40], np.int32)))
        cache.check()
        host.store(0, [x, x], table, [0], [0, 40])
        same(host, cache)
        s = cache.k_scale[int(table[0, 0]), 0].cpu().numpy()
        assert s[0, 0] == ref.SCALE_MIN and np.isnan(s[1, 0]) and np.isfinite(s[1, 1])
        assert np.isfinite(s[2, 0]) and np.isnan(s[2, 1]) and s[3, 0] == ref.SCALE_MIN
        # a later row of a poisoned block leaves it poisoned; a row at its beginning begins it anew
        row = dev(np.ones((1, 4, 64), np.float32))
        cache.store(0, row, row, dev(table), dev(np.array([40], np.int32)))
        assert np.isnan(cache.k_scale[int(table[0, 0]), 0, 2, 1].item())
        cache.store(0, row, row, dev(table), dev(np.array([32], np.int32)))
        assert np.isfinite(cache.k_scale[int(table[0, 0]), 0, 2, 1].item())
    del t


def test_strided_rows_and_rows_behind_the_last_sequence():
    t = torch()
    H, D = 2, 64
    packed = t.randn(9, 5 * H, D, device="cuda", dtype=t.bfloat16)  # a slice of a packed projection
    k, v = packed[:, 2:4], packed[:, 6:8]
    table, n_pages = make_table([20, 20], 32)
    host = ref.Cache(n_pages, 1, H, D, 32, 16, "int8", 1)
    cache = host.device()
    start = np.array([0, 3, 7], np.int32)  # rows 7 and 8 belong to nobody
    cache.store(0, k, v, dev(table), dev(np.array([10, 13], np.int32)), row_start=dev(start))
    cache.check()
    host.store(0, [k.float().cpu().numpy(), v.float().cpu().numpy()], table, [10, 13], start)
    same(host, cache)


def test_a_billion_rows_behind_the_last_sequence():
    """Positions and rows near 2^30 and 2^31: slots that belong to no block do nothing."""
    t = torch()
    n, c, P = (1 << 30) + 1024, (1 << 31) - (1 << 20), 128
    host = ref.Cache(1, 1, 1, 64, P, 128, "int8", 1)
    cache, want = host.device(), host.device()
    x = t.randn(1, 1, 64, device="cuda")
    table = t.full((1, c // P + 1), -1, dtype=t.int32, device="cuda")
    table[0, c // P] = 0
    rows = x.expand(n, 1, 64)
    cache.store(0, rows, rows, table, dev(np.array([c], np.int32)), row_start=dev(np.array([0, 1], np.int32)))
    cache.check()
    want.store(0, x, x, dev(np.zeros((1, 1), np.int32)), dev(np.zeros(1, np.int32)))
    for a, b in zip(cache.pools(), want.pools()):
        assert t.equal(a, b)


def test_strides_of_a_single_row_or_head_may_be_anything():
    t = torch()
    table, n_pages = make_table([20], 32)
    host = ref.Cache(n_pages, 1, 1, 64, 32, 16, "int8", 1)
    cache = host.device()
    x = t.randn(1, 1, 64, device="cuda").as_strided((1, 1, 64), (3, 5, 1))
    cache.store(0, x, x, dev(table), dev(np.array([10], np.int32)))
    cache.check()
    host.store(0, [x.cpu().numpy()] * 2, table, [10], [0, 1])
    same(host, cache)


def test_device_checks_leave_out_what_is_wrong():
    import persistent_runtime_b200 as prb
    table, n_pages = make_table([40, 40, 40], 32, extra=0)
    x = np.random.default_rng(2).standard_normal((3, 2, 64)).astype(np.float32)
    for lens, bad_page, check in (([10, -1, 5], False, 2), ([10, 64, 5], False, 2), ([10, 33, 5], True, 3)):
        host = ref.Cache(n_pages, 1, 2, 64, 32, 16, "int8", 1)
        cache = host.device()
        tab = table.copy()
        if bad_page:
            tab[1, 1] = n_pages
        cache.store(0, dev(x), dev(x), dev(tab), dev(np.array(lens, np.int32)))
        rc, detail = cache.sync_status()
        assert rc == prb.MK_ERR_DEVICE and detail[1] == 1 and detail[3] == check
        with pytest.raises(prb.MkError):
            cache.check()
        host.store(0, [x[[0, 2]]] * 2, tab[[0, 2]], [lens[0], lens[2]], [0, 1, 2])
        same(host, cache)
        cache.reset()
        cache.check()
    host = ref.Cache(n_pages, 1, 2, 64, 32, 16, "int8", 1)
    cache = host.device()
    cache.store(0, dev(x), dev(x), dev(table), dev(np.array([1, 2, 3], np.int32)),
                row_start=dev(np.array([0, 2, 1, 4], np.int32)))  # out of order, past the end
    assert cache.sync_status()[1][3] == 1
