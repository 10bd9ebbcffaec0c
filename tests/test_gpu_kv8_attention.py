"""mk_kv8_attention against softmax attention in 64 bits on the dequantised cache."""
import numpy as np
import pytest

import kv8_ref as ref
from kv8_ref import dev, make_table, torch

pytestmark = pytest.mark.gpu

CASES = [
    # q heads, kv heads, dim, page, block, format, dtype, cached, new rows
    (4, 2, 64, 64, 16, "int8", "bfloat16", [0], [1]),
    (4, 2, 64, 64, 64, "e4m3", "float32", [1], [1]),
    (16, 8, 128, 64, 64, "int8", "float16", [511, 0, 15, 16, 31, 32], [1] * 6),
    (32, 8, 128, 64, 32, "int8", "float32", [700, 3, 1200], [1] * 3),
    (32, 8, 128, 16, 16, "e4m3", "bfloat16", [1000, 17, 0, 300], [2, 0, 5, 1]),
    (16, 1, 128, 128, 128, "int8", "bfloat16", [900, 40], [1, 1]),
    (40, 2, 64, 48, 16, "e4m3", "float16", [100, 600], [3, 1]),
    (8, 8, 128, 256, 128, "e4m3", "float32", [2000, 255], [4, 16]),
    (6, 2, 64, 32, 32, "int8", "bfloat16", [5000], [16]),
    (24, 3, 128, 64, 16, "int8", "float32", [650, 1], [7, 2]),
]


def setup(case, seed, layers=2):
    Hq, H, D, P, T, fmt, dtype, cached, new = case
    t = torch()
    cached, new = np.array(cached), np.array(new)
    table, n_pages = make_table(cached + new, P, seed=seed)
    host = ref.Cache(n_pages, layers, H, D, P, T, fmt, seed)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = t.from_numpy(np.random.default_rng(seed + 7).standard_normal((start[-1], Hq, D)).astype(np.float32))
    q = q.to(getattr(t, dtype))
    return host, q, table, cached, new, start


def check(got, lse, host, layer, q, table, cached, start, scale, dtype):
    out, want_lse, tol, tol_lse = host.attention(layer, q.float().numpy(), table, cached, start, scale, dtype)
    err = np.abs(got.double().cpu().numpy() - out)
    worst = np.unravel_index(np.argmax(err / tol), err.shape)
    assert np.all(err <= tol), (worst, err[worst], tol[worst])
    err = np.abs(lse.double().cpu().numpy() - want_lse)
    assert np.all(err <= tol_lse), (err.max(), tol_lse.max())


@pytest.mark.parametrize("case", CASES, ids=[f"{c[5]}-{c[6]}-{c[0]}x{c[1]}-d{c[2]}-p{c[3]}-b{c[4]}" for c in CASES])
def test_against_64_bits(case):
    Hq, H, D, P, T, fmt, dtype, cached, new = case
    host, q, table, cached, new, start = setup(case, 11)
    cache = host.device()
    for scale in (None, 0.31):
        out, lse = cache.attention(1, q.cuda(), dev(table), dev(cached.astype(np.int32)),
                                   row_start=None if (new == 1).all() else dev(start),
                                   max_rows=int(new.max()), scale=scale, return_lse=True)
        cache.check()
        check(out, lse, host, 1, q, table, cached, start, scale or D ** -0.5, dtype)


def test_many_uneven_sequences():
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 700, 300)  # more sequences than threads of a block
    case = (8, 2, 64, 32, 32, "int8", "bfloat16", lens, np.ones(300, int))
    host, q, table, cached, new, start = setup(case, 12, layers=1)
    cache = host.device()
    out, lse = cache.attention(0, q.cuda(), dev(table), dev(cached.astype(np.int32)), return_lse=True)
    cache.check()
    check(out, lse, host, 0, q, table, cached, start, 64 ** -0.5, "bfloat16")


def test_large_and_small_scores_and_scales():
    """Scores of +-hundreds (one position takes all), blocks whose scales differ by 2^60."""
    case = (4, 2, 128, 64, 16, "int8", "float32", [333], [1])
    for k_size, v_size in ((50.0, 1.0), (1e-12, 2.0 ** 30)):
        host, q, table, cached, new, start = setup(case, 13)
        host.scales[0] *= np.float32(k_size)
        host.scales[1][:, :, :, ::2] *= np.float32(v_size)
        host.scales[1][:, :, :, 1::2] /= np.float32(v_size)
        cache = host.device()
        out, lse = cache.attention(1, q.cuda(), dev(table), dev(cached.astype(np.int32)), return_lse=True)
        check(out, lse, host, 1, q, table, cached, start, 128 ** -0.5, "float32")


def test_what_lies_behind_the_end_does_not_matter():
    """Codes (NaN ones too), scales and table entries past the last position, and a later
    row's block that reads as NaN, do not reach the rows that do not see them."""
    for fmt in ("int8", "e4m3"):
        case = (4, 2, 64, 64, 16, fmt, "bfloat16", [70, 41], [3, 2])
        host, q, table, cached, new, start = setup(case, 14)
        clean = host.device().attention(1, q.cuda(), dev(table), dev(cached.astype(np.int32)),
                                        row_start=dev(start), max_rows=3)
        for s in range(2):
            n = int(cached[s] + new[s])
            for which in range(2):
                host.codes[which][table[s][(n - 1) // 64], :, :, n % 64:] = 0xff
                host.scales[which][table[s][(n - 1) // 64], :, :, (n - 1) % 64 // 16 + 1:] = np.nan
        cache = host.device()
        table[:, -1] = 1 << 30
        got = cache.attention(1, q.cuda(), dev(table), dev(cached.astype(np.int32)),
                              row_start=dev(start), max_rows=3)
        cache.check()
        assert torch().equal(got, clean)
    # rows 0 and 1 of sequence 1 (positions 46, 47) do not see the block of position 48
    case = (4, 2, 64, 64, 16, "int8", "float32", [10, 46], [1, 4])
    host, q, table, cached, new, start = setup(case, 15)
    host.scales[0][table[1][0], :, :, 3] = np.nan
    host.scales[1][table[1][0], :, :, 3] = np.nan
    cache = host.device()
    out = cache.attention(1, q.cuda(), dev(table), dev(cached.astype(np.int32)), row_start=dev(start),
                          max_rows=4).cpu().numpy()
    assert np.isfinite(out[:3]).all() and np.isnan(out[3:]).all()


def test_rows_with_nan_or_infinity_stay_by_themselves():
    case = (8, 2, 128, 64, 64, "int8", "bfloat16", [200, 90], [2, 1])
    host, q, table, cached, new, start = setup(case, 16)
    cache = host.device()
    args = (dev(table), dev(cached.astype(np.int32)))
    clean = cache.attention(1, q.cuda(), *args, row_start=dev(start), max_rows=2)
    q2 = q.clone()
    q2[1, 3, 7] = float("nan")
    q2[2, 0, 0] = float("inf")
    q2[0, 5] = 0.0
    got = cache.attention(1, q2.cuda(), *args, row_start=dev(start), max_rows=2)
    t = torch()
    assert bool(t.isnan(got[1, 3]).all()) and bool(t.isnan(got[2, 0]).all())
    keep = t.ones(3, 8, dtype=t.bool)
    keep[1, 3] = keep[2, 0] = keep[0, 5] = False
    assert t.equal(got[keep.cuda()], clean[keep.cuda()])
    mean = host.rows(1, 1, table[0], 201).mean(0)[5 // 4]  # a zero query weighs all positions alike
    np.testing.assert_allclose(got[0, 5].float().cpu().numpy(), mean, rtol=0, atol=2.0 ** -7 * np.abs(mean).max())


def test_strides_bounds_and_repeats():
    t = torch()
    case = (8, 4, 64, 32, 16, "e4m3", "float16", [300, 20, 0], [2, 0, 3])
    host, q, table, cached, new, start = setup(case, 17)
    cache = host.device()
    args = (dev(table), dev(cached.astype(np.int32)))
    want = cache.attention(1, q.cuda(), *args, row_start=dev(start), max_rows=3)
    packed = t.zeros(7, 20, 64, dtype=t.float16, device="cuda")
    packed[:5, 3:11] = q.cuda()
    out = t.full((7, 8, 64), 7.0, dtype=t.float16, device="cuda")
    got = cache.attention(1, packed[:, 3:11], *args, row_start=dev(start), max_rows=16, out=out)
    cache.check()
    assert got is out and t.equal(out[:5], want) and bool((out[5:] == 7).all())
    for _ in range(3):
        assert t.equal(cache.attention(1, q.cuda(), *args, row_start=dev(start), max_rows=3), want)


def test_no_rows():
    t = torch()
    case = (4, 2, 64, 32, 16, "int8", "bfloat16", [40, 50], [0, 0])
    host, q, table, cached, new, start = setup(case, 18)
    cache = host.device()
    args = (dev(table), dev(cached.astype(np.int32)))
    out, lse = cache.attention(0, q.cuda(), *args, row_start=dev(start), max_rows=1, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    cache.store(0, q[:, :2].cuda(), q[:, :2].cuda(), *args, row_start=dev(start))
    # rows that belong to nobody, and a batch without any row in its sequences
    two = t.ones(2, 4, 64, device="cuda", dtype=t.bfloat16)
    out = t.full_like(two, 3.0)
    cache.attention(0, two, *args, row_start=dev(start), max_rows=1, out=out)
    before = [x.clone() for x in cache.pools()]
    cache.store(0, two[:, :2], two[:, :2], *args, row_start=dev(start))
    cache.check()
    assert bool((out == 3).all()) and all(t.equal(x, y) for x, y in zip(cache.pools(), before))


def test_the_binding_refuses():
    import persistent_runtime_b200 as prb
    t = torch()
    case = (4, 2, 64, 32, 16, "int8", "bfloat16", [40, 50], [1, 1])
    host, q, table, cached, new, start = setup(case, 18)
    cache = host.device()
    q, table, lens, start = q.cuda(), dev(table), dev(cached.astype(np.int32)), dev(start)
    k = t.zeros(2, 2, 64, device="cuda")
    bad = [lambda: cache.attention(1, q, table, lens, out=q), lambda: cache.attention(1, q.double(), table, lens),
           lambda: cache.attention(1, q, table.long(), lens), lambda: cache.attention(1, q, table, lens[:1]),
           lambda: cache.attention(1, q[:, :, :32], table, lens), lambda: cache.attention(1, q[:1], table, lens),
           lambda: cache.attention(1, q, table, lens, row_start=start), lambda: cache.attention(2, q, table, lens),
           lambda: cache.attention(1, q, table, lens, row_start=start, max_rows=17),
           lambda: cache.attention(1, q, table[:, ::2], lens), lambda: cache.attention(1, q[:, :3], table, lens),
           lambda: cache.attention(1, q.cpu(), table, lens), lambda: cache.attention(1, q, table, lens.cpu()),
           lambda: cache.attention(1, q, table, lens, out=t.zeros(2, 4, 64, device="cuda")),
           lambda: cache.store(1, k, k[:1], table, lens), lambda: cache.store(1, k, k.half(), table, lens),
           lambda: cache.store(1, k[:, :1], k[:, :1], table, lens), lambda: cache.store(-1, k, k, table, lens),
           lambda: cache.store(1, k[:1], k[:1], table, lens),
           lambda: cache.store(1, t.zeros(2, 2, 66, device="cuda")[:, :, 1:65], k, table, lens),
           lambda: prb.KV8Cache(cache.k, cache.v, cache.k_scale[:, :, :, :1], cache.v_scale),
           lambda: prb.KV8Cache(cache.k.float(), cache.v, cache.k_scale, cache.v_scale),
           lambda: prb.KV8Cache(cache.k, cache.v[:2], cache.k_scale, cache.v_scale),
           lambda: prb.KV8Cache.empty(4, 1, 2, 96), lambda: prb.KV8Cache.empty(4, 1, 2, 64, 64, 48)]
    for i, call in enumerate(bad):
        with pytest.raises(prb.MkError):
            call()
            pytest.fail(f"call {i} was not refused")
    cache.check()


def test_device_checks_make_the_sequence_nan():
    import persistent_runtime_b200 as prb
    t = torch()
    case = (4, 2, 64, 32, 16, "int8", "bfloat16", [600, 700, 40], [1, 1, 1])
    host, q, table, cached, new, start = setup(case, 18)
    cache = host.device()
    d_len = dev(cached.astype(np.int32))
    clean, clean_lse = cache.attention(1, q.cuda(), dev(table), d_len, return_lse=True)
    cap = table.shape[1] * 32
    for what, check_id in (("page", 3), ("negative", 2), ("long", 2)):
        tab, lens = table.copy(), cached.astype(np.int32).copy()
        if what == "page":
            tab[1, 9] = -1
        else:
            lens[1] = -1 if what == "negative" else cap
        out, lse = cache.attention(1, q.cuda(), dev(tab), dev(lens), return_lse=True)
        rc, d = cache.sync_status()
        assert rc == prb.MK_ERR_DEVICE and d[1] == 1 and d[3] == check_id
        assert t.equal(out[[0, 2]], clean[[0, 2]]) and bool(t.isnan(out[1]).all())
        assert t.equal(lse[[0, 2]], clean_lse[[0, 2]]) and bool(t.isnan(lse[1]).all())
        cache.reset()
    # more rows than max_rows
    q3 = t.cat([q, q]).cuda()
    out = cache.attention(1, q3, dev(table), dev(np.array([5, 6, 7], np.int32)),
                          row_start=dev(np.array([0, 1, 5, 6], np.int32)), max_rows=2)
    assert cache.sync_status()[1][3] == 1
    assert bool(t.isnan(out[1:5]).all()) and not bool(t.isnan(out[[0, 5]]).any())


def test_streams_graphs_and_two_calls_at_once():
    t = torch()
    case = (16, 8, 128, 64, 64, "int8", "bfloat16", [3000, 2500], [1, 1])
    host, q, table, cached, new, start = setup(case, 19)
    cache = host.device()
    a, d_table, d_len = q.cuda(), dev(table), dev(cached.astype(np.int32))
    b = (a * 0.5).contiguous()
    want = [cache.attention(1, x, d_table, d_len) for x in (a, b)]
    side = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    got = []
    for _ in range(5):
        for st, x in zip(side, (a, b)):
            with t.cuda.stream(st):
                got.append(cache.attention(1, x, d_table, d_len))
    got.append(cache.attention(1, a, d_table, d_len, stream=side[0]))
    t.cuda.synchronize()
    for i, x in enumerate(got[:-1]):
        assert t.equal(x, want[i % 2])
    assert t.equal(got[-1], want[0])
    graphs = []
    for x in (a, b):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            out = cache.attention(1, x, d_table, d_len)
        graphs.append((g, out))
    for _ in range(5):
        for (g, out), st in zip(graphs, side):
            out.zero_()
            t.cuda.synchronize()
        for (g, out), st in zip(graphs, side):
            with t.cuda.stream(st):
                g.replay()
        t.cuda.synchronize()
        for (g, out), w in zip(graphs, want):
            assert t.equal(out, w)
    cache.check()


def test_offsets_beyond_32_bits():
    """The last pages of pools of more than 2^32 codes: store, attention and page copies."""
    import persistent_runtime_b200 as prb
    t = torch()
    P, T, layers, H, D = 64, 64, 36, 8, 128
    n_pages = (1 << 32) // (layers * H * P * D) + 40
    if t.cuda.mem_get_info()[0] < 2 * n_pages * layers * H * P * D + (1 << 30):
        pytest.skip("not enough free device memory")
    cache = prb.KV8Cache.empty(n_pages, layers, H, D, P, T)
    lens, new = np.array([100, 30]), np.array([3, 1])
    pages = np.arange(n_pages - 3, n_pages, dtype=np.int32)
    assert (int(pages[0]) * layers + 35) * H * P * D > 1 << 32
    table = np.array([[pages[1], pages[2], -1], [pages[0], -1, -1]], np.int32)
    small = ref.Cache(3, 1, H, D, P, T, "int8", 20)  # the same pages as 0, 1, 2 of a small host cache
    for x, y in zip((cache.k, cache.v), small.codes):
        x[n_pages - 3:, 35] = t.from_numpy(y[:, 0].view(np.int8)).cuda()
    for x, y in zip((cache.k_scale, cache.v_scale), small.scales):
        x[n_pages - 3:, 35] = t.from_numpy(y[:, 0]).cuda()
    start = np.array([0, 3, 4], np.int32)
    rng = np.random.default_rng(21)
    k, v = (rng.standard_normal((4, H, D)).astype(np.float32) for _ in range(2))
    q = t.from_numpy(rng.standard_normal((4, 32, D)).astype(np.float32))
    d_len = dev(lens.astype(np.int32))
    cache.store(35, dev(k), dev(v), dev(table), d_len, row_start=dev(start))
    out, lse = cache.attention(35, q.cuda(), dev(table), d_len, row_start=dev(start), max_rows=3, return_lse=True)
    cache.check()
    small_table = [[1, 2], [0]]
    small.store(0, [k, v], small_table, lens.tolist(), start)
    check(out, lse, small, 0, q, np.array([[1, 2], [0, 0]]), lens, start, D ** -0.5, "float32")
    for x, y in zip((cache.k, cache.v), small.codes):
        np.testing.assert_array_equal(x[n_pages - 3:, 35].cpu().numpy().view(np.uint8), y[:, 0])
    held = prb.PagePool(dev(table), t.zeros(n_pages, dtype=t.int32, device="cuda"), P, cache.pools())
    held.copy(dev(pages[:1]), dev(np.array([5], np.int32)))
    held.check()
    assert t.equal(cache.k[5, 35], cache.k[n_pages - 3, 35]) and t.equal(cache.v_scale[5, 35], cache.v_scale[n_pages - 3, 35])


def test_a_given_stream_gets_memory_of_its_own():
    """What a call allocates must not be memory that was freed on the current stream, whose work may
    still be using it."""
    t = torch()
    case = (16, 8, 128, 64, 64, "int8", "bfloat16", [3000, 2500], [1, 1])
    host, q, table, cached, new, start = setup(case, 19)
    cache = host.device()
    args = 1, q.cuda(), dev(table), dev(cached.astype(np.int32))
    made, make = [], cache._bytes

    def spy(n):
        made.append(make(n))
        return made[-1]

    cache._bytes = spy
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    first = cache.attention(*args, return_lse=True)
    freed = {x.data_ptr() for x in (*first, *made)}
    want = [x.clone() for x in first]
    assert len(made) == 1
    del first
    made.clear()
    got = cache.attention(*args, return_lse=True, stream=side)
    assert len(made) == 1 and not freed & {x.data_ptr() for x in (*got, *made)}
    t.cuda.synchronize()
    for a, b in zip(got, want):
        assert t.equal(a, b)


@pytest.mark.parametrize("wide", [False, True])  # short tables (a CTA per pair), long ones
def test_many_failing_sequences_and_rows(wide):
    t = torch()
    rng = np.random.default_rng(5)
    n, bad = 200, [7, 40, 41, 199]
    lens = rng.integers(0, 600, n)
    new = np.ones(n, np.int64)
    new[7] = 3000  # far above max_rows
    new[150] = 2
    case = (4, 2, 64, 64, 32, "int8", "bfloat16", list(lens), list(new))
    case[7][7] = case[8][7] = 0  # the host's cache need not hold its rows
    case[8][7] = 1
    host, _, table, cached, _, _ = setup(case, 29)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = t.from_numpy(rng.standard_normal((start[-1], 4, 64)).astype(np.float32)).to(t.bfloat16)
    given = cached.astype(np.int32)
    given[bad[1:]] = -1
    tab = np.full((n, 200), -1, np.int32) if wide else table
    tab[:, :table.shape[1]] = table
    cache = host.device()
    out, lse = cache.attention(0, q.cuda(), dev(tab), dev(given), row_start=dev(start), max_rows=2, return_lse=True)
    assert cache.sync_status()[1][1] in bad
    owner = np.repeat(np.arange(n), new)
    fails = t.from_numpy(np.isin(owner, bad)).cuda()
    assert bool(t.isnan(out[fails]).all()) and bool(t.isnan(lse[fails]).all())
    good = np.setdiff1d(np.arange(n), bad)
    check(out[~fails], lse[~fails], host, 0, q[~fails.cpu()], table[good], cached[good],
          np.concatenate([[0], np.cumsum(new[good])]), 64 ** -0.5, "bfloat16")


@pytest.mark.parametrize("dim,fmt,dtype,wide", [(64, "int8", "bfloat16", False), (64, "e4m3", "float32", True),
                                                (64, "int8", "float32", True), (64, "e4m3", "float16", True),
                                                (128, "int8", "float16", False), (128, "e4m3", "bfloat16", False)])
def test_more_pairs_than_ctas(dim, fmt, dtype, wide):
    rng = np.random.default_rng(dim)
    cached = rng.integers(0, 70, 340)
    cached[[3, 200]] = 900
    if wide:  # longer than a whole CTA's share of the line
        cached[[17, 339]] = 6000, 2500
    case = (4, 2, dim, 32, 16, fmt, dtype, list(cached), [1] * 340)
    host, q, table, cached, new, start = setup(case, 31)
    cache = host.device()
    out, lse = cache.attention(1, q.cuda(), dev(table), dev(cached.astype(np.int32)), return_lse=True)
    cache.check()
    check(out, lse, host, 1, q, table, cached, start, dim ** -0.5, dtype)
