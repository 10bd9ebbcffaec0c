"""What the attention's fixed-point and fp16 probabilities cost, on inputs whose scores are exact
but for a few roundings, so that little else is left in the error."""
import numpy as np
import pytest

from kv8_ref import dev, encode, torch

pytestmark = pytest.mark.gpu


def one_hot_cache(n, fmt, k_code, k_scale, v_code, v_scale, D=64, T=16):
    """n sequences of one page of T positions; K is k_code [n][T] in dim 0, V is v_code in all dims."""
    import persistent_runtime_b200 as prb
    t = torch()
    kind = t.int8 if fmt == "int8" else t.float8_e4m3fn
    codes = np.zeros((2, n, 1, 1, T, D), np.uint8)
    codes[0, :, 0, 0, :, 0] = encode(k_code.astype(np.float32), fmt)
    codes[1, :, 0, 0] = encode(v_code.astype(np.float32), fmt)[:, :, None]
    scales = [np.broadcast_to(np.float32(x), n).astype(np.float32).reshape(n, 1, 1, 1) for x in (k_scale, v_scale)]
    return prb.KV8Cache(*(dev(c).view(kind) for c in codes), *(dev(s) for s in scales))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_scores_a_little_below_the_largest(fmt, dtype):
    """Position 0 has score 0 and value 1, the positions 1 to 3 a score x in (-0.17, 0] and value 0:
    the output is 1 / (1 + 3 e^x), the log-sum-exp log(1 + 3 e^x).

    Bounds, with u = 2^-24.  The score in base 2 has at most 0.25 and four roundings (the factor's
    constant and its two products, the sum's product): u ln 2 of e^x.  The exponential is off by 2 ulp
    of a value in (0.84, 1], 2 u / 0.84; together 3.1 u of e^x, and 0.75 times that of the sum, whose
    two additions add 2 u: 4.4 u.  The output (fp32 rows) adds a reciprocal and a product, and the
    reciprocal's factor may have been rounded once: 7.4 u.  The logarithm, at most 1.4 (2 in base 2),
    is off by an ulp of 2^-23, and its product with ln 2 by a rounding of each: 4.4 u + 1.4 * 4 u."""
    t = torch()
    u = 2.0 ** -24
    n = 2000
    rng = np.random.default_rng(4)
    code = np.zeros((n, 16))
    code[:, 1:4] = -104 if fmt == "int8" else -104.0  # a value of both types
    k_scale = (rng.random(n) * 0.17 / 104).astype(np.float32)
    value = np.zeros((n, 16))
    value[:, 0] = 64
    cache = one_hot_cache(n, fmt, code, k_scale, value, 2.0 ** -6)
    q = t.zeros(n, 1, 64, dtype=getattr(t, dtype), device="cuda")
    q[:, :, 0] = 1.0
    table = dev(np.arange(n, dtype=np.int32).reshape(n, 1))
    out, lse = cache.attention(0, q, table, dev(np.full(n, 3, np.int32)), scale=1.0, return_lse=True)
    cache.check()
    total = 1.0 + 3.0 * np.exp(-104.0 * k_scale.astype(np.float64))
    lse = lse.double().cpu().numpy()[:, 0]
    assert np.abs(lse - np.log(total)).max() <= 10.0 * u
    if dtype == "float32":
        got = out.double().cpu().numpy()[:, 0]
        assert (np.abs(got * total[:, None] - 1.0)).max() <= 7.4 * u


RANGE_CASES = [
    # q heads, kv heads, dim, page, block, cached, new rows
    (4, 2, 64, 64, 16, [40, 333], [1, 1]),             # whole pairs
    (8, 1, 128, 64, 64, [5000, 700], [1, 2]),          # cut ones
    (16, 1, 64, 32, 16, [900, 30], [3, 1]),            # sixteen rows
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("case", RANGE_CASES, ids=["whole", "cut", "rows16"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_large_and_small_values(case, fmt, dtype):
    """Values times a power of two give the output times that power, bit for bit, as long as the
    values' sum and the scales stay in fp32's normal range: each operation commutes with it."""
    import kv8_ref as ref
    t = torch()
    Hq, H, D, P, T, cached, new = case
    cached, new = np.array(cached), np.array(new)
    table, n_pages = ref.make_table(cached + new, P, seed=3)
    host = ref.Cache(n_pages, 1, H, D, P, T, fmt, 5)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = t.from_numpy(np.random.default_rng(6).standard_normal((start[-1], Hq, D)).astype(np.float32))
    args = (q.to(getattr(t, dtype)).cuda(), dev(table), dev(cached.astype(np.int32)))

    def run(power):
        cache = host.device()
        cache.v_scale *= 2.0 ** power
        out, lse = cache.attention(0, *args, row_start=dev(start), max_rows=int(new.max()), return_lse=True)
        cache.check()
        return out.double(), lse

    want, want_lse = run(0)
    # e4m3 values are up to 448 (0.7 + 0.6) / 90 = 6.5, int8 1.9; 5001 of them sum to 2^15 at most
    for power in (112, 100, 60, -60, -90):
        out, lse = run(power)
        assert t.equal(out, want * 2.0 ** power), power
        assert t.equal(lse, want_lse)
