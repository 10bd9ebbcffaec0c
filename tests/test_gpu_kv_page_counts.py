"""Page tables that name a page whose count is not positive: every call that would act on such
an entry refuses, and changes nothing."""
import numpy as np
import pytest

from kv8_ref import dev, torch

pytestmark = pytest.mark.gpu


def i32(x):
    return dev(np.array(x, np.int32))


@pytest.mark.parametrize("n_pages", [8, 5000])  # one CTA, two
@pytest.mark.parametrize("count", [0, -1])
@pytest.mark.parametrize("call", ["fork", "free", "reserve", "compact"])
def test_an_entry_that_names_a_free_page(call, count, n_pages):
    import persistent_runtime_b200 as prb
    t = torch()
    table = np.full((4, 3), -1, np.int32)
    table[0, :2] = 5, 2
    table[1, :1] = 6
    counts = np.zeros(n_pages, np.int32)
    counts[[5, 6]] = 1
    counts[2] = count
    pool = dev(np.arange(n_pages * 4, dtype=np.int32).reshape(n_pages, 4))
    before = pool.clone()
    pages = prb.PagePool(dev(table), dev(counts), 16, [pool])
    {"fork": lambda: pages.fork(i32([1, 0]), i32([2, 3])), "free": lambda: pages.free(i32([1, 0])),
     "reserve": lambda: pages.reserve(i32([20, 0, 0, 0]), i32([1, 0, 40, 0])), "compact": pages.compact}[call]()
    rc, d = pages.sync_status()
    assert rc == prb.MK_ERR_DEVICE and d == [rc, 0, 2, 3]
    np.testing.assert_array_equal(pages.page_table.cpu().numpy(), table)
    np.testing.assert_array_equal(pages.ref_count.cpu().numpy(), counts)
    assert t.equal(pool, before)
    # what does not act on the entry goes on
    pages.reset()
    if call in ("free", "reserve"):
        if call == "free":
            pages.free(i32([1]))
            table[1], counts[6] = -1, 0
        else:
            pages.reserve(i32([5, 0, 0, 0]), i32([1, 0, 17, 0]))
            free = np.flatnonzero(counts == 0)[:2]
            table[2, :2], counts[free] = free, 1
        pages.check()
        np.testing.assert_array_equal(pages.page_table.cpu().numpy(), table)
        np.testing.assert_array_equal(pages.ref_count.cpu().numpy(), counts)
