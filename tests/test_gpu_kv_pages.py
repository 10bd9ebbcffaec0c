"""The page calls against a sequential restatement: tables, counts and contents, exactly."""
import numpy as np
import pytest

import kv8_ref as ref
from kv8_ref import dev, torch

pytestmark = pytest.mark.gpu


class Host:
    """Tables, counts and pools on the host; a page's contents are a number in every pool."""

    def __init__(self, n_seqs, max_pages, page, n_pages, seed=0):
        self.page, self.n_pages = page, n_pages
        self.table = np.full((n_seqs, max_pages), -1, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        rng = np.random.default_rng(seed)
        # 16-byte pages, pages with a 4-byte rest, pages longer than a copy step
        self.pools = [rng.integers(0, 1 << 30, (n_pages, w)).astype(np.int32) for w in (4, 7, 8200 + 1024, 9001)]

    def hold(self, s, pages):
        self.table[s, :len(pages)] = pages
        np.add.at(self.ref, pages, 1)

    def device(self):
        import persistent_runtime_b200 as prb
        return prb.PagePool(dev(self.table), dev(self.ref), self.page, [dev(p) for p in self.pools])

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            self.table[d] = self.table[s]
            for p in self.table[s]:
                if p >= 0:
                    self.ref[p] += 1

    def free(self, seqs):
        for s in seqs:
            for p in self.table[s]:
                if p >= 0:
                    self.ref[p] -= 1
            self.table[s] = -1

    def reserve(self, kv_len, n_new):
        free = [p for p in range(self.n_pages) if self.ref[p] == 0]
        P = self.page
        entries = [(s, j) for s in range(len(kv_len)) if n_new[s] > 0
                   for j in range(kv_len[s] // P, -(-(kv_len[s] + n_new[s]) // P))]
        writers = {}
        for s, j in entries:
            if self.table[s, j] >= 0:
                writers.setdefault(self.table[s, j], []).append((s, j))
        start = self.ref.copy()
        for s, j in entries:
            p = self.table[s, j]
            if p >= 0 and (start[p] == 1 or (len(writers[p]) == start[p] and writers[p][-1] == (s, j))):
                continue
            fresh = free.pop(0)
            self.table[s, j], self.ref[fresh] = fresh, 1
            if p >= 0:
                self.ref[p] -= 1
                if j * P < kv_len[s]:
                    for pool in self.pools:
                        pool[fresh] = pool[p]

    def compact(self):
        used = [p for p in range(self.n_pages) if self.ref[p] > 0]
        U = len(used)
        to = dict(zip([p for p in used if p >= U], [p for p in range(U) if self.ref[p] == 0]))
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
            for pool in self.pools:
                pool[b] = pool[a]
        self.table = np.array([[to.get(p, p) for p in row] for row in self.table], np.int32)


def same(host, pages):
    pages.check()
    np.testing.assert_array_equal(pages.page_table.cpu().numpy(), host.table)
    np.testing.assert_array_equal(pages.ref_count.cpu().numpy(), host.ref)
    for got, want in zip(pages.pools, host.pools):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    named = np.bincount(host.table[host.table >= 0], minlength=host.n_pages)
    np.testing.assert_array_equal(host.ref, named)


def i32(x):
    return dev(np.array(x, np.int32))


@pytest.mark.parametrize("n_seqs,max_pages,page,n_pages,seed", [(3, 4, 16, 20, 0), (40, 9, 64, 300, 1),
                                                              (700, 5, 16, 5000, 2), (9, 2000, 16, 40000, 3)])
def test_a_life_of_sequences(n_seqs, max_pages, page, n_pages, seed):
    """Reserve, fork, write on, free and compact in random order, as a server does."""
    rng = np.random.default_rng(seed)
    host = Host(n_seqs, max_pages, page, n_pages, seed)
    if n_pages > 10000:  # contents of a few words are enough here
        host.pools = host.pools[:2]
    pages = host.device()
    lens = np.zeros(n_seqs, np.int64)
    for step in range(12):
        n_new = rng.integers(0, 3 * page, n_seqs) * (rng.random(n_seqs) < 0.7)
        n_new = np.minimum(n_new, max_pages * page - lens)
        need = sum(-(-(int(c) + int(n)) // page) - int(c) // page for c, n in zip(lens, n_new) if n > 0)
        if need <= (host.ref == 0).sum():
            host.reserve(lens.tolist(), n_new.tolist())
            pages.reserve(i32(lens), i32(n_new))
            same(host, pages)
            lens += n_new
        empty = np.flatnonzero(lens == 0)
        full = np.flatnonzero(lens > 0)
        if len(empty) and len(full):
            k = rng.integers(1, len(empty) + 1)
            dst = rng.permutation(empty)[:k]
            src = rng.choice(full, k)
            host.fork(src, dst)
            pages.fork(i32(src), i32(dst))
            same(host, pages)
            lens[dst] = lens[src]
            # forked sequences may be cut back: their next rows land in shared pages
            lens[dst] -= rng.integers(0, 1 + lens[dst])
            for s in dst:
                lens[s] = max(lens[s], 1)
        gone = np.flatnonzero(rng.random(n_seqs) < 0.3)
        if len(gone):
            twice = np.concatenate([gone, gone[:2]])  # a sequence may be named twice
            host.free(gone)
            pages.free(i32(twice))
            same(host, pages)
            lens[gone] = 0
        if step % 3 == 2:
            host.compact()
            pages.compact()
            same(host, pages)
            used = int((host.ref > 0).sum())
            assert (host.ref[:used] > 0).all()


def test_all_holders_write_the_last_keeps_the_page():
    host = Host(5, 3, 16, 12)
    host.hold(0, [7, 3])
    pages = host.device()
    host.fork([0, 0], [2, 4])
    pages.fork(i32([0, 0]), i32([2, 4]))
    host.reserve([20, 0, 20, 0, 20], [1, 0, 1, 0, 1])
    pages.reserve(i32([20, 0, 20, 0, 20]), i32([1, 0, 1, 0, 1]))
    same(host, pages)
    assert host.table[4, 1] == 3 and host.table[0, 1] != 3 and host.ref[3] == 1
    # only one of two holders writes: the other keeps the page
    host.fork([2], [1])
    pages.fork(i32([2]), i32([1]))
    host.reserve([0, 21, 0, 0, 0], [0, 1, 0, 0, 0])
    pages.reserve(i32([0, 21, 0, 0, 0]), i32([0, 1, 0, 0, 0]))
    same(host, pages)


def test_copy():
    host = Host(1, 1, 16, 50)
    pages = host.device()
    src, dst = [3, 3, 9, 49], [0, 48, 4, 17]
    pages.copy(i32(src), i32(dst))
    for pool in host.pools:
        pool[dst] = pool[src]
    same(host, pages)
    pages.copy(i32([]), i32([]))
    same(host, pages)


def test_failures_change_nothing():
    import persistent_runtime_b200 as prb

    def fails(call, check, code=prb.MK_ERR_DEVICE):
        call()
        rc, d = pages.sync_status()
        assert rc == code and d[3] == check, (rc, d)
        pages.reset()
        same(host, pages)
        return d

    host = Host(4, 3, 16, 8)
    host.hold(0, [5, 2])
    host.hold(1, [6])
    pages = host.device()
    fails(lambda: pages.fork(i32([0, 1]), i32([2, 2])), 4)
    fails(lambda: pages.fork(i32([0, 2]), i32([2, 3])), 4)
    fails(lambda: pages.fork(i32([0]), i32([4])), 4)
    fails(lambda: pages.fork(i32([-1]), i32([2])), 4)
    fails(lambda: pages.fork(i32([0]), i32([1])), 5)
    fails(lambda: pages.free(i32([0, 4])), 4)
    fails(lambda: pages.copy(i32([0]), i32([8])), 4)
    fails(lambda: pages.copy(i32([0, 1]), i32([3, 3])), 4)
    fails(lambda: pages.copy(i32([0, 1]), i32([1, 3])), 4)
    fails(lambda: pages.reserve(i32([0, 0, -1, 0]), i32([0, 0, 1, 0])), 2)
    fails(lambda: pages.reserve(i32([0, 0, 40, 0]), i32([0, 0, 9, 0])), 2)
    d = fails(lambda: pages.reserve(i32([32, 16, 0, 0]), i32([16, 32, 48, 1])), 6, prb.MK_ERR_OOM)
    assert d[2] == 1 + 2 + 3 + 1 - 5
    pages.reserve(i32([32, 16, 0, 0]), i32([16, 32, 0, 32]))  # exactly the free ones
    host.reserve([32, 16, 0, 0], [16, 32, 0, 32])
    same(host, pages)
    for bad, calls in ((8, ("fork", "free", "reserve", "compact")), (-2, ("fork", "free", "reserve", "compact"))):
        pages.page_table[0, 2] = bad
        host.table[0, 2] = bad
        for name in calls:
            {"fork": lambda: pages.fork(i32([0]), i32([2])), "free": lambda: pages.free(i32([1, 0])),
             "reserve": lambda: pages.reserve(i32([32, 0, 0, 0]), i32([1, 0, 0, 0])),
             "compact": pages.compact}[name]()
            rc, d = pages.sync_status()
            assert rc == prb.MK_ERR_DEVICE and d[3] == 3
            pages.reset()
            np.testing.assert_array_equal(pages.page_table.cpu().numpy(), host.table)
            np.testing.assert_array_equal(pages.ref_count.cpu().numpy(), host.ref)
    pages.page_table[0, 2] = 0
    pages.ref_count[0] = 0  # an entry that names a free page
    pages.compact()
    assert pages.sync_status()[1][3] == 3


@pytest.mark.parametrize("n_pages", [9, 4200])  # one CTA, two
def test_reserve_without_room_for_shared_pages(n_pages):
    """Too few free pages while several sequences write shared pages: nothing is copied, whatever an earlier call
    has left in the workspace."""
    import persistent_runtime_b200 as prb

    host = Host(7, n_pages, 16, 9)
    host.n_pages, host.ref = n_pages, np.zeros(n_pages, np.int32)
    host.pools = [np.arange(n_pages * w, dtype=np.int32).reshape(n_pages, w) for w in (4, 1027)]
    used = n_pages - 4
    host.hold(0, [0, 1, 2])
    host.hold(1, [3])
    host.hold(6, range(4, used))
    pages = host.device()
    fork = [0, 0, 1], [2, 3, 4]
    pages.fork(*map(i32, fork))
    host.fork(*fork)
    lens, new = [40, 5, 40, 40, 5, 0, 0], [1, 0, 1, 0, 1, 0, 0]
    pages.reserve(i32(lens), i32(new))  # three copies, listed in the workspace
    host.reserve(lens, new)
    same(host, pages)
    for pool, dev_pool in zip(host.pools, pages.pools):  # a repeated copy would show
        pool += 1
        dev_pool += 1
    fork = [0, 1], [2, 4]
    pages.free(i32([2, 4]))
    host.free([2, 4])
    pages.fork(*map(i32, fork))
    host.fork(*fork)
    for lens, new in (([3, 3, 3, 3, 3, 0, 0], [1, 1, 1, 1, 1, 64, 0]), ([0] * 7, [48, 16, 48, 48, 16, 64, 16])):
        pages.reserve(i32(lens), i32(new))
        rc, d = pages.sync_status()
        assert rc == prb.MK_ERR_OOM and d[3] == 6
        pages.reset()
        same(host, pages)


def test_captured_calls_and_another_stream():
    t = torch()
    host = Host(6, 4, 16, 30)
    host.hold(0, [20, 21, 29])
    host.hold(1, [11])
    pages = host.device()
    src, dst, lens, new = i32([0, 0]), i32([2, 3]), i32([40, 3, 40, 40, 0, 0]), i32([1, 1, 1, 1, 0, 20])
    gone = i32([0])
    pages.fork(src, dst)  # warm-up outside the capture, taken back
    pages.free(dst)
    table0, ref0 = pages.page_table.clone(), pages.ref_count.clone()
    pools0 = [p.clone() for p in pages.pools]
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        pages.fork(src, dst)
        pages.reserve(lens, new)
        pages.free(gone)
        pages.compact()
    host.fork([0, 0], [2, 3])
    host.reserve([40, 3, 40, 40, 0, 0], [1, 1, 1, 1, 0, 20])
    host.free([0])
    host.compact()
    for _ in range(3):
        pages.page_table.copy_(table0)
        pages.ref_count.copy_(ref0)
        for p, p0 in zip(pages.pools, pools0):
            p.copy_(p0)
        g.replay()
        same(host, pages)
    st = t.cuda.Stream()
    st.wait_stream(t.cuda.current_stream())
    pages.page_table.copy_(table0)
    pages.ref_count.copy_(ref0)
    for p, p0 in zip(pages.pools, pools0):
        p.copy_(p0)
    t.cuda.synchronize()
    pages.fork(src, dst, stream=st)
    pages.reserve(lens, new, stream=st)
    pages.free(gone, stream=st)
    pages.compact(stream=st)
    same(host, pages)


def test_the_binding_refuses():
    import persistent_runtime_b200 as prb
    t = torch()
    host = Host(4, 3, 16, 8)
    pages = host.device()
    table, counts, pool = pages.page_table, pages.ref_count, pages.pools[0]
    bad = [lambda: pages.fork(i32([0]), i32([1, 2])), lambda: pages.fork(i32([0]).long(), i32([1])),
           lambda: pages.free(i32([0]).cpu()), lambda: pages.reserve(i32([0]), i32([1, 1, 1, 1])),
           lambda: pages.copy(i32([0, 1, 2, 3])[::2], i32([4, 5])),
           lambda: prb.PagePool(table, counts, 16, [pool[:7]]), lambda: prb.PagePool(table, counts, 0, [pool]),
           lambda: prb.PagePool(table, counts.float(), 16, [pool]), lambda: prb.PagePool(table[0], counts, 16, [pool]),
           lambda: prb.PagePool(table, counts, 16, [pool] * 9), lambda: prb.PagePool(table, counts, 16, [pool.t()]),
           lambda: prb.PagePool(table, counts, 16, [t.zeros(8, 3, dtype=t.int8, device="cuda")])]
    for i, call in enumerate(bad):
        with pytest.raises(prb.MkError):
            call()
            pytest.fail(f"call {i} was not refused")
    same(host, pages)


@pytest.mark.usefixtures("built_libs")
def test_the_paged_step_on_shared_pages():
    """Sequences forked between steps of mk_decode_steps_paged: bitwise the contiguous step on
    caches that are copied."""
    import persistent_runtime_b200 as prb
    import synth
    from gpu_helpers import dev_weights
    t = torch()
    B, P, cap = 3, 64, 200
    w = synth.TINY.with_(name="tiny-b3", batch=B, kv_len=0, steps=1)
    weights = dev_weights(synth.make_weights(w, 8))
    flat, paged = prb.Megakernel(w, cap, 0), prb.Megakernel(w, cap, 0, kv_page_size=P)
    flat.load_weights(weights)
    paged.load_weights(weights)
    k, v = (t.zeros(w.n_layers, B, w.n_kv_heads, cap, w.head_dim, dtype=t.int16, device="cuda") for _ in range(2))
    pools = [t.zeros(10, w.n_layers, w.n_kv_heads, P, w.head_dim, dtype=t.int16, device="cuda") for _ in range(2)]
    pages = prb.PagePool.empty(B, -(-cap // P), P, pools)
    ones = i32([1] * B)
    tok_f, len_f, out_f = i32([5, 9, 11]), i32([0, 0, 0]), t.zeros(B, w.vocab, device="cuda")
    tok_p, len_p, out_p = tok_f.clone(), len_f.clone(), out_f.clone()

    def steps(n):
        for _ in range(n):
            pages.reserve(len_p, ones)
            paged.decode_steps_paged(1, tok_p, tok_p, len_p, *pools, 10, pages.page_table, out_p)
            flat.decode_step(tok_f, tok_f, len_f, k, v, out_f)
            assert t.equal(tok_f, tok_p) and t.equal(out_f, out_p) and t.equal(len_f, len_p)
        assert paged.sync_status()[0] == 0 and flat.sync_status()[0] == 0
        pages.check()

    steps(70)
    for a, b in ((0, 2), (2, 1)):  # one continued as two, then again
        pages.free(i32([b]))
        pages.fork(i32([a]), i32([b]))
        for x in (k, v):
            x[:, b] = x[:, a]
        for length in (len_f, len_p):
            length[b] = length[a]
        for tok in (tok_f, tok_p):
            tok[b] = (int(tok[a]) + 1) % w.vocab
        steps(3)
        assert int(pages.ref_count.max()) > 1
        pages.compact()
        steps(30)
    flat.close()
    paged.close()


def test_a_given_stream_gets_a_workspace_of_its_own():
    t = torch()
    host = Host(3, 4, 16, 8)
    host.hold(0, [5, 2])
    pages = host.device()
    made, make = [], pages._bytes

    def spy(n):
        made.append(make(n))
        return made[-1]

    pages._bytes = spy
    side = t.cuda.Stream()
    pages.fork(i32([0]), i32([1]))
    host.fork([0], [1])
    freed = made.pop().data_ptr()
    src, dst = i32([0]), i32([2])
    t.cuda.synchronize()
    pages.fork(src, dst, stream=side)
    host.fork([0], [2])
    assert made.pop().data_ptr() != freed
    same(host, pages)
