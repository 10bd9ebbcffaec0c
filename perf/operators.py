"""The operators of the 8-bit paged K/V cache, as they are measured.

Four kinds of call:
  store    quantise new K/V rows and append them to a paged 8-bit cache that keeps one scale for every `block`
           positions of a (page, layer, head)
  attend   attention of new query rows over such a cache
  branch   fork sequences (their pages are shared) and reserve a token for each: shared pages that are about to be
           written are copied first
  compact  free sequences and move the pages that are left to the lowest page numbers

Where `own` is false, run() computes them with elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

INT8_MAX, E4M3_MAX, SCALE_MIN = 127.0, 448.0, 2.0 ** -126
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a decode step of the tiny decoder: one new row, the smallest call
        dict(name="store one token", kind="store", batch=1, past=33, rows=1, kv_heads=2, dim=64, page=64, block=16,
             layers=2, format="int8", dtype="bf16"),
        # a decode step of the 8B decoder at batch 16; the step's own rows are fp32
        dict(name="store a token of each", kind="store", batch=16, past=8192, rows=1, kv_heads=8, dim=128, page=64,
             block=64, layers=1, format="e4m3", dtype="f32"),
        # prompts of uneven lengths on their way into the cache
        dict(name="store prompts", kind="store", batch=16, past=100, rows=8192, kv_heads=8, dim=128, page=128,
             block=32, layers=1, format="int8", dtype="bf16"),
        # the tiny decoder's step: latency alone
        dict(name="attend short", kind="attend", batch=1, kv=33, mixed=False, new=1, q_heads=4, kv_heads=2, dim=64,
             page=64, block=16, layers=2, format="int8", dtype="bf16"),
        # the 8B decoder at batch 8, lengths 256 to 4096, fp32 queries as the step has them
        dict(name="attend batch 8", kind="attend", batch=8, kv=4096, mixed=True, new=1, q_heads=32, kv_heads=8, dim=128,
             page=64, block=64, layers=1, format="int8", dtype="f32"),
        # the 8B decoder at batch 16, every sequence at 8192
        dict(name="attend batch 16", kind="attend", batch=16, kv=8192, mixed=False, new=1, q_heads=32, kv_heads=8,
             dim=128, page=64, block=64, layers=1, format="int8", dtype="bf16"),
        # drafted tokens that are checked together, small pages, odd sizes
        dict(name="attend drafts", kind="attend", batch=7, kv=6001, mixed=True, new=5, q_heads=16, kv_heads=8, dim=128,
             page=16, block=16, layers=1, format="e4m3", dtype="f16"),
        # one long document
        dict(name="attend long", kind="attend", batch=1, kv=131071, mixed=False, new=1, q_heads=32, kv_heads=8, dim=128,
             page=128, block=128, layers=1, format="e4m3", dtype="bf16"),
        # a request that is continued four ways, tiny pools in bf16
        dict(name="branch one", kind="branch", groups=1, ways=4, past=150, kv_heads=2, dim=64, page=64, layers=2,
             block=0),
        # a batch of prompts, each continued four ways, 8-bit pools of the 8B decoder
        dict(name="branch a batch", kind="branch", groups=32, ways=4, past=700, kv_heads=8, dim=128, page=64, layers=36,
             block=64),
        # a small pool after half its sequences have ended
        dict(name="compact small", kind="compact", batch=9, past=300, kv_heads=8, dim=128, page=64, layers=2, block=0),
        # the 8B decoder's 8-bit pools after half the sequences have ended
        dict(name="compact large", kind="compact", batch=32, past=1000, kv_heads=8, dim=128, page=64, layers=36,
             block=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["store", "store", "attend", "attend", "attend", "branch", "compact"])
    dim = rng.choice([64, 128])
    block = rng.choice([16, 32, 64, 128])
    page = block * rng.choice([1, 1, 2, 4])
    q_heads, kv_heads = rng.choice([(4, 2), (16, 8), (32, 8), (8, 8), (16, 1), (24, 2), (40, 8)])
    format = rng.choice(["int8", "e4m3"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if kind == "store":
        rows = rng.choice([1, _log(rng, 2, 4096)])
        return dict(kind=kind, batch=_log(rng, 1, 64 if rows == 1 else max(1, min(64, 65536 // rows))),
                    past=_log(rng, 1, 4096), rows=rows, kv_heads=kv_heads, dim=dim, page=page, block=block,
                    layers=rng.choice([1, 2]), format=format, dtype=dtype)
    if kind == "attend":
        kv = _log(rng, 1, 65536)
        return dict(kind=kind, batch=_log(rng, 1, max(1, min(64, 131072 // kv))), kv=kv, mixed=rng.random() < 0.5,
                    new=rng.choice([1, 1, 2, 3, 4, 7, 8]), q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page,
                    block=block, layers=1, format=format, dtype=dtype)
    layers = rng.choice([2, 8, 28])
    if kind == "branch":
        return dict(kind=kind, groups=_log(rng, 1, 32), ways=rng.randint(2, 5), past=_log(rng, 1, 700),
                    kv_heads=kv_heads, dim=dim, page=64, layers=layers, block=rng.choice([0, 16, 64]))
    return dict(kind=kind, batch=_log(rng, 2, 32), past=_log(rng, 64, 1000), kv_heads=kv_heads, dim=dim, page=64,
                layers=layers, block=rng.choice([0, 16, 64]))


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)


def _codes(shape, format, g):
    """A cache's 8-bit contents with a standard deviation near 1 once scaled, and the scales' mean size."""
    if format == "int8":
        return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8), 1.0 / 73.0
    x = torch.empty(shape, device="cuda", dtype=torch.float8_e4m3fn)
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 26):
        part = flat[at:at + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(110.0).clamp_(-E4M3_MAX, E4M3_MAX))
    return x, 1.0 / 110.0


def _table(lens, page, spare, g):
    """Page tables for sequences of `lens` positions, pages in random order; entries that are not used are -1."""
    used = [-(-n // page) for n in lens]
    width, n_pages = max(used) + 1, sum(used) + spare
    order = torch.randperm(n_pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(lens), width), -1, device="cuda", dtype=torch.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    return table, n_pages


def _lengths(n, g, *ranges):
    """A tensor of n lengths for each (lo, hi): the case's own numbers, so that the pools have one size, in the order
    that the seed gives.  The first range's first length is hi."""
    rng = random.Random(n)
    drawn = [[rng.randint(lo, hi) for _ in range(n)] for lo, hi in ranges]
    drawn[0][0] = ranges[0][1]
    order = torch.randperm(n, generator=g, device="cuda")
    return [torch.tensor(d, device="cuda", dtype=torch.int32)[order] for d in drawn]


def _cache(case, lens, g):
    table, n_pages = _table(lens, case["page"], 3, g)
    shape = (n_pages, case["layers"], case["kv_heads"], case["page"], case["dim"])
    s = {"page_table": table}
    for name in ("k", "v"):
        s[name], size = _codes(shape, case["format"], g)
        scales = (n_pages, case["layers"], case["kv_heads"], case["page"] // case["block"])
        s[name + "_scale"] = size * (0.7 + 0.6 * torch.rand(scales, generator=g, device="cuda"))
    if own:
        import persistent_runtime_b200 as prb
        s["cache"] = prb.KV8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


def _prepare_store(case, g):
    B, n = case["batch"], case["rows"]
    rows, past = _lengths(B, g, (n // 2 if n > 1 else 1, n), (case["past"] // 2, case["past"]))
    lens = (past + rows).tolist()
    s = _cache(case, lens, g)
    start = torch.zeros(B + 1, device="cuda", dtype=torch.int32)
    start[1:] = rows.cumsum(0)
    total = sum(lens) - int(past.sum())
    shape = (total, case["kv_heads"], case["dim"])
    s.update(kv_len=past, row_start=start if n > 1 else None, layer=case["layers"] - 1)
    for name in ("new_k", "new_v"):
        s[name] = torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    return s


def _prepare_attend(case, g):
    B, n, kv = case["batch"], case["new"], case["kv"]
    rows, past = _lengths(B, g, (0 if n > 1 else 1, n), (kv // 16 if case["mixed"] else kv, kv))
    s = _cache(case, (past + rows).tolist(), g)
    start = torch.zeros(B + 1, device="cuda", dtype=torch.int32)
    start[1:] = rows.cumsum(0)
    s.update(kv_len=past, row_start=start if n > 1 else None, max_rows=n, layer=case["layers"] - 1)
    shape = (int(start[-1]), case["q_heads"], case["dim"])
    s["q"] = torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    return s


def _pools(case, n_pages, g):
    """The pools of a decoder's pages: bf16 K and V (block 0), or 8-bit K and V and their scales."""
    shape = (n_pages, case["layers"], case["kv_heads"], case["page"], case["dim"])
    if not case["block"]:
        return [torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    scales = shape[:3] + (case["page"] // case["block"],)
    return ([torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8) for _ in range(2)] +
            [torch.rand(scales, generator=g, device="cuda") for _ in range(2)])


def _page_state(case, table, ref, n_pages, g):
    s = dict(table0=table, ref0=ref, pools=_pools(case, n_pages, g), page=case["page"])
    s["page_table"], s["ref_count"] = table.clone(), ref.clone()
    if own:
        import persistent_runtime_b200 as prb
        s["pages"] = prb.PagePool(s["page_table"], s["ref_count"], case["page"], s["pools"])
    return s


def _prepare_branch(case, g):
    G, W = case["groups"], case["ways"]
    past, = _lengths(G, g, (case["past"] // 2, case["past"]))
    parents, n_pages = _table(past.tolist(), case["page"], G * W + 2, g)
    table = torch.full((G * W, parents.shape[1] + 1), -1, device="cuda", dtype=torch.int32)
    table[:G, :-1] = parents
    ref = torch.zeros(n_pages, device="cuda", dtype=torch.int32)
    ref[table[table >= 0].long()] = 1
    s = _page_state(case, table, ref, n_pages, g)
    s["src"] = torch.arange(G, device="cuda", dtype=torch.int32).repeat(W - 1)
    s["dst"] = torch.arange(G, G * W, device="cuda", dtype=torch.int32)
    s["kv_len"] = past.repeat(W)
    s["n_new"] = torch.ones(G * W, device="cuda", dtype=torch.int32)
    return s


def _prepare_compact(case, g):
    B = case["batch"]
    past, = _lengths(B, g, (case["past"] // 2, case["past"]))
    table, n_pages = _table(past.tolist(), case["page"], 2, g)
    ref = torch.zeros(n_pages, device="cuda", dtype=torch.int32)
    ref[table[table >= 0].long()] = 1
    s = _page_state(case, table, ref, n_pages, g)
    s["seqs"] = torch.randperm(B, generator=g, device="cuda", dtype=torch.int32)[:max(1, B // 2)].contiguous()
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = {"store": _prepare_store, "attend": _prepare_attend, "branch": _prepare_branch,
         "compact": _prepare_compact}[case["kind"]](case, g)
    s["kind"] = case["kind"]
    return s


# ----------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------
def _round(y, dtype):
    """y, already scaled, in a cache's 8-bit type (both roundings go to the nearest, ties to even)."""
    if dtype == torch.int8:
        return y.round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8)
    return y.clamp(-E4M3_MAX, E4M3_MAX).to(dtype)


def _row_places(row_start, kv_len, n_rows):
    """Sequence and position of every new row."""
    r = torch.arange(n_rows, device=kv_len.device)
    if row_start is None:
        return r, kv_len.long()
    s = torch.searchsorted(row_start[1:].long(), r, right=True)
    return s, kv_len.long()[s] + r - row_start.long()[s]


def _plain_store_one(x, codes, scales, layer, table, kv_len, row_start):
    P, T = codes.shape[3], codes.shape[3] // scales.shape[3]
    per = P // T
    qmax = INT8_MAX if codes.dtype == torch.int8 else E4M3_MAX
    seq, pos = _row_places(row_start, kv_len, x.shape[0])
    page, at = table[seq, pos // P].long(), pos % P
    block = page * per + at // T                                   # a number for every block of the layer
    H = x.shape[1]
    x = x.float()
    amax = torch.zeros(codes.shape[0] * per, H, device=x.device)
    amax.index_reduce_(0, block, x.abs().amax(2), "amax")
    old = scales[:, layer].transpose(1, 2).reshape(-1, H)          # [pages * per, H]
    new = (amax / qmax).clamp(min=SCALE_MIN)
    begun = torch.zeros(amax.shape[0], 1, dtype=torch.bool, device=x.device)
    begun[block] = (pos - at % T < kv_len.long()[seq])[:, None]    # the block has earlier rows
    new = torch.where(begun, torch.maximum(new, old), new)
    inv = 1.0 / new
    # the earlier rows of the blocks that were begun: they follow a scale that grew
    raw = torch.uint8 if codes.dtype != torch.int8 else torch.int8
    n = torch.diff(row_start.long()) if row_start is not None else torch.ones_like(kv_len, dtype=torch.long)
    c = kv_len.long()
    first = c // T * T
    open_ = (n > 0) & (c > first)
    op = table[torch.arange(c.numel(), device=c.device), (first // P).clamp(max=table.shape[1] - 1)].long()
    op, n_old, first = op[open_], (c - first)[open_], first[open_] % P
    i = torch.arange(T, device=c.device)
    at_old = first[:, None] + i                                    # [open, T]
    b = op * per + first // T
    rows = codes.view(raw)[op[:, None], layer, :, at_old]          # [open, T, H, D]
    moved = _round(rows.view(codes.dtype).float() * (old[b] * inv[b])[:, None, :, None], codes.dtype)
    stays = (i >= n_old[:, None])[:, :, None] | (new[b] == old[b])[:, None, :]
    codes.view(raw)[op[:, None], layer, :, at_old] = torch.where(stays[..., None], rows, moved.view(raw))
    codes.view(raw)[page, layer, :, at] = _round(x * inv[block][:, :, None], codes.dtype).view(raw)
    touched = torch.zeros(amax.shape[0], 1, dtype=torch.bool, device=x.device)
    touched[block] = True
    out = torch.where(touched, new, old)
    scales[:, layer] = out.view(codes.shape[0], per, H).transpose(1, 2)


def _plain_store(s):
    for x, name in ((s["new_k"], "k"), (s["new_v"], "v")):
        _plain_store_one(x, s[name], s[name + "_scale"], s["layer"], s["page_table"], s["kv_len"], s["row_start"])
    return {name: s[name] for name in ("k", "v", "k_scale", "v_scale")}


def _plain_rows(codes, scales, layer, table):
    """A layer's rows in fp32, [B][Hkv][positions][D]."""
    page = table.long().clamp(min=0)
    x = codes.view(torch.uint8)[:, layer][page].view(codes.dtype).float()  # [B][pages][Hkv][P][D]
    T = codes.shape[3] // scales.shape[3]
    x = x * scales[:, layer][page].repeat_interleave(T, dim=3)[..., None]
    B, n, H, P, D = x.shape
    return x.transpose(1, 2).reshape(B, H, n * P, D)


def _plain_attend(s):
    q, table, kv_len, n = s["q"], s["page_table"], s["kv_len"], s["max_rows"]
    R, Hq, D = q.shape
    k = _plain_rows(s["k"], s["k_scale"], s["layer"], table)
    v = _plain_rows(s["v"], s["v_scale"], s["layer"], table)
    B, H, L, _ = k.shape
    seq, pos = _row_places(s["row_start"], kv_len, R)
    i = pos - kv_len.long()[seq]
    x = torch.zeros(B, n, Hq, D, device=q.device)
    x[seq, i] = q.float()
    x = x.view(B, n, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * (Hq // H), D)
    score = (x @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    last = (kv_len.long()[:, None] + torch.arange(n, device=q.device)).repeat_interleave(Hq // H, 1)
    seen = torch.arange(L, device=q.device) <= last[:, None, :, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(3, keepdim=True)
    e = torch.exp(score - top)
    total = e.sum(3, keepdim=True)
    v = v.masked_fill(~seen.any(2)[:, :, :, None], 0.0)
    o = (e @ v) / total
    lse = (top + total.log())[..., 0]
    o = o.view(B, H, n, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    lse = lse.view(B, H, n, Hq // H).permute(0, 2, 1, 3).reshape(B, n, Hq)
    return {"out": o[seq, i].to(q.dtype), "lse": lse[seq, i]}


def _plain_branch(s):
    table, ref, P = s["table0"].clone(), s["ref0"].clone(), s["page"]
    src, dst = s["src"].long(), s["dst"].long()
    table[dst] = table[src]
    named = table[src]
    ref.index_add_(0, named.clamp(min=0).view(-1).long(), (named >= 0).int().view(-1))
    c, n = s["kv_len"].long()[:, None], s["n_new"].long()[:, None]
    j = torch.arange(table.shape[1], device=table.device)[None]
    wanted = (j * P < c + n) & (n > 0)
    missing = wanted & (table < 0)
    p = table.clamp(min=0).long()
    write = wanted & ((j + 1) * P > c) & (table >= 0) & (ref[p] > 1)
    entry = torch.arange(table.numel(), device=table.device).view_as(table)
    writers = torch.zeros_like(ref).index_add_(0, p.view(-1), write.int().view(-1))
    last = torch.full_like(ref, -1, dtype=torch.long)
    last.index_reduce_(0, p.view(-1), torch.where(write, entry, -1).view(-1), "amax")
    copied = write & ~((writers[p] == ref[p]) & (last[p] == entry))
    fresh = missing | copied
    free = (ref == 0).nonzero()[:, 0]
    page = free[fresh.view(-1).cumsum(0).sub(1).clamp(min=0)].view_as(table)
    moved = copied & (j * P < c)
    for pool in s["pools"]:
        pool[page[moved]] = pool[p[moved]]
    ref.index_add_(0, p.view(-1), -copied.int().view(-1))
    ref[page[fresh]] = 1
    table = torch.where(fresh, page.int(), table)
    return {"page_table": table, "ref_count": ref, "pools": s["pools"]}


def _plain_compact(s):
    table, ref = s["table0"].clone(), s["ref0"].clone()
    named = table[s["seqs"].long()]
    ref.index_add_(0, named.clamp(min=0).view(-1).long(), -(named >= 0).int().view(-1))
    table[s["seqs"].long()] = -1
    used = ref > 0
    low = torch.arange(ref.numel(), device=ref.device) < used.sum()
    src = (used & ~low).nonzero()[:, 0]
    dst = (~used & low).nonzero()[:, 0]
    to = torch.arange(ref.numel(), device=ref.device)
    to[src] = dst
    for pool in s["pools"]:
        pool[dst] = pool[src]
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
    ref[dst] = ref[src]
    ref[src] = 0
    return {"page_table": table, "ref_count": ref, "pools": s["pools"]}


def run(s):
    if own:
        return _own(s)
    return {"store": _plain_store, "attend": _plain_attend, "branch": _plain_branch,
            "compact": _plain_compact}[s["kind"]](s)


# ----------------------------------------------------------------------------
# The framework's calls
# ----------------------------------------------------------------------------
def _own(s):
    if s["kind"] == "store":
        s["cache"].store(s["layer"], s["new_k"], s["new_v"], s["page_table"], s["kv_len"], row_start=s["row_start"])
        return {name: s[name] for name in ("k", "v", "k_scale", "v_scale")}
    if s["kind"] == "attend":
        out, lse = s["cache"].attention(s["layer"], s["q"], s["page_table"], s["kv_len"], row_start=s["row_start"],
                                        max_rows=s["max_rows"], return_lse=True)
        return {"out": out, "lse": lse}
    pages = s["pages"]
    s["page_table"].copy_(s["table0"])  # every pass begins with the same pages in use
    s["ref_count"].copy_(s["ref0"])
    if s["kind"] == "branch":
        pages.fork(s["src"], s["dst"])
        pages.reserve(s["kv_len"], s["n_new"])
    else:
        pages.free(s["seqs"])
        pages.compact()
    return {"page_table": s["page_table"], "ref_count": s["ref_count"], "pools": s["pools"]}


# ----------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    c = case
    if c["kind"] == "store":
        rows = c["batch"] * (c["rows"] if c["rows"] == 1 else 0.75 * c["rows"])
        one = rows * c["kv_heads"] * c["dim"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": 2 * one * (size + 1) + 8 * rows * c["kv_heads"] / c["block"] + 8 * c["batch"],
                "flops": 6 * one}
    if c["kind"] == "attend":
        kv = c["kv"] * 17 / 32 if c["mixed"] else c["kv"]
        new = c["new"] / 2 if c["new"] > 1 else 1
        cached = c["batch"] * (kv + new) * c["kv_heads"]
        size = 4 if c["dtype"] == "f32" else 2
        rows = c["batch"] * new * c["q_heads"]
        return {"bytes": 2 * cached * (c["dim"] + 4 / c["block"]) + rows * (2 * size * c["dim"] + 4),
                "flops": 4 * rows * (kv + new) * c["dim"]}
    elements = c["layers"] * c["kv_heads"] * c["page"]
    page = 4 * elements * c["dim"] if not c["block"] else 2 * elements * (c["dim"] + 4 / c["block"])
    past = 0.75 * c["past"]
    per = max(1, past / c["page"])
    if c["kind"] == "branch":
        copies = c["groups"] * (c["ways"] - 1) * (1 - 1 / c["page"])  # unless the prompt ends with its page
        return {"bytes": 2 * copies * page + 8 * c["groups"] * c["ways"] * per, "flops": 0}
    gone = max(1, c["batch"] // 2) / c["batch"]
    moved = c["batch"] * per * gone * (1 - gone)
    return {"bytes": 2 * moved * page + 8 * c["batch"] * per, "flops": 0}


# ----------------------------------------------------------------------------
# The definitions in 64 bits, sequence by sequence
# ----------------------------------------------------------------------------
def _spans(s):
    past = s["kv_len"].tolist()
    start = s["row_start"].tolist() if s["row_start"] is not None else list(range(len(past) + 1))
    return [(b, past[b], start[b], start[b + 1]) for b in range(len(past))]


def _e4m3(y):
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_store(s):
    out = {}
    for x, name in ((s["new_k"].double(), "k"), (s["new_v"].double(), "v")):
        codes, scales, l = s[name], s[name + "_scale"].double(), s["layer"]
        P, T = codes.shape[3], codes.shape[3] // scales.shape[3]
        whole = codes.dtype == torch.int8
        val = codes.double()
        for b, c, r0, r1 in _spans(s):
            end = c + r1 - r0
            for p0 in range(c // T * T, end, T):
                page, at = int(s["page_table"][b, p0 // P]), p0 % P
                lo, hi = max(p0, c), min(p0 + T, end)
                new = x[r0 + lo - c:r0 + hi - c]                     # [rows][H][D]
                size = (new.abs().amax((0, 2)) / (INT8_MAX if whole else E4M3_MAX)).clamp(min=SCALE_MIN)
                if p0 < c:
                    old = scales[page, l, :, at // T].clone()
                    size = torch.maximum(size, old)
                    if not whole:
                        part = val[page, l, :, at:at + c - p0]
                        val[page, l, :, at:at + c - p0] = torch.where((size == old)[:, None, None], part,
                                                                      _e4m3(part * (old / size)[:, None, None]))
                scales[page, l, :, at // T] = size
                if not whole:
                    val[page, l, :, at + lo - p0:at + hi - p0] = _e4m3(new.transpose(0, 1) / size[:, None, None])
        out[name], out[name + "_scale"] = None if whole else val, scales
    return out


def _exact_attend(s):
    R, Hq, D = s["q"].shape
    out = torch.zeros(R, Hq, D, device="cuda", dtype=torch.float64)
    lse = torch.zeros(R, Hq, device="cuda", dtype=torch.float64)
    l = s["layer"]
    P = s["k"].shape[3]
    T = P // s["k_scale"].shape[3]
    H = s["k"].shape[2]
    for b, c, r0, r1 in _spans(s):
        n = c + r1 - r0
        page = s["page_table"][b, :-(-n // P)].long()
        for h in range(H):
            rows = []
            for name in ("k", "v"):
                x = s[name][page, l, h].double()
                w = s[name + "_scale"][page, l, h].double()
                rows.append((x.view(len(page), P // T, T, D) * w[:, :, None, None]).reshape(-1, D)[:n])
            for i in range(r1 - r0):
                q = s["q"][r0 + i, h * (Hq // H):(h + 1) * (Hq // H)].double()
                z = rows[0][:c + i + 1] @ q.T / math.sqrt(D)
                m = torch.logsumexp(z, 0)
                out[r0 + i, h * (Hq // H):(h + 1) * (Hq // H)] = torch.exp(z - m).T @ rows[1][:c + i + 1]
                lse[r0 + i, h * (Hq // H):(h + 1) * (Hq // H)] = m
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["kind"] == "attend":
        return _exact_attend(prepare(case, seed))
    if case["kind"] == "store":
        return _exact_store(prepare(case, seed))
    return None  # pages are numbers and copies: nothing is computed
