"""Plain restatements of the 8-bit cache and page calls, for the tests."""
import math

import numpy as np

SCALE_MIN = np.float32(2.0 ** -126)


def torch():
    import torch as t
    return t


def fp8_values():
    """The 256 e4m3 codes as float32 (0x7f, 0xff: NaN)."""
    out = np.empty(256, np.float32)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = -x if s else x
    return out


FP8 = fp8_values()


def decode(codes, fmt):
    """uint8 codes -> float32 values."""
    return codes.view(np.int8).astype(np.float32) if fmt == "int8" else FP8[codes]


def encode(y, fmt):
    """float32 values (already divided by the scale) -> uint8 codes, to nearest even, clamped."""
    if fmt == "int8":
        return np.clip(np.rint(y), -127, 127).astype(np.int8).view(np.uint8)
    y = np.clip(y.astype(np.float64), -448, 448)
    with np.errstate(divide="ignore"):
        e = np.clip(np.floor(np.log2(np.abs(y))), -6, 8)
    step = 2.0 ** (e - 3)
    q = np.rint(y / step) * step  # may be 2 ** (e + 1): still a code's value
    mag = np.abs(q)
    with np.errstate(divide="ignore"):
        e = np.clip(np.floor(np.log2(mag)), -6, 8)
    m = np.rint(mag / 2.0 ** (e - 3)).astype(np.int64)  # 8 .. 15, below 8: subnormal
    code = np.where(m < 8, m, ((e + 7).astype(np.int64) << 3) | (m & 7))
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


class Cache:
    """Host copy of a cache: uint8 codes and float32 scales of K and V."""

    def __init__(self, n_pages, n_layers, n_kv_heads, head_dim, page, block, fmt, seed=0):
        rng = np.random.default_rng(seed)
        self.fmt, self.page, self.block = fmt, page, block
        shape = (n_pages, n_layers, n_kv_heads, page, head_dim)
        self.codes, self.scales = [], []
        for _ in range(2):
            if fmt == "int8":
                c = rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8)
            else:
                c = encode(rng.standard_normal(shape).astype(np.float32) * 110, fmt)
            self.codes.append(c)
            self.scales.append(((0.7 + 0.6 * rng.random(shape[:3] + (page // block,))) / 90)
                               .astype(np.float32))

    def device(self):
        import persistent_runtime_b200 as prb
        t = torch()
        kind = t.int8 if self.fmt == "int8" else t.float8_e4m3fn
        dev = [t.from_numpy(c.copy()).cuda().view(kind) for c in self.codes]
        dev += [t.from_numpy(s.copy()).cuda() for s in self.scales]
        return prb.KV8Cache(*dev)

    def rows(self, which, layer, pages, n):
        """The first n positions of a sequence in float64 [n][heads][dim]."""
        c = decode(self.codes[which][pages, layer], self.fmt).astype(np.float64)
        s = np.repeat(self.scales[which][pages, layer].astype(np.float64), self.block, axis=2)
        x = c * s[..., None]                       # [pages][heads][page][dim]
        return x.transpose(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])[:n]

    def store(self, layer, x, table, kv_len, start):
        """mk_kv8_store in float32, block by block; x = (k, v) float32 [rows][heads][dim]."""
        inv_qmax = np.float32(1) / np.float32(127 if self.fmt == "int8" else 448)
        for which in range(2):
            codes, scales = self.codes[which], self.scales[which]
            for s, c in enumerate(kv_len):
                r0, n = start[s], start[s + 1] - start[s]
                end = c + n
                for p0 in range(c // self.block * self.block, end, self.block):
                    if n == 0:
                        break
                    page, at = table[s][p0 // self.page], p0 % self.page
                    lo, hi = max(p0, c), min(p0 + self.block, end)
                    for h in range(x[which].shape[1]):
                        new = x[which][r0 + lo - c:r0 + hi - c, h].astype(np.float32)
                        old = scales[page, layer, h, at // self.block]
                        bad = not np.isfinite(new).all() or (p0 < c and np.isnan(old))
                        if bad:
                            scales[page, layer, h, at // self.block] = np.nan
                            codes[page, layer, h, at + lo - p0:at + hi - p0] = 0
                            continue
                        size = max(np.float32(np.abs(new).max() * inv_qmax), SCALE_MIN)
                        if p0 < c:
                            size = max(size, old)
                        inv = np.float32(1) / size
                        if p0 < c and size != old:
                            was = codes[page, layer, h, at:at + c - p0]
                            ratio = np.float32(old * inv)
                            codes[page, layer, h, at:at + c - p0] = encode(
                                decode(was, self.fmt) * ratio, self.fmt)
                        codes[page, layer, h, at + lo - p0:at + hi - p0] = encode(new * inv, self.fmt)
                        scales[page, layer, h, at // self.block] = size

    def attention(self, layer, q, table, kv_len, start, scale, dtype):
        """Output and log-sum-exp in float64, and how far a kernel may be off (see below)."""
        R, Hq, D = q.shape
        H = self.codes[0].shape[2]
        out, lse = np.zeros((R, Hq, D)), np.zeros((R, Hq))
        tol, tol_lse = np.zeros((R, Hq, D)), np.zeros((R, Hq))
        # probabilities: e4m3, one rounding to fp16 (half a step, 2^-11; fp32 rows: two terms,
        # 2^-21); int8, 16-bit integers (fp32 rows: 24-bit, the largest 2^23) relative to the
        # largest of the 32 positions of their chunk: off by half a unit of that, 2^-16.9 (2^-24)
        wide = dtype == "float32"
        t_p = 0.0 if self.fmt == "int8" else 2.0 ** -21 if wide else 2.0 ** -11
        t_c = 0.0 if self.fmt != "int8" else 2.0 ** -24 if wide else 2.0 ** -16.9
        # query elements: e4m3, fp16 terms, below 2^-25 of the row's largest rounded away; int8, an
        # integer of at most 127 2^14 for a row whose largest has at least half of that: half a
        # unit is at most 2^-21 of the largest
        t_q = 2.0 ** -21 if self.fmt == "int8" else 2.0 ** -25
        t_o = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}[dtype]
        for s, c in enumerate(kv_len):
            n = c + start[s + 1] - start[s]
            if start[s + 1] == start[s]:
                continue
            pages = table[s][:-(-n // self.page)]
            k, v = self.rows(0, layer, pages, n), self.rows(1, layer, pages, n)
            for i in range(start[s + 1] - start[s]):
                L = c + i + 1
                for h in range(Hq):
                    g = h // (Hq // H)
                    x = q[start[s] + i, h].astype(np.float64)
                    z = k[:L, g] @ x * scale
                    m = z.max()
                    e = np.exp(z - m)
                    w = e / e.sum()
                    out[start[s] + i, h] = w @ v[:L, g]
                    lse[start[s] + i, h] = m + math.log(e.sum())
                    # scores: the tensor cores add D / 16 <= 8 partial products and keep at
                    # least 22 bits of the largest magnitude each time (int8: exact, then one
                    # rounding to fp32): at most 2^-18 of sum |q k|, in the numerator and in the
                    # denominator (2^-17), and so do the elements' own errors.  The sums over
                    # positions: a warp adds at most L / 128 + 8 products of 16 positions, each
                    # off by 2^-22, and the exponential by 2^-21.
                    size = ((np.abs(k[:L, g]) @ np.abs(x)) * 2.0 ** -17 + 2 * t_q * np.abs(x).max() * np.abs(k[:L, g]).sum(1)).max() * abs(scale)
                    rel = t_p + size + 2.0 ** -22 * (L / 64 + 32)
                    at = np.arange(0, L, 32)
                    held = t_c * np.maximum.reduceat(w, at) @ np.add.reduceat(np.abs(v[:L, g]), at)
                    tol[start[s] + i, h] = t_o * np.abs(out[start[s] + i, h]) + 1.01 * (rel * (w @ np.abs(v[:L, g])) + held) + 1e-30
                    if dtype == "float16":  # smallest steps of the type
                        tol[start[s] + i, h] += 2.0 ** -25
                    tol_lse[start[s] + i, h] = rel + 2.0 ** -23 * (abs(lse[start[s] + i, h]) + 40)
        return out, lse, tol, tol_lse


def make_table(lens, page, spare=3, seed=0, extra=1):
    """Tables with pages in random order; unused entries name no page."""
    rng = np.random.default_rng(seed)
    used = [-(-int(n) // page) for n in lens]
    n_pages = sum(used) + spare
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), max(max(used), 1) + extra), -1, np.int32)
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    return table, n_pages


def dev(a, dtype=None):
    t = torch()
    x = t.from_numpy(np.ascontiguousarray(a)).cuda()
    return x if dtype is None else x.to(dtype)
