"""Float64 forms of the calls for the verification pass's rows, from their formulas
(include/spec_verify.h): rotary positions, the 8-bit cache, attention over it, and
logit adjustments. Test infrastructure; shares no code with the HIP path.
"""

import numpy as np

BLOCK = 32
E4M3_MAX = 448.0


def rotate(x, positions, freqs, interleaved=False, scale=1.0, inverse=False):
    """x [N, heads, D] turned at `positions` [N]."""
    y = np.array(x, dtype=np.float64)
    R = 2 * len(freqs)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freqs)[None]
    if inverse:
        a = -a
    c, s = np.cos(a)[:, None] * scale, np.sin(a)[:, None] * scale
    lo, hi = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    p, q = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo], y[..., hi] = p * c - q * s, q * c + p * s
    return y


def e4m3_table():
    """The values of the 256 codes: sign, 4 bits of exponent (bias 7), 3 of fraction;
    code 127 (and 255) is NaN, there are no infinities."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if e == 15 and m == 7 else x
        if c & 128:
            v[c] = -v[c]
    return v


TABLE = e4m3_table()


def encode(x):
    """Codes of values within 448, nearest, ties to the even code; NaN to NaN."""
    x = np.asarray(x, dtype=np.float64)
    grid = TABLE[:127]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    down, up = a - grid[hi - 1], grid[hi] - a
    code = np.where(down < up, hi - 1, np.where(down > up, hi, hi - 1 + (hi - 1) % 2))
    code = np.where(np.isnan(x), 127, code)
    return (code + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_scale(x):
    """The smallest 2^e, e >= -126, that brings the finite values within 448."""
    a = np.abs(x[np.isfinite(x)])
    amax = a.max() if a.size else 0.0
    if amax == 0:
        return 1.0
    e = -126
    while E4M3_MAX * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def place(s, d, values):
    """Byte of token s and dimension d in a brick."""
    if values:
        return 256 * (s // 8) + 16 * (d % 16) + 8 * (d // 16) + s % 8
    return 256 * (d // 8) + 16 * (4 * (s // 8) + s % 4) + 8 * (s // 4 % 2) + d % 8


def _places(D, values):
    s, d = np.meshgrid(np.arange(BLOCK), np.arange(D), indexing="ij")
    return d // 32, place(s, d % 32, values)


class Cache:
    """codes [pages, heads, blocks a page, bricks, 1024] uint8 and scales of keys or values."""

    def __init__(self, codes, scale, D, values):
        self.codes, self.scale, self.D, self.values = codes, scale, D, values
        self.brick, self.byte = _places(D, values)
        pb, pbyte = _places(codes.shape[3] * 32, values)
        self.pad = (pb[:, D:], pbyte[:, D:])

    def block(self, page, head, i):
        """Values [32, D] of a block."""
        c = self.codes[page, head, i]
        return TABLE[c[self.brick, self.byte]] * np.float64(self.scale[page, head, i])

    def at(self, table, pos):
        per = self.codes.shape[2]
        return int(table[pos // (per * BLOCK)]), pos // BLOCK % per

    def write(self, table, first, x):
        """Rows x [n, heads, D] at positions first ..; table: the request's pages."""
        for t0 in range(first // BLOCK * BLOCK, first + len(x), BLOCK):
            page, i = self.at(table, t0)
            if not 0 <= page < len(self.codes):
                continue
            n = min(BLOCK, first + len(x) - t0)       # rows that the block holds afterwards
            for h in range(self.codes.shape[1]):
                y = self.block(page, h, i)
                a = max(t0, first)
                y[a - t0: n] = x[a - first: t0 + n - first, h]
                y = y[:n]
                scale = block_scale(y)
                z = np.where(np.isfinite(y), y / scale, np.nan)
                if scale == 2.0 ** 120:          # 256 * 2^120 is beyond float32
                    z = np.clip(z, -240.0, 240.0)
                self.codes[page, h, i][self.brick[:n], self.byte[:n]] = encode(z)
                self.codes[page, h, i][self.pad[0][:n], self.pad[1][:n]] = 0
                self.scale[page, h, i] = scale

    def read(self, table, first, n):
        """Values [n, heads, D]; NaN in unknown pages."""
        out = np.full((n, self.codes.shape[1], self.D), np.nan)
        for t0 in range(first // BLOCK * BLOCK, first + n, BLOCK):
            page, i = self.at(table, t0)
            if 0 <= page < len(self.codes):
                a, b = max(t0, first), min(t0 + BLOCK, first + n)
                for h in range(self.codes.shape[1]):
                    out[a - first: b - first, h] = self.block(page, h, i)[a - t0: b - t0]
        return out


def attention(q, k, v, first, scale, window=0):
    """q [N, q_heads, D] over k, v [tokens, heads, D], row j at position first + j.
    Returns out, lse, and for tolerances sum p |v|, the largest sum |q k| scale, and
    the largest p times sum |v|."""
    N, qh, D = q.shape
    group = qh // k.shape[1]
    out, lse, size = np.zeros_like(q), np.zeros((N, qh)), np.zeros_like(q)
    reach, most = np.zeros((N, qh)), np.zeros_like(q)
    for j in range(N):
        p = first + j
        low = max(0, p - window + 1) if window else 0
        for h in range(qh):
            kk, vv = k[low: p + 1, h // group], v[low: p + 1, h // group]
            s = kk @ q[j, h] * scale
            m = s.max()
            w = np.exp(s - m)
            lse[j, h] = m + np.log(w.sum())
            w /= w.sum()
            out[j, h], size[j, h] = w @ vv, w @ np.abs(vv)
            reach[j, h] = (np.abs(kk) @ np.abs(q[j, h])).max() * abs(scale)
            most[j, h] = w.max() * np.abs(vv).sum(0)
    return out, lse, size, reach, most


def adjust(z, j, tokens=(), history=(), prompt=(), repetition=1.0, frequency=0.0, presence=0.0,
           bias=(), allowed=None):
    """One row z [V]; bias: (id, value) pairs; allowed: truth values [V] or None."""
    V = len(z)
    out = np.array(z, dtype=np.float64)
    count, seen = {}, set()
    for v in list(history) + list(tokens[:j]):
        if 0 <= v < V:
            count[int(v)] = count.get(int(v), 0) + 1
    seen = set(count) | {int(v) for v in prompt if 0 <= v < V}
    for v in seen:
        out[v] = out[v] / repetition if out[v] > 0 else out[v] * repetition
    for v, c in count.items():
        out[v] -= frequency * c + presence
    last = {}
    for v, x in bias:
        if 0 <= v < V:
            last[int(v)] = x
    for v, x in last.items():
        out[v] += x
    if allowed is not None:
        out[~np.asarray(allowed, dtype=bool)] = -np.inf
    return out
