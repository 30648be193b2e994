"""Oracle: the paged KV cache in 8 bits (test infrastructure only).

A cache value is an e4m3 number times a power-of-two scale of its page and
head.  e4m3 (no infinities): sign, 4 exponent bits with bias 7, 3 mantissa
bits; exponent 0 is subnormal, 0x7f and 0xff are NaN, the largest is 448.
"""
import math

import numpy as np

E_MIN, E_MAX = -64, 64


def _table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if (c & 127) == 127:
            v = math.nan
        t[c] = -v if c & 128 else v
    return t


TABLE = _table()


def decode(codes):
    return TABLE[np.asarray(codes, dtype=np.uint8)]


def encode(y):
    """Nearest e4m3 number, ties to the even code; saturating; NaN to 0x7f."""
    y = np.asarray(y, dtype=np.float64)
    pos = TABLE[:127]
    a = np.minimum(np.abs(np.where(np.isnan(y), 0.0, y)), 448.0)
    hi = np.minimum(np.searchsorted(pos, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(y), code | 128, code)
    return np.where(np.isnan(y), 127, code).astype(np.uint8)


def block_exponent(amax):
    """The least e in [E_MIN, E_MAX] with amax <= 448 * 2^e (E_MAX if none)."""
    for e in range(E_MIN, E_MAX + 1):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def append(rows, slots, codes, scale):
    """rows fp64 [T, Hkv, dh] to slots (negative: skipped), in place, in
    codes uint8 [num_pages, Hkv, P, dh] and scale [num_pages, Hkv].  The rows
    of one page are taken together."""
    P = codes.shape[2]
    by_page = {}
    for t, s in enumerate(slots):
        if s >= 0:
            by_page.setdefault(int(s) // P, []).append((int(s) % P, t))
    for page, items in by_page.items():
        first = min(r for r, _ in items)
        for g in range(codes.shape[1]):
            x = np.stack([rows[t, g] for _, t in items])
            fin = np.isfinite(x)
            e = block_exponent(np.abs(x[fin]).max() if fin.any() else 0.0)
            if first > 0:
                old = int(math.log2(scale[page, g]))
                if e > old:
                    codes[page, g, :first] = encode(decode(codes[page, g, :first]) * 2.0 ** (old - e))
                e = max(e, old)
            scale[page, g] = 2.0 ** e
            for (r, _), row, f in zip(items, x, fin):
                codes[page, g, r] = encode(np.where(f, np.where(f, row, 0.0) / 2.0 ** e, np.nan))
    return codes, scale


def gather(codes, scale, table, L):
    """Values fp64 [Hkv, L, dh] of the first L positions behind a block table row."""
    P = codes.shape[2]
    pages = np.asarray(table[:-(-L // P)], dtype=np.int64)
    v = decode(codes[pages]) * scale[pages][..., None, None]
    return v.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :L]
