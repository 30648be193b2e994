"""Oracle: pages of a paged 8-bit cache that a query selects (test
infrastructure only), in fp64.

A page's bounds are the least and the greatest e4m3 number of each column over
its rows, rounded outwards to multiples of 1/2.  A query row counts as whole
numbers q' = rint(q / 2^e), 64 <= max |q'| <= 128; its product with a page's keys is at
most the sum of q'_c hi_c over the positive q'_c and of q'_c lo_c over the negative
ones, times 2^e and the page's scale.
"""
import math

import numpy as np


def bounds(x):
    """lo, hi [dh] of rows x [rows, dh] of e4m3 numbers (NaN: as wide as can be)."""
    bad = np.isnan(x).any(0)
    lo = np.floor(2 * np.where(np.isnan(x), 0.0, x).min(0)) / 2
    hi = np.ceil(2 * np.where(np.isnan(x), 0.0, x).max(0)) / 2
    return np.where(bad, -448.0, lo), np.where(bad, 448.0, hi)


def whole(q):
    """A row q [dh] as (whole numbers, e)."""
    q = np.where(np.isfinite(q), q, 0.0)
    size = np.abs(q).max()
    e = 0
    if size > 0:
        e = min(max(math.frexp(size)[1] - 7, -32), 32)
    return np.clip(np.rint(q * 2.0 ** -e), -128, 128), e


def scores(q, lo, hi, scale):
    """q [G, dh] of one node and KV head, bounds [pages, dh] with scales [pages]
    -> the pages' scores."""
    best = np.full(len(scale), -np.inf)
    for row in q:
        w, e = whole(row)
        u = np.where(w > 0, w * hi, w * lo).sum(1)
        best = np.maximum(best, u * 2.0 ** e * scale)
    return best


def choose(score, top, first, last):
    """Selected pages, ascending."""
    n = len(score)
    order = sorted(range(n), key=lambda p: (not (p < first or p >= n - last), -score[p], p))
    return sorted(order[:top])
