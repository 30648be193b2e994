"""Pins of the oracle of the page selection, on the CPU."""
import itertools

import numpy as np

from oracle import kv8, select


def test_bounds_hold_every_row_and_are_e4m3_numbers():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (40, 7, 16)).astype(np.uint8)
    for page in kv8.decode(codes):
        lo, hi = select.bounds(page)
        good = ~np.isnan(page)
        assert (np.where(good, page, lo) >= lo).all() and (np.where(good, page, hi) <= hi).all()
        assert (kv8.decode(kv8.encode(lo)) == lo).all() and (kv8.decode(kv8.encode(hi)) == hi).all()
        assert (2 * lo == np.rint(2 * lo)).all() and (2 * hi == np.rint(2 * hi)).all()
    # every e4m3 number alone, and halves stay as they are
    x = kv8.TABLE[~np.isnan(kv8.TABLE)][None]
    lo, hi = select.bounds(x)
    assert (hi - x < 0.5).all() and (x - lo < 0.5).all() and ((lo == hi) == (2 * x[0] == np.rint(2 * x[0]))).all()


def test_score_is_the_greatest_product_in_the_box():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((3, 4))
    lo = np.floor(rng.standard_normal((5, 4)) * 20) / 2
    hi = lo + np.floor(rng.random((5, 4)) * 10) / 2
    scale = 2.0 ** rng.integers(-3, 4, 5)
    got = select.scores(q, lo, hi, scale)
    for p in range(5):
        corners = [np.where(c, hi[p], lo[p]) for c in itertools.product([0, 1], repeat=4)]
        rows = [select.whole(r) for r in q]
        want = max(float(w @ c) * 2.0 ** e for w, e in rows for c in corners) * scale[p]
        assert got[p] == want
        # the whole numbers are the row to within half a unit
        for r, (w, e) in zip(q, rows):
            assert np.abs(w).max() >= 64 and np.abs(w).max() <= 128 and np.abs(w * 2.0 ** e - r).max() <= 2.0 ** (e - 1)


def test_choice():
    s = np.array([1.0, 5.0, 3.0, 5.0, 2.0, 0.0])
    assert select.choose(s, 2, 0, 0) == [1, 3]
    assert select.choose(s, 1, 0, 0) == [1]                     # ties to the lower page
    assert select.choose(s, 3, 1, 1) == [0, 1, 5]
    assert select.choose(s, 9, 1, 1) == [0, 1, 2, 3, 4, 5]
    assert select.choose(s[:1], 2, 1, 1) == [0] and select.choose(s[:0], 2, 1, 1) == []
    assert select.choose(np.zeros(9), 4, 0, 2) == [0, 1, 7, 8]
