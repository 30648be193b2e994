"""Frequencies on the host: defaults of each kind, refusals of what is not finite,
and the ramp's rounded ends."""
import math

import numpy as np
import pytest

import tree_speculative_decoding_eagle_gb300 as eg


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tree_speculative_decoding_eagle_gb300 import build
    build.build()


def freqs(**kw):
    f, factor = eg.rope_freqs(kw.pop("rot_dim", 64), device="cpu", **kw)
    return f.numpy(), factor


def test_the_upper_end_where_it_is_not_given():
    for kind, high in (("bands", 4.0), ("yarn", 32.0)):
        args = dict(theta=500000.0, kind=kind, stretch=8.0, orig_len=8192)
        np.testing.assert_array_equal(freqs(**args)[0], freqs(high=high, **args)[0])
    # frequencies that turn more often than that over the trained context stay as they are
    plain = freqs(theta=500000.0)[0]
    turns = 8192 * plain / (2 * math.pi)
    got = freqs(theta=500000.0, kind="bands", stretch=8.0, orig_len=8192)[0]
    np.testing.assert_array_equal(got[turns >= 4], plain[turns >= 4])
    np.testing.assert_allclose(got[turns <= 1], plain[turns <= 1] / 8, rtol=1e-15)
    between = (turns > 1) & (turns < 4)
    assert between.any() and (got[between] < plain[between]).all() and (got[between] > plain[between] / 8).all()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_what_is_not_finite_is_refused(bad):
    for kw in (dict(theta=bad), dict(kind="linear", stretch=bad), dict(kind="bands", high=bad), dict(kind="yarn", high=bad),
               dict(kind="yarn", low=bad), dict(kind="bands", low=bad)):
        with pytest.raises(eg.EagleError):
            freqs(**kw)


def test_the_yarn_ramp_ends_at_whole_pairs():
    theta, orig, low, high, rot = 150000.0, 4096, 1.0, 32.0, 64
    at = lambda r: rot * math.log(orig / (2 * math.pi * r)) / (2 * math.log(theta))
    lo, hi = math.floor(at(high)), math.ceil(at(low))
    got, _ = freqs(rot_dim=rot, theta=theta, kind="yarn", stretch=32.0, orig_len=orig, low=low, high=high)
    plain = freqs(rot_dim=rot, theta=theta)[0]
    np.testing.assert_array_equal(got[:lo + 1], plain[:lo + 1])
    np.testing.assert_allclose(got[hi:], plain[hi:] / 32, rtol=1e-15)
    j = np.arange(lo, hi + 1)
    w = (j - lo) / (hi - lo)
    np.testing.assert_allclose(got[lo:hi + 1], plain[lo:hi + 1] * (1 - w) + plain[lo:hi + 1] / 32 * w, rtol=1e-13)
