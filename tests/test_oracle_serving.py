"""Pins of the serving loop's oracles (pages, rotary positions, the 8-bit
cache) and of the host-side frequencies, on the CPU."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8, pages, rope


def test_page_map_by_hand():
    # 4-token pages would be below the limit; the oracle itself takes any
    table = [[5, -1, -1], [-1, -1, -1], [7, 2, -1]]
    err, t, c, fc, slots, starts = pages.page_map([3, 0, 8], [3, 0, 1], table, [1, 0, 2], [9, 4, 1, 0], 3, 4, 10, T=6)
    assert err is None and fc == 1
    assert t == [[5, 1, -1], [-1, -1, -1], [7, 2, 4]] and c == [2, 0, 3]      # the top of the stack goes first
    assert slots == [23, 4, 5, 16, -1, -1] and starts == [0, 3, 3, 4]


def test_release_undoes_a_map():
    rng = np.random.default_rng(0)
    for _ in range(50):
        B, P, mp = 5, 16, 6
        N = B * mp
        order = rng.permutation(N).tolist()
        kv = rng.integers(0, 60, B).tolist()
        new = rng.integers(0, 36, B).tolist()
        count = [-(-k // P) for k in kv]
        table = [[order.pop() if p < c else -1 for p in range(mp)] for c in count]
        free, fc = order + [-5] * (N - len(order)), len(order)
        err, t2, c2, fc2, slots, starts = pages.page_map(kv, new, table, count, free, fc, P, N)
        assert err is None and len(slots) == sum(new) == starts[-1]
        t3, c3, f3, fc3 = pages.page_release(kv, t2, c2, free, fc2, P)
        assert (t3, c3, f3, fc3) == (table, count, free, fc)


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(1)
    f, _ = rope.freqs(16)
    q, k = rng.standard_normal((2, 1, 1, 24))
    at = lambda x, p, il: rope.rotate(x, np.array([p]), f, interleaved=il)
    for il in (False, True):
        a = (at(q, 7, il) * at(k, 3, il)).sum()
        b = (at(q, 107, il) * at(k, 103, il)).sum()
        assert abs(a - b) < 1e-12                                    # only the distance counts
        assert (at(q, 5, il)[..., 16:] == q[..., 16:]).all()         # the rest of the head is copied
        np.testing.assert_allclose(at(q, 5, il)[0, 0, :16:1].dot(at(q, 5, il)[0, 0, :16]), q[0, 0, :16].dot(q[0, 0, :16]))
    one = rope.rotate(np.array([[[1.0, 0.0]]]), np.array([1]), np.array([math.pi / 2]))
    np.testing.assert_allclose(one, [[[0.0, 1.0]]], atol=1e-15)


@pytest.mark.parametrize("kind", ["plain", "linear", "bands", "yarn"])
@pytest.mark.parametrize("rot", [2, 20, 64, 128])
def test_frequencies(kind, rot):
    args = dict(theta=500000.0, kind=kind, stretch=8.0, orig_len=8192, low=1.0, high=4.0)
    got, factor = eg.rope_freqs(rot, device="cpu", **args)
    want, wf = rope.freqs(rot, **args)
    np.testing.assert_allclose(got.numpy(), want, rtol=1e-13)
    assert abs(factor - wf) <= 2 ** -24 * wf
    plain = rope.freqs(rot, theta=500000.0)[0]
    assert (got.numpy() <= plain * (1 + 1e-13)).all() and (got.numpy() >= plain / 8 * (1 - 1e-13)).all()


def test_frequencies_refused():
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(theta=1.0), dict(stretch=0.5), dict(kind="bands", low=4.0, high=4.0),
                dict(kind="yarn", orig_len=0), dict(kind="spiral")):
        with pytest.raises(eg.EagleError):
            eg.rope_freqs(**{"rot_dim": 64, "device": "cpu", **bad})


def test_e4m3_against_torch():
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(kv8.decode(codes), t)              # every number, NaN among them
    fin = codes[(codes & 127) != 127]
    np.testing.assert_array_equal(kv8.encode(kv8.decode(fin)), fin)
    rng = np.random.default_rng(2)
    y = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 8, 4000), (kv8.TABLE[:126] + kv8.TABLE[1:127]) / 2])
    y = np.clip(y, -448, 448).astype(np.float32)                     # the midpoints are ties
    np.testing.assert_array_equal(kv8.encode(y.astype(np.float64)), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_block_exponent_is_the_least_that_fits():
    for a in (1.0, 448.0, 448.0000001, 449.0, 0.875, 0.8750001, 3e-5, 1e10):
        e = kv8.block_exponent(a)
        assert a <= 448 * 2.0 ** e and a > 448 * 2.0 ** (e - 1)
    assert kv8.block_exponent(0.0) == kv8.E_MIN and kv8.block_exponent(1e30) == kv8.E_MAX


def test_growing_scale_only_touches_subnormals():
    rng = np.random.default_rng(3)
    codes, scale = np.zeros((1, 1, 16, 32), np.uint8), np.ones((1, 1))
    x = rng.standard_normal((2, 1, 32))
    x[1] *= 16
    kv8.append(x[:1], [0], codes, scale)
    before, s0 = codes.copy(), scale.copy()
    kv8.append(x[1:], [1], codes, scale)
    assert scale[0, 0] > s0[0, 0]
    v0, v1 = kv8.decode(before[0, 0, 0]) * s0[0, 0], kv8.decode(codes[0, 0, 0]) * scale[0, 0]
    big = np.abs(v0) >= 2.0 ** -6 * scale[0, 0]
    assert big.any() and (v0[big] == v1[big]).all()
    assert np.abs(v0 - v1).max() <= 2.0 ** -10 * scale[0, 0]         # half a step of the subnormals
