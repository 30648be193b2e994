"""Oracle: rotary positions (test infrastructure only), in fp64 as complex
multiplication: pair j of a head at position p times exp(i p f_j)."""
import math

import numpy as np


def rotate(x, pos, inv_freq, factor=1.0, interleaved=False):
    """x fp64 [..., heads, dh], pos [...] -> the rotated heads."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    turn = factor * np.exp(1j * np.asarray(pos, dtype=np.float64)[..., None] * inv_freq)
    z = (x[..., a] + 1j * x[..., b]) * turn[..., None, :]
    x[..., a], x[..., b] = z.real, z.imag
    return x


def freqs(rot_dim, theta=10000.0, kind="plain", stretch=1.0, orig_len=4096, low=1.0, high=32.0):
    """(inv_freq, factor); kinds as rope_freqs describes them."""
    out = []
    for j in range(rot_dim // 2):
        f = theta ** (-2.0 * j / rot_dim)
        if kind == "linear":
            f = f / stretch
        elif kind == "bands":
            turns = orig_len * f / (2 * math.pi)
            w = min(max((turns - low) / (high - low), 0.0), 1.0)
            f = (1 - w) * f / stretch + w * f
        elif kind == "yarn":
            at = lambda r: rot_dim * math.log(orig_len / (2 * math.pi * r)) / (2 * math.log(theta))
            lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot_dim - 1)
            ramp = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f / stretch * ramp + f * (1 - ramp)
        out.append(f)
    return np.array(out), (0.1 * math.log(stretch) + 1.0 if kind == "yarn" else 1.0)
