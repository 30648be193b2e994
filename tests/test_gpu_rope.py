"""eagle_rope on the GPU against complex multiplication in fp64.

Tolerance, per element: half a step of the output type (relative 2^-8 in
bf16, 2^-24 in fp32) plus, of |x_a| + |x_b| times the factor: the phase's
float rounding (2^-25 half turns = 2^-25 pi), sincospif (2 ulp = 2^-23 each)
and the rotation's three roundings (2^-24 each): below 2^-21 together."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import rope as orope

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(got, x, pos, freqs, factor, interleaved):
    """got, x [..., heads, dh] (numpy fp64), pos [...]."""
    want = orope.rotate(x, pos, freqs, factor, interleaved)
    half = len(freqs)
    size = np.abs(x[..., :2 * half])
    pair = size[..., 0::2] + size[..., 1::2] if interleaved else size[..., :half] + size[..., half:]
    both = np.zeros_like(x)
    both[..., :2 * half] = np.repeat(pair, 2, -1) if interleaved else np.concatenate([pair, pair], -1)
    return np.abs(got - want), both * abs(factor) * 2.0 ** -21, want


def run(B, n, Hq, Hkv, dh, rot, dtype, interleaved=False, kind="plain", far=1000, fused=True, v=True, tree=True, shift=-1):
    g = torch.Generator().manual_seed(B * 1000 + n + rot)
    qkv = torch.randn((B, n, (Hq + 2 * Hkv) * dh), generator=g).to(dtype).cuda()
    q, k, vv = qkv.split([Hq * dh, Hkv * dh, Hkv * dh], 2)
    if not fused:
        q, k, vv = (x.contiguous() for x in (q, k, vv))
    q, k, vv = q.unflatten(2, (Hq, dh)), k.unflatten(2, (Hkv, dh)), vv.unflatten(2, (Hkv, dh))
    freqs, factor = eg.rope_freqs(rot, kind=kind, stretch=16.0, orig_len=4096, low=1.0, high=16.0)
    base = torch.randint(0, far + 1, (B,), generator=g).to(torch.int32)
    off = torch.randint(0, 7, (B, n), generator=g).to(torch.int32)
    got = eg.rope(q, k, vv if v else None, freqs, pos_base=base.cuda() if tree else None, pos_off=off.cuda() if tree else None,
                  shift=shift, factor=factor, interleaved=interleaved)
    torch.cuda.synchronize()
    pos = (base[:, None] + off).numpy().astype(np.float64) if tree else np.broadcast_to(np.arange(n, dtype=np.float64), (B, n))
    pos = pos + shift
    f64 = lambda t: t.double().cpu().numpy()
    for out, x, heads_first in ((got[0], q, False), (got[1], k, True)):
        o = f64(out).transpose(0, 2, 1, 3) if heads_first else f64(out)
        err, tol, want = check(o, f64(x), pos, freqs.cpu().numpy(), factor, interleaved)
        assert (err <= tol + HALF_STEP[dtype] * np.abs(want) * (1 + 2 ** -8)).all(), float((err - tol).max())
    if v:
        assert torch.equal(got[2], vv.transpose(1, 2))
    else:
        assert got[2] is None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dh,rot", [(64, 64), (128, 128), (128, 32), (64, 20), (128, 2), (64, 16), (80, 80), (16, 6), (512, 512)])
def test_heads_and_parts(dtype, interleaved, dh, rot):
    run(3, 5, 4, 2, dh, rot, dtype, interleaved)


@pytest.mark.parametrize("B,n,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 32, 32), (64, 1, 64, 8), (2, 61, 5, 1), (1, 1023, 3, 3), (7, 13, 10, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes(B, n, Hq, Hkv, dtype):
    run(B, n, Hq, Hkv, 128, 128, dtype)
    run(B, n, Hq, Hkv, 64, 32, dtype, interleaved=True, fused=False)


@pytest.mark.parametrize("kind", ["linear", "bands", "yarn"])
def test_scaled_frequencies(kind):
    run(2, 9, 4, 2, 128, 64, torch.float32, kind=kind)


def test_far_positions_lose_nothing():
    run(4, 9, 2, 1, 128, 128, torch.float32, far=2 ** 31 - 10)
    run(4, 9, 2, 1, 128, 128, torch.float32, far=2 ** 24, interleaved=True, kind="yarn")


def test_prompt_positions_and_missing_values():
    run(2, 33, 4, 4, 64, 64, torch.bfloat16, tree=False, shift=0)
    run(2, 33, 4, 4, 64, 64, torch.bfloat16, tree=False, shift=-5, v=False)        # positions below zero
    run(1, 1, 4, 4, 64, 64, torch.bfloat16, tree=False, shift=2 ** 30)


def test_queries_in_place_and_rows_that_hold_nan():
    q = torch.randn((2, 7, 4, 64), device="cuda").to(torch.bfloat16)
    k = torch.randn((2, 7, 2, 64), device="cuda").to(torch.bfloat16)
    q[1, 3] = math.nan                                               # a padding row: it stays its own affair
    f, _ = eg.rope_freqs(64)
    want = eg.rope(q, k, None, f)[0]
    got = eg.rope(q, k, None, f, q_out=q)[0]
    assert got.data_ptr() == q.data_ptr()
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
    assert torch.isnan(got[1, 3]).all() and torch.isfinite(got[0]).all() and torch.isfinite(got[1, 4:]).all()


def test_refused_by_the_binding():
    q = torch.zeros((2, 3, 4, 64), device="cuda", dtype=torch.bfloat16)
    k = torch.zeros((2, 3, 2, 64), device="cuda", dtype=torch.bfloat16)
    f, _ = eg.rope_freqs(64)
    for bad in (dict(k=k.float()), dict(k=k[:, :2]), dict(q=q.transpose(1, 2)), dict(inv_freq=f.float()), dict(v=k[:, :, :1]),
                dict(pos_base=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(pos_off=torch.zeros((2, 3), device="cuda")),
                dict(q=q[..., ::2]), dict(inv_freq=eg.rope_freqs(80)[0]), dict(k_tree=k)):
        with pytest.raises(eg.EagleError):
            eg.rope(**{"q": q, "k": k, "v": k, "inv_freq": f, **bad})


def test_on_another_stream_and_captured():
    q = torch.randn((2, 5, 4, 128), device="cuda")
    k = torch.randn((2, 5, 2, 128), device="cuda")
    f, _ = eg.rope_freqs(128)
    base = torch.tensor([3, 9], dtype=torch.int32, device="cuda")
    want = eg.rope(q, k, k, f, pos_base=base)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = eg.rope(q, k, k, f, pos_base=base)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = eg.rope(q, k, k, f, pos_base=base)
    base += 11
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(eg.rope(q, k, k, f, pos_base=base), out))
