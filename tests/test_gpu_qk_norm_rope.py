"""eagle_qk_norm_rope on the GPU against fp64.

Tolerance, per element, on the normed head y (before the rotation): a sum of dh
squares in float32 is off by at most dh 2^-24 of itself, its root by half of
that; division by dh and + eps 2^-24 each, halved; rsqrtf 2 ulp (2^-22); x r,
w + offset and their product 2^-24 each: below dh 2^-25 + 2^-21 of |y|.  The
rotation adds 2^-21 of |y_a| + |y_b| (test_gpu_rope.py).  Then half a step of
the output type."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import rope as orope

pytestmark = pytest.mark.gpu
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
f64 = lambda t: t.double().cpu().numpy()


def normed(x, w, eps, offset):
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * (1.0 if w is None else w + offset)


def check(got, x, w, pos, freqs, factor, interleaved, eps, offset, dtype):
    dh, half = x.shape[-1], len(freqs)
    y = normed(x, w, eps, offset)
    want = orope.rotate(y, pos, freqs, factor, interleaved)
    size = np.abs(y[..., :2 * half])
    pair = size[..., 0::2] + size[..., 1::2] if interleaved else size[..., :half] + size[..., half:]
    both = np.abs(y)
    both[..., :2 * half] = abs(factor) * (np.repeat(pair, 2, -1) if interleaved else np.concatenate([pair, pair], -1))
    tol = both * (2.0 ** -20 + dh * 2.0 ** -25) + HALF_STEP[dtype] * np.abs(want) * (1 + 2 ** -8) + 1e-38
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())


def run(B, n, Hq, Hkv, dh, rot, dtype, interleaved=False, kind="plain", far=1000, fused=True, v=True, tree=True, weights=(True, True),
        eps=1e-6, offset=0.0, size=1.0, in_place=False):
    g = torch.Generator().manual_seed(B * 1000 + n + rot)
    qkv = (torch.randn((B, n, Hq + 2 * Hkv, dh), generator=g) * torch.exp2(2 * torch.randn((Hq + 2 * Hkv, 1), generator=g)) * size)
    qkv = qkv.to(dtype).view(B, n, -1).cuda()
    q, k, vv = qkv.split([Hq * dh, Hkv * dh, Hkv * dh], 2)
    if not fused:
        q, k, vv = (x.contiguous() for x in (q, k, vv))
    q, k, vv = q.unflatten(2, (Hq, dh)), k.unflatten(2, (Hkv, dh)), vv.unflatten(2, (Hkv, dh))
    w = [(1 + 0.3 * torch.randn(dh, generator=g)).to(dtype).cuda() if there else None for there in weights]
    freqs, factor = eg.rope_freqs(rot, kind=kind, stretch=16.0, orig_len=4096, low=1.0, high=16.0)
    base = torch.randint(0, far + 1, (B,), generator=g).to(torch.int32)
    off = torch.randint(0, 7, (B, n), generator=g).to(torch.int32)
    x = [f64(q), f64(k)]
    got = eg.qk_norm_rope(q, k, vv if v else None, freqs, *w, eps=eps, weight_offset=offset, pos_base=base.cuda() if tree else None,
                          pos_off=off.cuda() if tree else None, shift=-1, factor=factor, interleaved=interleaved,
                          q_out=q if in_place else None)
    torch.cuda.synchronize()
    pos = (base[:, None] + off).numpy().astype(np.float64) if tree else np.broadcast_to(np.arange(n, dtype=np.float64), (B, n))
    for out, xs, ws, heads_first in ((got[0], x[0], w[0], False), (got[1], x[1], w[1], True)):
        o = f64(out).transpose(0, 2, 1, 3) if heads_first else f64(out)
        check(o, xs, None if ws is None else f64(ws), pos - 1, freqs.cpu().numpy(), factor, interleaved, eps, offset, dtype)
    if v:
        assert torch.equal(got[2], vv.transpose(1, 2))
    else:
        assert got[2] is None
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dh,rot", [(64, 64), (128, 128), (128, 32), (64, 20), (128, 2), (64, 16), (80, 80), (16, 6), (16, 16), (8, 8),
                                    (512, 512), (512, 16), (256, 256), (384, 130)])
def test_heads_and_parts(dtype, interleaved, dh, rot):
    run(3, 5, 4, 2, dh, rot, dtype, interleaved)


@pytest.mark.parametrize("B,n,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 32, 32), (64, 1, 64, 8), (2, 61, 5, 1), (1, 1023, 3, 3), (7, 13, 10, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes(B, n, Hq, Hkv, dtype):
    run(B, n, Hq, Hkv, 128, 128, dtype)
    run(B, n, Hq, Hkv, 64, 32, dtype, interleaved=True, fused=False)
    run(B, n, Hq, Hkv, 64, 20, dtype, v=False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weights", [(False, False), (True, False), (False, True)])
def test_weights_and_offset(weights, dtype):
    run(2, 9, 4, 2, 128, 64, dtype, weights=weights, offset=1.0)
    run(2, 9, 4, 2, 64, 10, dtype, weights=weights, offset=1.0)
    run(2, 9, 4, 2, 128, 128, dtype, offset=-0.5, kind="yarn", far=2 ** 24)


@pytest.mark.parametrize("rot", [128, 10])
@pytest.mark.parametrize("size,eps", [(1e-4, 1e-6), (1e-12, 1e-5), (1e12, 1e-6), (1e-4, 1e-30)])
def test_magnitudes(rot, size, eps):
    run(2, 5, 4, 2, 128, rot, torch.float32, size=size, eps=eps)
    run(2, 5, 4, 2, 128, rot, torch.bfloat16, size=size, eps=eps)


@pytest.mark.parametrize("dh,rot", [(128, 128), (128, 10), (512, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_without_v_and_positions(dh, rot, dtype):
    run(2, 5, 4, 2, dh, rot, dtype, fused=False, in_place=True)
    run(1, 9, 4, 2, dh, rot, dtype, v=False, tree=False)


def test_odd_heads_stay_alone():
    """A head of zeros gives zeros; an infinity or a NaN spoils its own head."""
    B, n, Hq, Hkv, dh = 2, 3, 4, 2, 64
    freqs, _ = eg.rope_freqs(dh)
    q = torch.randn((B, n, Hq, dh), device="cuda").bfloat16()
    k = torch.randn((B, n, Hkv, dh), device="cuda").bfloat16()
    want = eg.qk_norm_rope(q, k, None, freqs)
    q2, k2 = q.clone(), k.clone()
    q2[1, 2, 3] = 0
    q2[0, 1, 0, 5] = float("inf")
    k2[1, 0, 1, 7] = float("nan")
    got = eg.qk_norm_rope(q2, k2, None, freqs)
    assert not got[0][1, 2, 3].any() and got[0][0, 1, 0].isnan().any() and got[1][1, 1, 0].isnan().all()
    keep = torch.ones((B, n, Hq), dtype=torch.bool)
    keep[1, 2, 3] = keep[0, 1, 0] = False
    assert torch.equal(got[0][keep.cuda()], want[0][keep.cuda()])
    keep = torch.ones((B, Hkv, n), dtype=torch.bool)
    keep[1, 1, 0] = False
    assert torch.equal(got[1][keep.cuda()], want[1][keep.cuda()])


@pytest.mark.parametrize("rot", [64, 20])
def test_a_node_does_not_depend_on_the_others(rot):
    B, n, Hq, Hkv, dh = 3, 7, 5, 1, 64
    freqs, _ = eg.rope_freqs(rot)
    q = torch.randn((B, n, Hq, dh), device="cuda").bfloat16()
    k, v = (torch.randn((B, n, Hkv, dh), device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(dh, device="cuda").bfloat16()
    pos = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)
    whole = eg.qk_norm_rope(q, k, v, freqs, w, w, pos_off=pos)
    for b, i in ((0, 0), (1, 3), (2, 6)):
        part = eg.qk_norm_rope(q[b:b + 1, i:i + 1], k[b:b + 1, i:i + 1], v[b:b + 1, i:i + 1], freqs, w, w,
                               pos_off=pos[b:b + 1, i:i + 1].contiguous())
        assert torch.equal(part[0][0, 0], whole[0][b, i]) and torch.equal(part[1][0, :, 0], whole[1][b, :, i])


def test_stream_and_capture():
    B, n, Hq, Hkv, dh = 2, 9, 8, 2, 128
    freqs, _ = eg.rope_freqs(dh)
    q, k = torch.randn((B, n, Hq, dh), device="cuda").bfloat16(), torch.randn((B, n, Hkv, dh), device="cuda").bfloat16()
    want = eg.qk_norm_rope(q, k, k, freqs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = eg.qk_norm_rope(q, k, k, freqs, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.qk_norm_rope(q, k, k, freqs, q_out=out[0], k_tree=out[1], v_tree=out[2])
    q.mul_(-2)
    graph.replay()
    want = eg.qk_norm_rope(q, k, k, freqs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_wrong_weights_are_refused():
    q, k = torch.zeros((1, 2, 4, 64), device="cuda"), torch.zeros((1, 2, 2, 64), device="cuda")
    freqs, _ = eg.rope_freqs(64)
    for w in (torch.ones(32, device="cuda"), torch.ones(64, device="cuda").bfloat16(), torch.ones(64), torch.ones(128, device="cuda")[::2]):
        with pytest.raises(eg.EagleError):
            eg.qk_norm_rope(q, k, None, freqs, w, None)
        with pytest.raises(eg.EagleError):
            eg.qk_norm_rope(q, k, None, freqs, None, w)
    with pytest.raises(eg.EagleError):
        eg.qk_norm_rope(q, k, None, freqs, eps=0.0)
