"""A path of a tree verified over selected pages, and its tokens decoded one by one
over a second cache, from every place of a page and past its end: the lists are the
same as long as the path stays in the page of the prefix's last position, and each
output is within its tolerance of fp64 over its own cache."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8 as okv8
from tree_speculative_decoding_eagle_gb300.cache import KV8Cache

pytestmark = pytest.mark.gpu
HQ, HKV, DH, P, TOP = 4, 2, 64, 16, 4
G, N, MP = HQ // HKV, 12, 12
bf = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def prefix(cache):
    """The cache's keys and values [Hkv, kv_len, dh] of its one request."""
    L = int(cache.kv_len)
    pages = cache.block_table[0, :-(-L // P)].tolist()
    got = []
    for codes, scale in ((cache.k_pages, cache.k_scale), (cache.v_pages, cache.v_scale)):
        x = okv8.decode(codes[0].view(torch.uint8).cpu().numpy()[pages]) * f64(scale[0])[pages][:, :, None, None]
        got.append(x.transpose(1, 0, 2, 3).reshape(HKV, -1, DH)[:, :L])
    return got


def check(cache, q, sel, out, lse, own_k, own_v):
    """One node: q, out [Hq, dh], lse [Hq], sel [Hkv, top], the rows of the tree that it names [Hkv, .., dh]."""
    K, W = prefix(cache)
    q, out, lse = f64(q), f64(out), f64(lse)
    for g in range(HKV):
        took = np.isin(np.arange(K.shape[1]) // P, [p for p in sel[g].tolist() if p >= 0])
        k, v = np.concatenate([K[g][took], own_k[g]]), np.concatenate([W[g][took], own_v[g]])
        heads = slice(g * G, (g + 1) * G)
        x = q[heads] @ k.T * DH ** -0.5
        assert np.abs(x).max() < 2 ** 5 and (np.abs(q[heads]) @ np.abs(k).T).max() * DH ** -0.5 < 2 ** 6
        top = x.max(1, keepdims=True)
        p = np.exp(x - top)
        total = p.sum(1, keepdims=True)
        p /= total
        ref, A = p @ v, p @ np.abs(v)
        # scores: DH products in float32, their sizes' sum below 2^6, and ex2 to 2^-21, above and below the line; sums of keys in float32
        w = 2 * (DH * 2.0 ** -23 * 2 ** 6 + 2.0 ** -21) + 2 * len(k) * 2.0 ** -24
        # the output's bf16, the weights' f16 (half a step is 2^-11, at least 2^-31 of the greatest weight; the scales of
        # values of N(0, 1) lie less than 2^4 apart)
        tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (2.0 ** -11 + w) * A + 2.0 ** -27 * np.abs(v).sum(0)
        assert (np.abs(out[heads] - ref) <= tol).all()
        want = (top + np.log(total))[:, 0]
        assert (np.abs(lse[heads] - want) <= w + 2.0 ** -22 * np.abs(want)).all()


@pytest.mark.parametrize("first,last", [(1, 1), (0, 2)])
def test_a_path_from_every_place_of_a_page(first, last):
    g = torch.Generator().manual_seed(10 * first + last)
    n = P + 4                                      # longer than a page
    mask, alone = eg.tree_mask(i32([[-1] + list(range(n - 1))])), eg.tree_mask(i32([[-1]]))
    one, slot = i32([1]), torch.empty(1, dtype=torch.int32, device="cuda")
    differ = 0
    for L in range(7 * P + 1, 8 * P + 1):
        caches = [KV8Cache(1, HKV, DH, P, N, MP, bounds=True) for _ in range(2)]
        x = torch.randn((2, L, HKV, DH), generator=g).to(bf).cuda()
        for c in caches:
            slots = torch.empty(L, dtype=torch.int32, device="cuda")
            c.reserve(i32([L]), slots)
            c.append(0, x[0], x[1], slots)
            c.grow(L)
        q = torch.randn((1, n, HQ, DH), generator=g).to(bf).cuda()
        kt, vt = (torch.randn((1, HKV, n, DH), generator=g).to(bf).cuda() for _ in range(2))
        tree_sel = caches[0].select(0, q, TOP, first, last)
        tree_out, tree_lse = caches[0].attend_pages(0, q, kt, vt, mask, tree_sel)
        for i in range(n):
            check(caches[0], q[0, i], tree_sel[0, i], tree_out[0, i], tree_lse[0, i], f64(kt[0, :, :i + 1]), f64(vt[0, :, :i + 1]))
            c, qi = caches[1], q[:, i:i + 1].contiguous()
            ki, vi = kt[:, :, i:i + 1].contiguous(), vt[:, :, i:i + 1].contiguous()
            sel = c.select(0, qi, TOP, first, last)
            out, lse = c.attend_pages(0, qi, ki, vi, alone, sel)
            check(c, qi[0, 0], sel[0, 0], out[0, 0], lse[0, 0], f64(ki[0]), f64(vi[0]))
            if (L + i - 1) // P == (L - 1) // P:
                assert torch.equal(sel[0, 0], tree_sel[0, i]), (L, i)
            else:                                  # the page behind the prefix takes a place of its own
                assert (sel[0, 0] == (L + i - 1) // P).any(-1).all()
                differ += not torch.equal(sel[0, 0], tree_sel[0, i])
            c.reserve(one, slot)
            c.append(0, ki[:, :, 0].contiguous(), vi[:, :, 0].contiguous(), slot)
            c.grow(one)
        assert int(caches[0].status) == 0 and int(caches[1].status) == 0
    assert differ > 0
