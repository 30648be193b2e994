"""Edges of the attention over the 8-bit cache at the sizes where a key tile has
one scale (more than 128 query rows a KV head, pages no shorter than a tile), whose
kernels are instances of their own; and the pages that no kernel may follow."""
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from test_gpu_kv8_attn import Case, random_tree

pytestmark = pytest.mark.gpu
ONE = [(61, 8, 64, 128), (61, 8, 128, 64), (200, 2, 64, 256), (333, 1, 128, 128)]          # n, G, dh, P
OTHERS = [(3, 2, 64, 16), (20, 1, 128, 32), (61, 1, 128, 16), (61, 2, 64, 64), (61, 2, 128, 16), (61, 8, 64, 64), (61, 8, 128, 32)]


@pytest.mark.parametrize("n,G,dh,P", ONE)
@pytest.mark.parametrize("which", [0, 1])
def test_a_nan_in_the_cache_reaches_the_rows_that_read_it(n, G, dh, P, which):
    c = Case([P + 40, P + 33], n, 2 * G, 2, dh, P)
    want, want_lse = c.run()
    c.pools[which][0][int(c.table[1, 1]), 1, 3, 7] = 0x7f
    out, lse = eg.tree_attn_kv8(*c.args())
    hit = torch.zeros((2, n, 2 * G), dtype=torch.bool, device="cuda")
    hit[1, :, G:] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    if which == 0:
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    else:
        assert torch.isnan(out[hit][:, 7]).all() and torch.equal(lse[hit], want_lse[hit])
        assert torch.isfinite(out[hit][:, :7]).all() and torch.isfinite(out[hit][:, 8:]).all()


@pytest.mark.parametrize("n,G,dh,P", ONE)
def test_rows_without_keys(n, G, dh, P):
    keep = random_tree(n, 3, torch.Generator().manual_seed(1))
    keep[:, 0] = False
    keep[1, n // 2] = False
    Case([0, 0, 20], n, 2 * G, 2, dh, P, keep=keep).run()
    Case([0, 0, 3 * P + 20], n, 2 * G, 2, dh, P, keep=torch.zeros_like(keep)).run()


@pytest.mark.parametrize("n,G,dh,P", ONE)
def test_scales_far_apart(n, G, dh, P):
    """Neighbouring pages whose scales differ by 2^40, and a page of zeros at the least scale."""
    c = Case([6 * P, 5 * P], n, 2 * G, 2, dh, P, seed=3)
    for codes, scale in c.pools:
        scale[c.table[0, 1].item()] *= 2.0 ** -40
        scale[c.table[0, 4].item()] *= 2.0 ** -20
        codes[c.table[1, 2].item()] = 0
        scale[c.table[1, 2].item()] = 2.0 ** -64
    c.pools[1][1][c.table[0, 2].item()] *= 2.0 ** 40
    c.run()


@pytest.mark.parametrize("n,G,dh,P", ONE)
def test_peaked_and_flat_softmax(n, G, dh, P):
    Case([3 * P + 9, 77], n, 2 * G, 2, dh, P, q_size=30.0).run()
    Case([3 * P + 9, 77], n, 2 * G, 2, dh, P, q_size=0.0).run()
    Case([3 * P + 9, 77], n, 2 * G, 2, dh, P).run(scale=3.0)
    Case([3 * P + 9, 77], n, 2 * G, 2, dh, P).run(scale=1e-6)


@pytest.mark.parametrize("n,G,dh,P", ONE[:2])
def test_wide_table_and_far_pages(n, G, dh, P):
    Case([3, 0, P + 40], n, 8 * G, 8, dh, P, extra_pages=200).run()
    Case([200, 17], n, 8 * G, 8, dh, P, num_pages=(9 << 29) // (8 * P * dh)).run()


@pytest.mark.parametrize("n,G,dh,P", ONE)
def test_same_bits_on_every_call_stream_and_replay(n, G, dh, P):
    c = Case([1500, 900], n, 4 * G, 4, dh, P)
    args, ws = c.args(), eg.Workspace("cuda")
    out, lse = c.run(workspace=ws)
    for _ in range(3):
        o, l = eg.tree_attn_kv8(*args, workspace=ws)
        assert torch.equal(o, out) and torch.equal(l, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, l = eg.tree_attn_kv8(*args)
    s.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    g = torch.cuda.CUDAGraph()
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.graph(g):
        eg.tree_attn_kv8(*args, out=o2, lse=l2, workspace=ws)
    g.replay()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    args[6].fill_(333)                              # kv_len in place: the graph reads it anew
    c.kv_len = [333, 333]
    g.replay()
    torch.cuda.synchronize()
    c.check(o2, l2)


@pytest.mark.parametrize("n,G,dh,P", ONE + OTHERS)
def test_page_0_is_read_in_place_of_an_unmapped_page(n, G, dh, P):
    c = Case([4 * P, 4 * P], n, 2 * G, 2, dh, P)
    for i, (codes, scale) in enumerate(c.pools):    # page 0: numbers of its own, whoever maps it
        codes[0], scale[0] = 0x30 + 9 * i, 2.0 ** (-7 - i)
    good = list(c.args())
    for bad in (-1, c.pools[0][0].shape[0], 2 ** 31 - 1, -2 ** 31):
        args, status = list(good), torch.zeros(1, dtype=torch.int32, device="cuda")
        args[5] = good[5].clone()
        args[5][1, 2] = bad
        out, lse = eg.tree_attn_kv8(*args, status=status)
        assert int(status) == -1
        args[5][1, 2] = 0
        want, want_lse = eg.tree_attn_kv8(*args)
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and torch.isfinite(out).all()
