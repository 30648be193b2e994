"""Attention over selected pages of the 8-bit cache on the GPU against fp64.

Tolerances are those of test_gpu_kv8_attn.py, over the keys that a row's list and
mask leave; the tree's blocks of 16 nodes take their power of two from the nodes
that the row's own mask names."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from test_gpu_kv8_attn import Case, pack

pytestmark = pytest.mark.gpu


class Listed(Case):
    def __init__(self, kv_len, n, Hq, Hkv, dh, P, top, share=0.5, full=False, **kw):
        super().__init__(kv_len, n, Hq, Hkv, dh, P, **kw)
        rng = np.random.default_rng(kw.get("seed", 0) + top)
        B = len(kv_len)
        sel = np.full((B, n, Hkv, top), -1, np.int32)
        for b, L in enumerate(kv_len):
            live = -(-L // P)
            for g in range(Hkv):
                for i in range(n):
                    want = min(top, live) if full else int(rng.integers(0, min(top, live) + 1))
                    pages = set(rng.permutation(live)[:want].tolist())
                    if want and rng.random() < share:
                        pages = set(list(pages)[:want - 1]) | {live - 1}      # often the last, partial page
                    sel[b, i, g, :len(pages)] = sorted(pages)
        self.sel = torch.from_numpy(sel)

    def check(self, out, lse, scale=None):
        B, n, Hq, dh = self.q.shape
        Hkv, G, P = self.Hkv, Hq // self.Hkv, self.P
        scale = dh ** -0.5 if scale is None else scale
        for b, L in enumerate(self.kv_len):
            live_pages = -(-L // P)
            pages = self.table[b, :live_pages].long().cuda()
            K, V = (torch.cat([(codes[pages].view(torch.float8_e4m3fn).double() * sc[pages].double()[:, :, None, None])
                               .transpose(0, 1).reshape(Hkv, -1, dh)[:, :L], t[b].cuda().double()], 1)
                    for (codes, sc), t in zip(self.pools, (self.kt, self.vt)))
            took = torch.zeros((n, Hkv, live_pages + 1), dtype=torch.bool)
            took.scatter_(2, torch.where(self.sel[b] < 0, live_pages, self.sel[b]).long(), True)
            took = took[..., :live_pages].repeat_interleave(P, 2)[..., :L]
            live = torch.cat([took, self.keep[b][:, None].expand(n, Hkv, n)], 2).permute(1, 0, 2).cuda()     # [Hkv, n, L + n]
            q = self.q[b].cuda().double().view(n, Hkv, G, dh)
            x = torch.einsum("ngjd,gld->gjnl", q, K) * scale
            smax = (torch.einsum("ngjd,gld->gjnl", q.abs(), K.abs()) * scale).masked_fill(~live[:, None], 0.0).amax(-1)
            x = x.masked_fill(~live[:, None], -math.inf)
            ref_lse = torch.logsumexp(x, -1)
            p = torch.exp(x - ref_lse[..., None]).nan_to_num(0.0)
            ref = torch.einsum("gjnl,gld->ngjd", p, V.nan_to_num(0.0)).reshape(n, Hq, dh)
            A = torch.einsum("gjnl,gld->ngjd", p, V.nan_to_num(0.0).abs()).reshape(n, Hq, dh)
            w = (2 * (dh * 2.0 ** -23 * smax + 2.0 ** -21) + 2 * (L + n) * 2.0 ** -24).permute(2, 0, 1).reshape(n, Hq)
            # exponents: a page's, and of each row's blocks of 16 tree nodes: amax / 2^e in [2^8, 2^9)
            size = self.vt[b].cuda().double().abs().amax(2)[:, None] * self.keep[b].cuda()[None]              # [Hkv, n, n]
            size = torch.nn.functional.pad(size, (0, -n % 16)).view(Hkv, n, -1, 16).amax(3)
            te = torch.where(size > 0, torch.floor(torch.log2(size)) - 8, 0.0).repeat_interleave(16, 2)[..., :n]
            pe = self.pools[1][1][pages].double().log2().repeat_interleave(P, 0).T[:, :L]
            e = torch.cat([pe[:, None].expand(Hkv, n, L), te], 2)                                             # [Hkv, n, L + n]
            far = 2.0 ** -31 * (p * torch.exp2(e)[:, None]).amax(-1)                                          # [Hkv, G, n]
            # sum over a row's keys of |v| 2^-e
            sub = torch.einsum("gnl,gld->gnd", live.double() * torch.exp2(-e), V.nan_to_num(0.0).abs())
            sub = torch.einsum("gjn,gnd->ngjd", far, sub).reshape(n, Hq, dh)
            got = out[b].double()
            tol = sub + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + (2.0 ** -11 + w[..., None]) * A + 1e-30
            worst = float(((got - ref).abs() / tol).max())
            assert worst <= 1, (b, L, worst)
            rl, gl = ref_lse.permute(2, 0, 1).reshape(n, Hq), lse[b].double()
            empty = torch.isinf(rl)
            assert torch.equal(empty, torch.isinf(gl)) and (gl[empty] < 0).all()
            assert ((gl - rl).abs()[~empty] <= (w + 2.0 ** -22 * rl.abs())[~empty]).all(), (b, L)
            assert not got[empty].any()

    def call(self, scale=None, **kw):
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = eg.tree_attn_kv8_pages(*self.args(), self.sel.cuda(), scale=scale, status=self.status, **kw)
        torch.cuda.synchronize()
        return got

    def run(self, scale=None, **kw):
        out, lse = self.call(scale, **kw)
        assert int(self.status) == 0
        self.check(out, lse, scale)
        return out, lse


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_lengths_around_tiles_and_pages(P, dh):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 1000]
    for n in (1, 13):
        Listed(lens, n, 4, 2, dh, P, 5, seed=P).run()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (10, 2), (40, 8), (16, 1), (17, 1), (64, 2)])
@pytest.mark.parametrize("n", [1, 2, 17, 33, 65, 130])
def test_heads_and_nodes(Hq, Hkv, n):
    Listed([70, 0, 331], n, Hq, Hkv, 64 if n % 2 else 128, 16, 7, seed=n).run()


@pytest.mark.parametrize("n,Hq,Hkv,dh,top", [(1, 8, 1, 128, 64), (1, 4, 4, 64, 300), (1, 32, 1, 128, 64), (61, 8, 1, 64, 16), (7, 2, 1, 128, 40)])
@pytest.mark.parametrize("L", [4096, 20011])
def test_long_prefixes(n, Hq, Hkv, dh, top, L):
    """Split over CTAs, with a cluster's merge and with the merge kernel."""
    Listed([L], n, Hq, Hkv, dh, 64, top, seed=L, full=True).run()


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n,Hq", [(17, 4), (61, 2), (61, 16), (140, 4)])
def test_trees_of_many_rows(P, dh, n, Hq):
    """One, two and several groups of rows, whose nodes share lists."""
    Listed([0, 1, 15, 17, 64, 129, 255, 700], n, Hq, 2, dh, P, 5, seed=P).run()
    Listed([1500], n, Hq, 2, dh, P, 40, seed=P, full=True).run()


def test_nodes_that_share_no_page():
    """Each node lists pages of its own: the union is most of the prefix, in several words of bits."""
    c = Listed([61 * 32 + 7], 61, 16, 2, 128, 16, 2, full=True)
    c.sel[0] = (2 * torch.arange(61)[:, None, None] + torch.arange(2)).to(torch.int32).expand(61, 2, 2)
    c.sel[0, 60, :, 1] = 122
    c.run()
    c.sel[0, 1::2] = -1
    c.run()


def test_one_head_of_a_tree_lists_nothing():
    c = Listed([300, 40], 61, 16, 2, 64, 16, 4)
    c.sel[:, :, 1] = -1
    c.run()
    c.sel[0] = -1
    c.run()


def test_many_sequences_of_all_lengths():
    g = np.random.default_rng(0)
    Listed(g.integers(0, 2000, 70).tolist(), 1, 16, 8, 128, 32, 9).run()
    Listed(g.integers(0, 2000, 40).tolist(), 9, 16, 8, 64, 32, 9).run()
    Listed(g.integers(0, 2000, 40).tolist(), 1, 64, 8, 64, 16, 100, full=True).run()


def test_more_places_than_pages_and_a_wide_table():
    for n in (1, 30):
        Listed([3, 0, 40], n, 8, 8, 128, 64, 33, extra_pages=200).run()
        Listed([3, 0, 40], n, 8, 8, 128, 16, 1000, extra_pages=3, full=True).run()


def test_all_pages_is_the_whole_prefix():
    """Every page listed: the same keys as without a list, within both tolerances."""
    c = Listed([100, 333], 5, 8, 2, 128, 16, 21, full=True)
    c.sel = torch.full_like(c.sel, -1)
    for b, L in enumerate(c.kv_len):
        c.sel[b, ..., :-(-L // 16)] = torch.arange(-(-L // 16), dtype=torch.int32)
    out, lse = c.run()
    Case.check(c, out, lse)


def test_tables_too_wide_for_shared_lists():
    """More pages a request than a group's map holds: many rows node by node."""
    Listed([40, 300], 20, 4, 2, 64, 16, 3, extra_pages=16400).run()
    Listed([40, 300], 5, 24, 2, 64, 16, 3, extra_pages=16400).run()


def test_long_chains_of_nodes():
    for n in (200, 517):
        Listed([0, 75], n, 4, 2, 64, 16, 3, keep=torch.ones((2, n, n)).tril().bool()).run()
        Listed([0, 75], n, 2, 2, 128, 16, 3, keep=torch.ones((2, n, n)).tril().bool()).run()


def test_masks_that_leave_nothing():
    keep = torch.zeros((2, 40, 40), dtype=torch.bool)
    keep[0, 3, 39] = keep[1, 20, 16] = True
    c = Listed([0, 50], 40, 4, 2, 128, 16, 2, keep=keep)
    c.sel[1, ::2] = -1
    out, lse = c.run()
    assert not out[0, 0].any() and torch.isinf(lse[0, 0]).all() and not out[1, 0].any()


def test_nodes_that_a_row_does_not_name_do_not_count_whatever_they_hold():
    c = Listed([50], 20, 4, 2, 128, 16, 2)
    want, want_lse = c.run()
    gone = ~c.keep[0].any(0)
    c.keep[0, :, 7] = False
    c.keep[0, 7] = False
    want, want_lse = c.run()
    c.kt[0, :, 7], c.vt[0, :, 7] = float("nan"), float("inf")
    out, lse = c.call()
    assert torch.equal(out, want) and torch.equal(lse, want_lse), gone


def test_mask_bits_past_the_last_node_count_for_nothing():
    c = Listed([50], 20, 4, 2, 128, 16, 2)
    want, want_lse = c.run()
    a = list(c.args())
    a[9] = a[9] | (-1 << 20)
    out, lse = eg.tree_attn_kv8_pages(*a, c.sel.cuda())
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_scale_and_large_scores():
    Listed([100], 3, 4, 2, 128, 16, 3, q_size=30.0).run()
    Listed([100], 3, 4, 2, 64, 16, 3).run(scale=2.0)


def test_a_nan_reaches_the_rows_that_list_it():
    c = Listed([64], 4, 4, 2, 128, 16, 4)
    c.sel[:] = -1
    c.sel[0, 0, :, 0], c.sel[0, 1, :, 0], c.sel[0, 2, :, :2], c.sel[0, 3, :, 0] = 0, 1, torch.tensor([1, 3], dtype=torch.int32), 2
    want, want_lse = c.run()
    for pool in (0, 1):
        code = c.pools[pool][0][int(c.table[0, 1]), 1, 3, 7].clone()
        c.pools[pool][0][int(c.table[0, 1]), 1, 3, 7] = 0x7f
        out, lse = c.call()
        hit = torch.zeros((4, 4), dtype=torch.bool, device="cuda")
        hit[1:3, 2:] = True
        assert out[0][hit].isnan().any(-1).all()
        assert torch.equal(out[0][~hit], want[0][~hit]) and torch.equal(lse[0][~hit], want_lse[0][~hit])
        c.pools[pool][0][int(c.table[0, 1]), 1, 3, 7] = code


@pytest.mark.parametrize("n,Hq", [(3, 4), (61, 8)])
def test_lists_that_are_not_lists(n, Hq):
    """Pages past the prefix count for nothing, whatever else stands in the list
    stays in range; both are reported."""
    c = Listed([100, 40], n, Hq, 2, 128, 16, 6)
    c.sel[:] = -1
    c.sel[0, ..., :3] = torch.tensor([0, 2, 6], dtype=torch.int32)
    want, want_lse = c.run()
    for past in (7, 8, 1000, 2 ** 31 - 1):
        c.sel[0, ..., 3] = past
        out, lse = c.call()
        assert int(c.status) == -1 and torch.equal(out, want) and torch.equal(lse, want_lse)
    c.sel[0, ..., 3:] = torch.tensor([1, 6, 2], dtype=torch.int32)
    out, lse = c.call()
    assert int(c.status) == -1 and torch.isfinite(out.float()).all() and torch.equal(out[1], want[1])
    c.sel[0, ..., 3:] = torch.tensor([-5, 4, 5], dtype=torch.int32)      # behind the first negative entry
    out, lse = c.call()
    assert int(c.status) == 0 and torch.equal(out, want)
    c.table[0, 2] = -1                                                   # not a page of the pool: page 0 in its place
    c.pools[0][0][0], c.pools[1][0][0] = 0x30, 0x30
    c.pools[0][1][0], c.pools[1][1][0] = 1.0, 1.0
    out, lse = c.call()
    assert int(c.status) == -1 and torch.isfinite(out.float()).all()


def test_the_most_sequences():
    """65535 sequences of a KV head, with few rows and with many.  Rows are weighted
    means of values up to vmax, each side's off by at most (2^-8 + 2^-10) vmax."""
    g = torch.Generator(device="cuda").manual_seed(1)
    B, dh, N = 65535, 64, 300
    k, v = (torch.randn(N, 1, 16, dh, generator=g, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ones = torch.ones(N, 1, device="cuda")
    table = torch.randint(0, N, (B, 9), generator=g, device="cuda", dtype=torch.int32)
    kv = torch.randint(0, 9 * 16 + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    for n in (1, 33):
        q = torch.randn(B, n, 1, dh, generator=g, device="cuda").to(torch.bfloat16)
        kt, vt = (torch.randn(B, 1, n, dh, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        mask = (torch.ones(n, dtype=torch.int64, device="cuda") << torch.arange(n, device="cuda")).expand(B, n)[..., None].contiguous()
        sel = torch.randint(0, 9, (B, n, 1, 2), generator=g, device="cuda", dtype=torch.int32).sort(-1).values
        sel[..., 1] += 1                           # ascending; past the prefix: counts for nothing
        sel = torch.where(sel * 16 < kv[:, None, None, None], sel, -1).to(torch.int32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = eg.tree_attn_kv8_pages(q, k, v, ones, ones, table, kv, kt, vt, mask, sel, status=status)
        assert int(status) == 0
        for part in (slice(0, 50), slice(65485, 65535)):
            cut = [x[part].contiguous() for x in (table, kv, kt, vt, mask, sel)]
            got, got_lse = eg.tree_attn_kv8_pages(q[part].contiguous(), k, v, ones, ones, *cut)
            vmax = float(max(v.float().abs().max(), vt.float().abs().max()))
            assert float((got.float() - out[part].float()).abs().max()) <= 2 * (2.0 ** -8 + 2.0 ** -10) * vmax
            assert float((got_lse - lse[part]).abs().max()) <= 1e-4


def test_offsets_past_31_bits():
    """A pool of more than 2^31 bytes, its last pages in use."""
    Listed([200, 70], 2, 4, 2, 128, 256, 1, num_pages=40000).run()


def test_stream_workspace_and_capture():
    c = Listed([4096, 100], 2, 8, 2, 128, 64, 64, full=True)
    want, want_lse = c.run()
    a = (*c.args(), c.sel.cuda())
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, lse = eg.tree_attn_kv8_pages(*a, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    ws, out = eg.Workspace("cuda"), torch.zeros_like(got)
    eg.tree_attn_kv8_pages(*a, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.tree_attn_kv8_pages(*a, out=out, lse=lse, workspace=ws)
    a[-1][:, :, 0, 5:] = -1
    graph.replay()
    fresh, _ = eg.tree_attn_kv8_pages(*a)
    torch.cuda.synchronize()
    assert torch.equal(out, fresh) and not torch.equal(out, want)


def test_binding_refuses():
    c = Listed([70], 2, 4, 2, 64, 16, 3)
    a, sel = c.args(), c.sel.cuda()
    for bad in (sel.long(), sel[:, :1], sel.cpu(), sel[..., ::2], sel[:, :, :1]):
        with pytest.raises(eg.EagleError):
            eg.tree_attn_kv8_pages(*a, bad)
    with pytest.raises(eg.EagleError):
        eg.tree_attn_kv8_pages(a[0].float(), *a[1:], sel)
