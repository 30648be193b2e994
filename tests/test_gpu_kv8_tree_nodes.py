"""Attention over the 8-bit cache: tree nodes that no row attends to, and nodes
much larger than their neighbours."""
import math

import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from test_gpu_kv8_attn import Case, random_tree

pytestmark = pytest.mark.gpu

# few rows (one and two row tiles), one M-tile of 64 and 128 rows, two M-tiles with
# scales of groups and (pages no shorter than a key tile) of whole tiles, several tiles
SHAPES = [(5, 2, 64, 16), (5, 2, 128, 64), (13, 2, 64, 32), (13, 2, 128, 16), (61, 1, 128, 16), (61, 1, 64, 64), (61, 2, 128, 32),
          (61, 8, 64, 16), (61, 8, 128, 32), (61, 8, 64, 128), (61, 8, 128, 64), (200, 2, 64, 256), (333, 1, 128, 128), (150, 1, 64, 16)]


@pytest.mark.parametrize("n,G,dh,P", SHAPES)
@pytest.mark.parametrize("what", [2.0 ** 30, -2.0 ** 100, math.inf, math.nan])
def test_nodes_that_no_row_names_decide_nothing(n, G, dh, P, what):
    """Padding: the last third of the nodes and one in the middle.  The reference
    and its tolerance are those of a tree without them."""
    keep = random_tree(n, 2, torch.Generator().manual_seed(n))
    pad = torch.zeros(n, dtype=torch.bool)
    pad[n - n // 3:] = True
    pad[2] = True
    keep[:, :, pad] = False
    keep[:, pad] = False
    c = Case([77, 0], n, 2 * G, 2, dh, P, keep=keep)
    args = list(c.args())
    for i in (7, 8):
        args[i] = args[i].clone()
        args[i][:, :, pad.cuda()] = what
    out, lse = eg.tree_attn_kv8(*args)
    c.check(out, lse)
    # and not a bit depends on what they hold
    for i in (7, 8):
        args[i][:, :, pad.cuda()] = 0.5
    again, lse2 = eg.tree_attn_kv8(*args)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("n,G,dh,P", [(4096, 1, 64, 16), (2100, 2, 128, 64), (4096, 1, 128, 4096), (1300, 4, 64, 128)])
def test_long_chains_with_padding_between(n, G, dh, P):
    """A prompt chunk up to the largest, every eleventh node padding."""
    keep = torch.ones((1, n, n)).tril().bool()
    pad = torch.arange(n) % 11 == 5
    keep[:, :, pad] = False
    keep[:, pad] = False
    c = Case([70], n, G, 1, dh, P, keep=keep)
    args = list(c.args())
    for i in (7, 8):
        args[i] = args[i].clone()
        args[i][:, :, pad.cuda()] = math.nan
    c.check(*eg.tree_attn_kv8(*args))


class Uneven(Case):
    """The tolerance with blocks of `block` nodes and what a large node costs the
    others: every element of k_tree and v_tree is off by up to 2^-33 of its
    block's largest.  A score is then off by d = scale sum_c |q_c| 2^-33 max|k|,
    a weight by a factor of e^(+-2 d) at most (numerator and sum), the output by
    (e^(2 d) - 1) A + 2^-33 max|v|, lse by d."""

    def blocks(self, t, block):
        m = t.cuda().double().abs().amax(-1)                                   # [B, Hkv, n]
        m = torch.nn.functional.pad(m, (0, -self.n % block)).unflatten(-1, (-1, block)).amax(-1)
        return m.repeat_interleave(block, -1)[..., :self.n]

    def check(self, out, lse, block):
        B, n, Hq, dh = self.q.shape
        H, G = self.Hkv, Hq // self.Hkv
        kmax, vmax = self.blocks(self.kt, block), self.blocks(self.vt, block)
        for b, L in enumerate(self.kv_len):
            pages = self.table[b, :-(-L // self.P)].long().cuda()
            K, V = (torch.cat([(codes[pages].view(torch.float8_e4m3fn).double() * sc[pages].double()[:, :, None, None])
                               .transpose(0, 1).reshape(H, -1, dh)[:, :L], t[b].cuda().double()], 1)
                    for (codes, sc), t in zip(self.pools, (self.kt, self.vt)))
            q = self.q[b].cuda().double().view(n, H, G, dh)
            scale = dh ** -0.5
            live = torch.cat([torch.ones((n, L), dtype=torch.bool), self.keep[b]], 1).cuda()
            x = (torch.einsum("ngjd,gld->gjnl", q, K) * scale).masked_fill(~live, -math.inf)
            smax = (torch.einsum("ngjd,gld->gjnl", q.abs(), K.abs()) * scale).masked_fill(~live, 0.0).amax(-1)
            ref_lse = torch.logsumexp(x, -1)
            p = torch.exp(x - ref_lse[..., None])
            rows = lambda t: t.permute(2, 0, 1, *range(3, t.dim())).reshape(n, Hq, *t.shape[3:])
            ref, A = (rows(torch.einsum("gjnl,gld->gjnd", p, v)) for v in (V, V.abs()))
            d = scale * q.abs().sum(-1).permute(1, 2, 0) * 2.0 ** -33 * (live[:, L:][None] * kmax[b][:, None]).amax(-1)[:, None]
            w = 2 * (dh * 2.0 ** -23 * smax + 2.0 ** -21) + 2 * (L + n) * 2.0 ** -24
            pv = 2.0 ** -33 * torch.einsum("gjnl,gl->gjn", p[..., L:], vmax[b])
            e = torch.cat([self.pools[1][1][pages].double().log2().repeat_interleave(self.P, 0).T[:, :L],
                           torch.floor(torch.log2(vmax[b])) - 8], 1)
            far = 2.0 ** -31 * (p * torch.exp2(e)[:, None, None]).amax(-1)
            sub = torch.einsum("gnl,gld->gnd", live.double().expand(H, -1, -1), V.abs() * torch.exp2(-e)[..., None])
            sub = torch.einsum("gjn,gnd->gjnd", far, sub)
            tol = (rows(sub) + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + rows(pv)[..., None]
                   + (2.0 ** -11 + rows(w + torch.expm1(2 * d))[..., None]) * A)
            err = (out[b].double() - ref).abs()
            assert float((err / tol).max()) <= 1, (b, float((err / tol).max()))
            assert ((lse[b].double() - rows(ref_lse)).abs() <= rows(w + d) + 2.0 ** -22 * rows(ref_lse).abs()).all()


@pytest.mark.parametrize("n,G,dh,P", SHAPES)
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 20])
def test_a_node_far_larger_than_its_neighbours(n, G, dh, P, size):
    """One node, named by its own row alone (whose scores are then beyond any
    other's), among nodes of ordinary size: the other rows keep the stated bits."""
    keep = random_tree(n, 2, torch.Generator().manual_seed(n))
    keep[:, :, n - 2] = False
    keep[:, n - 2, n - 2] = True
    c = Uneven([77, 130], n, 2 * G, 2, dh, P, keep=keep)
    c.kt[:, :, n - 2] *= size
    c.vt[:, :, n - 2] *= size
    big = n * G > 128
    tile = 128 if dh == 64 else 64
    out, lse = eg.tree_attn_kv8(*c.args())
    c.check(out, lse, tile if big and P >= tile else 16)
