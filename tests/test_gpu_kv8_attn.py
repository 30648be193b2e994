"""Tree attention over the 8-bit paged cache on the GPU against fp64.

Tolerance of an output element, with A the row's softmax-weighted sum of |v|
and smax the row's largest sum of scale * |q_c k_c| over the columns:
  * the output's rounding, 2^-8 |o| (bf16);
  * weights rounded to f16 for the product with V, numerator only: f16 holds
    1 + 10 bits, so its step is 2^-10 of the value's power of two and half a
    step 2^-11 relative (torch.finfo(torch.float16).eps / 2): 2^-11 A;
  * f16's subnormals end at 2^-24, so a weight is also off by up to 2^-25 as it
    is held.  It is held as P' = 2^(s + e - m + 6), e its value's block
    exponent (v = 2^e v') and m at most max_k (s_k + e_k).  In the output, P' v'
    counts 2^(m - 6) / Z with Z = sum 2^s: key k is off by at most
    2^-25 |v'_k| 2^-6 max_j (2^(s_j + e_j)) / Z = 2^-31 |v_k| 2^-e_k max_j (p_j 2^e_j),
    summed over the keys that count;
  * scores: dh products accumulated in fp32, at most dh 2^-24 smax, the same
    again where they are scaled to base 2, and ex2's 2^-22: relative error of
    a weight in the numerator and in the sum below, so twice
    (dh 2^-23 smax + 2^-21) A;
  * the sums over N keys in fp32: 2 N 2^-24 A.
lse takes the last two without A, and 2^-22 of its own size."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8 as okv8

pytestmark = pytest.mark.gpu


def random_tree(n, B, g):
    keep = torch.zeros((B, n, n), dtype=torch.bool)
    for b in range(B):
        for i in range(n):
            if i:
                p = int(torch.randint(max(0, i - 8), i, (1,), generator=g))
                keep[b, i] = keep[b, p]
            keep[b, i, i] = True
    return keep


def pack(keep):
    B, n, _ = keep.shape
    W = (n + 63) // 64
    bits = torch.zeros((B, n, W * 64), dtype=torch.int64)
    bits[:, :, :n] = keep.long()
    return (bits.view(B, n, W, 64) << torch.arange(64)).sum(3).contiguous().cuda()


class Case:
    """Inputs: every page that no prefix uses, every row at or past kv_len and
    every unused scale hold rubbish (NaN numbers among it)."""

    def __init__(self, kv_len, n, Hq, Hkv, dh, P, seed=0, extra_pages=0, num_pages=None, keep=None, q_size=1.0):
        g = torch.Generator().manual_seed(seed + 31 * n + dh)
        B = len(kv_len)
        self.kv_len, self.n, self.P, self.Hkv = kv_len, n, P, Hkv
        self.mp = max(1, max(-(-k // P) for k in kv_len)) + extra_pages
        N = num_pages or B * self.mp + 3
        used = sum(-(-k // P) for k in kv_len)
        at = torch.randperm(N, generator=g)[:used] if N < 10 ** 6 else N - 1 - torch.randperm(used, generator=g)
        table = torch.full((B, self.mp), -1, dtype=torch.int32)
        i = 0
        for b, k in enumerate(kv_len):
            c = -(-k // P)
            table[b, :c] = at[i:i + c].int()
            i += c
        self.table = table
        self.pools = []
        for _ in range(2):
            codes = torch.empty((N, Hkv, P, dh), dtype=torch.uint8, device="cuda")
            codes.view(-1)[:1 << 20].fill_(0x7f)
            codes.fill_(0x7f) if N * Hkv * P * dh < 1 << 28 else None
            scale = torch.full((N, Hkv), 2.0 ** 60, device="cuda")
            if used:
                x = torch.randn((used, Hkv, P, dh), generator=g) * torch.exp2(torch.randn((used, Hkv, 1, 1), generator=g) * 1.5)
                e = np.vectorize(okv8.block_exponent)(x.abs().amax((2, 3)).double().numpy())
                s = torch.from_numpy(2.0 ** e).float()
                c = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                i = 0
                for k in kv_len:
                    m = -(-k // P)
                    if m and k % P:
                        c[i + m - 1, :, k % P:] = 0x7f
                    i += m
                codes[at.cuda()] = c.cuda()
                scale[at.cuda()] = s.cuda()
            self.pools.append((codes, scale))
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
        self.q = (bf(B, n, Hq, dh) * q_size).to(torch.bfloat16)
        self.kt, self.vt = bf(B, Hkv, n, dh), bf(B, Hkv, n, dh)
        self.keep = random_tree(n, B, g) if keep is None else keep

    def args(self):
        (kp, ks), (vp, vs) = self.pools
        return (self.q.cuda(), kp, vp, ks, vs, self.table.cuda(), torch.tensor(self.kv_len, dtype=torch.int32, device="cuda"),
                self.kt.cuda(), self.vt.cuda(), pack(self.keep))

    def tree_exponents(self, b):
        """Exponents of the tree's value blocks (16 nodes of a head): amax / 2^e in [2^8, 2^9)."""
        v = self.vt[b].cuda().double().abs().amax(2)                                  # [Hkv, n]
        v = torch.nn.functional.pad(v, (0, -self.n % 16)).view(self.Hkv, -1, 16).amax(2)
        return (torch.floor(torch.log2(v)) - 8).repeat_interleave(16, 1)[:, :self.n]

    def check(self, out, lse, scale=None):
        B, n, Hq, dh = self.q.shape
        G = Hq // self.Hkv
        scale = dh ** -0.5 if scale is None else scale
        for b, L in enumerate(self.kv_len):
            pages = self.table[b, :-(-L // self.P)].long().cuda()
            K, V = (torch.cat([(codes[pages].view(torch.float8_e4m3fn).double() * sc[pages].double()[:, :, None, None])
                               .transpose(0, 1).reshape(self.Hkv, -1, dh)[:, :L], t[b].cuda().double()], 1)
                    for (codes, sc), t in zip(self.pools, (self.kt, self.vt)))
            q = self.q[b].cuda().double().view(n, self.Hkv, G, dh)
            x = torch.einsum("ngjd,gld->gjnl", q, K) * scale
            smax = (torch.einsum("ngjd,gld->gjnl", q.abs(), K.abs()) * scale).amax(-1)
            live = torch.cat([torch.ones((n, L), dtype=torch.bool), self.keep[b]], 1).cuda()
            x = x.masked_fill(~live, -math.inf)
            ref_lse = torch.logsumexp(x, -1)
            p = torch.exp(x - ref_lse[..., None]).nan_to_num(0.0)
            ref = torch.einsum("gjnl,gld->ngjd", p, V).reshape(n, Hq, dh)
            A = torch.einsum("gjnl,gld->ngjd", p, V.abs()).reshape(n, Hq, dh)
            w = (2 * (dh * 2.0 ** -23 * smax + 2.0 ** -21) + 2 * (L + n) * 2.0 ** -24).permute(2, 0, 1).reshape(n, Hq)
            e = torch.cat([self.pools[1][1][pages].double().log2().repeat_interleave(self.P, 0).T[:, :L],
                           self.tree_exponents(b)], 1)                                # [Hkv, L + n]
            far = 2.0 ** -31 * (p * torch.exp2(e)[:, None, None]).amax(-1)
            sub = torch.einsum("gnl,gld->gnd", live.double().expand(self.Hkv, -1, -1), V.abs() * torch.exp2(-e)[..., None])
            sub = torch.einsum("gjn,gnd->ngjd", far, sub).reshape(n, Hq, dh)
            got = out[b].double()
            tol = sub + 2.0 ** -8 * ref.abs() * (1 + 2.0 ** -8) + (2.0 ** -11 + w[..., None]) * A + 1e-30
            err = (got - ref).abs()
            worst = float((err / tol).max())     # NaN where the output is
            assert worst <= 1, (b, L, worst)
            rl = ref_lse.permute(2, 0, 1).reshape(n, Hq)
            gl = lse[b].double()
            empty = torch.isinf(rl)
            assert torch.equal(empty, torch.isinf(gl)) and (gl[empty] < 0).all()
            assert ((gl - rl).abs()[~empty] <= (w + 2.0 ** -22 * rl.abs())[~empty]).all(), (b, L)
            assert not got[empty].any()

    def run(self, scale=None, **kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = eg.tree_attn_kv8(*self.args(), scale=scale, status=status, **kw)
        torch.cuda.synchronize()
        assert int(status) == 0
        self.check(out, lse, scale)
        return out, lse


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_lengths_around_tiles_and_pages(P, dh):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257]
    for n in (1, 13, 61):
        Case(lens, n, 4, 2, dh, P, seed=P).run()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (10, 2), (40, 8), (12, 4), (16, 1), (20, 1), (64, 2)])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 8, 16, 17, 33, 64, 65, 130])
def test_heads_and_nodes(Hq, Hkv, n):
    Case([70, 0, 131], n, Hq, Hkv, 64 if n % 2 else 128, 16, seed=n).run()


@pytest.mark.parametrize("n,Hq,Hkv,dh", [(1, 8, 1, 128), (1, 4, 4, 64), (7, 2, 1, 64), (61, 2, 2, 128), (49, 8, 1, 128), (61, 8, 1, 64)])
@pytest.mark.parametrize("L", [1000, 4096, 20011])
def test_long_prefixes(n, Hq, Hkv, dh, L):
    Case([L], n, Hq, Hkv, dh, 64, seed=L).run()


def test_many_sequences_of_all_lengths():
    g = np.random.default_rng(0)
    Case(g.integers(0, 700, 70).tolist(), 1, 16, 8, 128, 32).run()
    Case(g.integers(0, 700, 70).tolist(), 9, 16, 8, 64, 32).run()
    Case(g.integers(0, 700, 40).tolist(), 61, 8, 8, 128, 16).run()
    Case(g.integers(0, 700, 40).tolist(), 61, 64, 8, 64, 16).run()


def test_wide_table_and_short_prefixes():
    """A block table far wider than what is used: splits without any key."""
    for n in (1, 61):
        Case([3, 0, 40], n, 8, 8, 128, 64, extra_pages=200).run()


def test_long_chains_of_nodes():
    """A prompt chunk: causal chain, several tiles and mask words of nodes."""
    for n in (200, 517, 1030):
        Case([0, 75], n, 4, 2, 64, 16, keep=torch.ones((2, n, n)).tril().bool()).run()
        Case([0, 75], n, 2, 2, 128, 16, keep=torch.ones((2, n, n)).tril().bool()).run()


@pytest.mark.parametrize("n,Hq", [(1, 4), (5, 16), (61, 4), (61, 16)])
@pytest.mark.parametrize("which", [0, 1])
def test_a_nan_in_the_cache_reaches_the_rows_that_read_it(n, Hq, which):
    """A NaN key or value of one head and sequence; the others stay as they are."""
    c = Case([40, 33], n, Hq, 2, 128, 16)
    want, want_lse = c.run()
    page = int(c.table[1, 1])
    c.pools[which][0][page, 1, 3, 7] = 0x7f
    out, lse = eg.tree_attn_kv8(*c.args())
    hit = torch.zeros((2, n, Hq), dtype=torch.bool, device="cuda")
    hit[1, :, Hq // 2:] = True
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    if which == 0:
        assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    else:                                            # a NaN value: its column, in every row
        assert torch.isnan(out[hit][:, 7]).all() and torch.equal(lse[hit], want_lse[hit])
        assert torch.isfinite(out[hit][:, :7]).all() and torch.isfinite(out[hit][:, 8:]).all()


def test_captured_without_a_call_before():
    """Nothing that a first call sets up is forbidden during capture (a fresh
    process would show it; here at least a shape not met before)."""
    for n, Hq in ((3, 2), (90, 2)):
        c = Case([37], n, Hq, 1, 64, 256, seed=99)
        args, ws = c.args(), eg.Workspace("cuda")
        ws.get(1 << 20)
        out, lse = torch.empty((1, n, Hq, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((1, n, Hq), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            eg.tree_attn_kv8(*args, out=out, lse=lse, workspace=ws)
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_rows_without_keys():
    """Empty mask rows: no key at all where kv_len is 0, the prefix alone otherwise."""
    for n in (1, 4, 61):
        keep = random_tree(n, 3, torch.Generator().manual_seed(1))
        keep[:, 0] = False
        keep[1, n // 2] = False
        Case([0, 0, 20], n, 8, 2, 64, 16, keep=keep).run()
        Case([0, 0, 20], n, 8, 2, 128, 16, keep=torch.zeros_like(keep)).run()


@pytest.mark.parametrize("n", [1, 61])
def test_peaked_and_flat_softmax(n):
    Case([300, 77], n, 4, 2, 128, 16, q_size=30.0).run()
    Case([300, 77], n, 4, 2, 128, 16, q_size=0.0).run()
    Case([300, 77], n, 4, 2, 64, 16).run(scale=3.0)
    Case([300, 77], n, 4, 2, 64, 16).run(scale=1e-6)


@pytest.mark.parametrize("n,G", [(1, 1), (1, 8), (20, 1), (61, 8)])
def test_scales_far_apart(n, G):
    """Neighbouring pages whose scales differ by 2^40, and a page of zeros at the least scale."""
    c = Case([96, 80], n, 2 * G, 2, 64, 16, seed=3)
    for codes, scale in c.pools:
        scale[c.table[0, 1].item()] *= 2.0 ** -40
        scale[c.table[0, 4].item()] *= 2.0 ** -20
        codes[c.table[1, 2].item()] = 0
        scale[c.table[1, 2].item()] = 2.0 ** -64
    c.pools[1][1][c.table[0, 2].item()] *= 2.0 ** 40
    c.run()


@pytest.mark.parametrize("n", [1, 61])
def test_far_pages(n):
    """Pages past 2^32 bytes of a pool."""
    Case([200, 17], n, 16, 8, 128, 64, num_pages=(9 << 29) // (8 * 64 * 128)).run()


@pytest.mark.parametrize("n", [1, 7, 61])
def test_same_bits_on_every_call_stream_and_replay(n):
    c = Case([1500, 900], n, 8, 4, 128, 32)
    args = c.args()
    ws = eg.Workspace("cuda")
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


@pytest.mark.parametrize("n", [1, 61])
def test_unmapped_page_sets_status(n):
    c = Case([64, 64], n, 4, 2, 64, 16)
    for bad in (-1, c.pools[0][0].shape[0]):
        args = list(c.args())
        args[5][1, 2] = bad
        c.pools[0][0][0], c.pools[1][0][0] = 0x30, 0x30     # page 0 is read in its place
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        eg.tree_attn_kv8(*args, status=status)
        assert int(status) == -1


def test_refused_by_the_binding():
    c = Case([64, 64], 3, 4, 2, 64, 16)
    names = ("q", "k_pages", "v_pages", "k_scale", "v_scale", "block_table", "kv_len", "k_tree", "v_tree", "mask")
    good = dict(zip(names, c.args()))
    q = good["q"]
    for bad in (dict(q=q.float()), dict(q=q.transpose(1, 2)), dict(q=q[:, :, :3].contiguous()), dict(mask=good["mask"].int()),
                dict(mask=good["mask"][:, :2]), dict(kv_len=good["kv_len"].long()), dict(k_scale=good["k_scale"].double()),
                dict(v_scale=good["v_scale"][:2]), dict(k_tree=good["k_tree"].transpose(1, 2)), dict(v_pages=good["v_pages"].float()),
                dict(block_table=good["block_table"][:1]), dict(scale=0.0), dict(q=q.cpu()), dict(out=q.float())):
        with pytest.raises(eg.EagleError):
            eg.tree_attn_kv8(**{**good, **bad})


@pytest.mark.parametrize("P", [16, 64, 128, 4096])
@pytest.mark.parametrize("n,G,dh", [(61, 8, 64), (49, 8, 128), (200, 2, 64), (333, 1, 128), (150, 1, 64)])
def test_tree_rows_of_many_sizes(n, G, dh, P):
    """Neighbouring nodes' keys and values 2^-8 to 2^8 times apart, over pages
    shorter and longer than a key tile, one tree tile and several.  Within the
    tolerance: a row becomes f16 over a power of two that leaves the largest in
    [2^8, 2^9), so a number is exact unless its bits end below 2^-24, and off by
    at most 2^-25, 2^-33 of the largest (2^-23 where that is 2^10); its weight
    times that is far below 2^-11 A, the prefix alone giving A some tenths."""
    c = Case([300, 77], n, 2 * G, 2, dh, P)
    size = torch.exp2((torch.arange(n) % 17 - 8).float())[:, None]
    c.kt, c.vt = (c.kt.float() * size).bfloat16(), (c.vt.float() * size.flip(0)).bfloat16()
    c.run()


@pytest.mark.parametrize("L", [0, 1, 63, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("dh,P", [(64, 128), (64, 256), (128, 64), (128, 512)])
def test_grouped_heads_over_long_pages(L, dh, P):
    """129 query rows a KV head and more, pages no shorter than a key tile."""
    Case([L, 3 * L // 4 + 1], 43, 6, 2, dh, P).run()
    Case([L, 3 * L // 4 + 1], 129, 2, 2, dh, P).run()


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 1), (1, 40), (3, 2), (61, 1), (61, 8), (65, 1), (100, 2), (130, 4)])
def test_mask_bits_past_the_last_node(n, G, dh, P):
    """Words of all ones are a mask of all nodes: bits that name no node count for nothing."""
    c = Case([70, 0], n, 2 * G, 2, dh, P, keep=torch.ones((2, n, n), dtype=torch.bool))
    args = list(c.args())
    args[9] = torch.full_like(args[9], -1)
    c.check(*eg.tree_attn_kv8(*args))
