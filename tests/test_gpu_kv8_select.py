"""eagle_kv8_select on the GPU: scores and pages equal the oracle's.  Every score is
exact in float32 (a sum of at most 128 multiples of 1/2 up to 128 * 448, times a
power of two), so nothing is allowed to differ."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8, select

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def halves(rng, shape):
    """e4m3 codes that are multiples of 1/2."""
    ok = np.array([c for c in range(256) if (c & 127) != 127 and 2 * kv8.TABLE[c] == np.rint(2 * kv8.TABLE[c])], dtype=np.uint8)
    return ok[rng.integers(0, len(ok), shape)]


class Case:
    def __init__(self, kv, n, Hq, Hkv, dh, P, seed=0, extra=1, spread=2):
        rng = np.random.default_rng(seed)
        B = len(kv)
        self.kv, self.P = kv, P
        self.mp = max(1, max(-(-k // P) for k in kv)) + extra
        self.N = B * self.mp + 2
        self.codes = np.sort(kv8.decode(halves(rng, (self.N, Hkv, 2, dh))), axis=2)
        self.codes = kv8.encode(self.codes)
        self.scale = (2.0 ** rng.integers(-spread, spread + 1, (self.N, Hkv))).astype(np.float32)
        perm = rng.permutation(self.N)[:B * self.mp].reshape(B, self.mp)
        self.table = np.where(np.arange(self.mp)[None] < -(-np.array(kv)[:, None] // P), perm, -1).astype(np.int32)
        self.q = torch.from_numpy(rng.standard_normal((B, n, Hq, dh)) * 2.0 ** rng.integers(-3, 4, (B, n, Hq, 1))).to(torch.bfloat16)

    def call(self, top, first=1, last=1, **kw):
        self.status = i32([0])
        self.score = torch.full((*self.q.shape[:2], self.codes.shape[1], top), 77.0, device="cuda")
        sel = torch.full(self.score.shape, 77, dtype=torch.int32, device="cuda")
        got = eg.kv8_select(self.q.cuda(), torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scale).cuda(),
                            torch.from_numpy(self.table).cuda(), i32(self.kv), self.P, top, first, last, out=sel, score=self.score,
                            status=self.status, **kw)
        assert got is sel
        torch.cuda.synchronize()
        return sel.cpu().numpy(), self.score.cpu().numpy().astype(np.float64)

    def check(self, top, first=1, last=1, **kw):
        sel, score = self.call(top, first, last, **kw)
        assert int(self.status) == 0
        B, n, Hq, dh = self.q.shape
        Hkv = self.codes.shape[1]
        q = self.q.double().numpy().reshape(B, n, Hkv, Hq // Hkv, dh)
        for b, L in enumerate(self.kv):
            pages = self.table[b, :-(-L // self.P)]
            box = kv8.decode(self.codes[pages])
            for i in range(n):
                for g in range(Hkv):
                    s = select.scores(q[b, i, g], box[:, g, 0], box[:, g, 1], self.scale[pages, g].astype(np.float64))
                    want = select.choose(s, top, first, last)
                    pad = top - len(want)
                    assert sel[b, i, g].tolist() == want + [-1] * pad, (b, i, g)
                    assert score[b, i, g].tolist() == s[want].tolist() + [-np.inf] * pad, (b, i, g)
        return sel


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (4, 2), (3, 1), (5, 1), (8, 1), (10, 2), (16, 1), (9, 1), (20, 1), (64, 2), (32, 1)])
@pytest.mark.parametrize("n", [1, 2, 5, 19])
def test_heads_and_nodes(dh, Hq, Hkv, n):
    Case([70, 0, 331, 16], n, Hq, Hkv, dh, 16, seed=n).check(6)


@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("top,first,last", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (2, 1, 1), (5, 0, 3), (5, 5, 0), (5, 0, 5), (7, 2, 2), (200, 3, 4)])
def test_choices(P, top, first, last):
    lens = [0, 1, P - 1, P, P + 1, 2 * P, 5 * P, 5 * P + 1, 9 * P - 1, 33 * P]
    Case(lens, 2, 4, 2, 64, P, seed=P).check(top, first, last)


@pytest.mark.parametrize("pages", [511, 512, 513, 2047, 2048, 2049, 5000, 16384])
def test_many_pages(pages):
    """Each form of the choice, at and beside the sizes where it changes."""
    Case([pages * 16, 40 * 16, pages * 16 - 15], 2, 4, 2, 64, 16, seed=pages, extra=0).check(37)
    if pages < 3000:
        Case([pages * 16 - 7], 1, 8, 1, 128, 16, seed=pages, extra=0).check(min(pages - 1, 700), 3, 2)


def test_many_sequences():
    rng = np.random.default_rng(0)
    Case(rng.integers(0, 3000, 70).tolist(), 1, 16, 8, 128, 32).check(9)
    Case(rng.integers(0, 3000, 9).tolist(), 49, 8, 1, 64, 16).check(9)
    Case([500, 90], 200, 4, 2, 64, 16).check(4)


def test_ties_go_to_the_lower_pages():
    c = Case([40 * 16], 3, 4, 2, 64, 16)
    c.q[:, 0] = 0                                  # every score 0
    c.codes[:] = c.codes[:1]                       # every page alike, but for the scale
    c.check(7, 0, 0)
    sel = c.check(7, 1, 1)
    assert sel[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, 39]
    c = Case([3000 * 16], 1, 1, 1, 64, 16, extra=0)
    c.codes[c.table[0, 100:]] = c.codes[c.table[0, 50]]
    c.scale[:] = 1
    c.check(60, 0, 0)
    c.check(2000, 0, 0)


@pytest.mark.parametrize("n", [3, 49])
def test_zeros_of_either_sign_are_ties(n):
    """Products of a zero query, or with zero bounds, are zeros of both signs."""
    c = Case([40 * 16], n, 4, 2, 64, 16)
    number = np.random.default_rng(3).integers(1, 9, c.codes.shape) / 2.0
    number[c.table[0, ::2]] *= -1                  # pages of negative bounds alone, and of positive ones alone
    c.codes = kv8.encode(np.sort(number, axis=2))
    c.q[:, 0] = 0
    c.q[:, 1] = -0.0
    c.q[:, 2, :, 1:] = 0                           # one column counts; its bounds are zeros of either sign
    c.codes[..., 0] = np.where(np.arange(c.N) % 2, 0x80, 0)[:, None, None]
    sel = c.check(7, 0, 0)
    for i in range(3):
        assert sel[0, i, 0].tolist() == list(range(7))


def test_the_largest_sums_are_exact():
    """All columns at the edge: sums up to 128 * 128 * 448, neighbours half a unit apart."""
    for dh in (64, 128):
        c = Case([64 * 16], 1, 1, 1, dh, 16, spread=0)
        rng = np.random.default_rng(dh)
        c.q[:] = 127.5                             # whole number 128
        c.codes[:] = kv8.encode(np.full(c.codes.shape, 448.0))
        small = kv8.encode(np.arange(64) * 0.5)[rng.permutation(64)]
        c.codes[c.table[0, :64], 0, 1, 5] = small  # one column tells the pages apart
        c.q[..., 5] = 1.0
        c.check(9, 0, 0)
        c.q[..., 1::2] *= -1
        c.codes[..., 0, :] = kv8.encode(np.full(c.codes[..., 0, :].shape, -448.0))
        c.check(9, 0, 0)


def test_the_largest_sums_are_exact_for_many_rows():
    """The same on the tiles for many rows: odd multiples of half a unit at the top of the range."""
    for dh in (64, 128):
        c = Case([300 * 16], 40, 4, 1, dh, 16, spread=0)
        rng = np.random.default_rng(dh)
        c.q[:] = 127.5
        c.q[:, 1::2, :, 1::2] *= -1
        c.q[..., 7] = 1.0
        c.codes[..., 0, :] = kv8.encode(np.full(c.codes[..., 0, :].shape, -448.0))
        c.codes[..., 1, :] = kv8.encode(np.full(c.codes[..., 1, :].shape, 448.0))
        c.codes[..., 1, 7] = kv8.encode(rng.integers(0, 8, c.codes[..., 1, 7].shape) * 0.5)
        c.check(9, 0, 0)
        c.check(299, 0, 0)


def test_magnitudes_and_odd_queries():
    c = Case([50 * 16], 8, 4, 2, 64, 16, spread=64)
    c.scale[0], c.scale[1] = 2.0 ** 64, 2.0 ** -64
    for i, f in enumerate((2.0 ** 60, 2.0 ** -60, 2.0 ** 120, 2.0 ** -120, 2.0 ** 38, 2.0 ** -27)):
        c.q[:, i] = (c.q[:, i].double() * f).to(torch.bfloat16)
    c.q[0, 6, 0, 3], c.q[0, 6, 1, 4], c.q[0, 7, 2, 5] = float("inf"), float("-inf"), float("nan")
    c.check(9)
    c.q[:] = float("nan")
    c.check(9)


def test_scales_are_read_as_powers_of_two():
    c = Case([50 * 16], 2, 4, 2, 64, 16)
    want = c.check(9)
    c.scale *= np.random.default_rng(0).uniform(1, 1.99, c.scale.shape).astype(np.float32)
    assert (c.call(9)[0] == want).all()


def test_a_query_selects_the_same_alone_and_in_any_batch():
    c = Case([700, 1203, 31], 21, 10, 2, 128, 16)
    whole, score = c.call(8)
    for b, i in ((0, 0), (1, 20), (1, 7), (2, 3)):
        one = Case([1], 1, 10, 2, 128, 16)
        one.kv, one.codes, one.scale, one.table, one.q = [c.kv[b]], c.codes, c.scale, c.table[b:b + 1], c.q[b:b + 1, i:i + 1].contiguous()
        sel, s = one.call(8)
        assert (sel[0, 0] == whole[b, i]).all() and (s[0, 0] == score[b, i]).all()


def test_scores_past_31_bits_of_offset():
    """4096 nodes, 40 KV heads, 16384 pages: 2.7e9 scores in the workspace."""
    g = torch.Generator(device="cuda").manual_seed(0)
    Hkv, pages, dh = 40, 16384, 64
    q = torch.randn(1, 4096, Hkv, dh, generator=g, device="cuda").to(torch.bfloat16)
    numbers = torch.randint(-40, 41, (pages, Hkv, 2, dh), generator=g, device="cuda").float() / 2
    bounds = torch.sort(numbers, dim=2).values.to(torch.float8_e4m3fn)
    scale = torch.ones(pages, Hkv, device="cuda")
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    kv = i32([pages * 16 - 3])
    sel = eg.kv8_select(q, bounds, scale, table, kv, 16, 7)
    for i in (0, 1, 2047, 3277, 4094, 4095):
        one = eg.kv8_select(q[:, i:i + 1].contiguous(), bounds, scale, table, kv, 16, 7)
        assert torch.equal(one[0, 0], sel[0, i]), i
    torch.cuda.empty_cache()


def test_the_most_sequences():
    """65535 sequences of a KV head, with few rows and with many."""
    g = torch.Generator(device="cuda").manual_seed(1)
    B, dh, N = 65535, 64, 300
    bounds = torch.sort(torch.randint(-40, 41, (N, 1, 2, dh), generator=g, device="cuda").float() / 2, dim=2).values.to(torch.float8_e4m3fn)
    scale = torch.ones(N, 1, device="cuda")
    table = torch.randint(0, N, (B, 9), generator=g, device="cuda", dtype=torch.int32)
    kv = torch.randint(0, 9 * 16 + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    for n in (1, 33):
        q = torch.randn(B, n, 1, dh, generator=g, device="cuda").to(torch.bfloat16)
        sel = eg.kv8_select(q, bounds, scale, table, kv, 16, 3)
        for part in (slice(0, 50), slice(65485, 65535)):
            assert torch.equal(eg.kv8_select(q[part].contiguous(), bounds, scale, table[part].contiguous(), kv[part].contiguous(), 16, 3), sel[part])


def test_page_numbers_outside_the_pool():
    """Page 0's bounds are read in their place; entries past the prefix are not looked at."""
    c = Case([40 * 16, 90], 2, 4, 2, 64, 16)
    c.table[0, 5], c.table[0, 6] = -3, c.N
    sel, score = c.call(9)
    assert int(c.status) == -1
    c.table[0, 5] = c.table[0, 6] = 0
    want, want_score = c.call(9)
    assert int(c.status) == 0 and (sel == want).all() and (score == want_score).all()
    c.kv = [10 ** 9, 90]                           # clamped to the table
    c.table[0] = np.where(c.table[0] < 0, 1, c.table[0])
    assert c.call(c.mp + 3)[0][0, 0, 0].tolist() == list(range(c.mp)) + [-1] * 3


def test_nan_bounds_stay_in_range():
    c = Case([40 * 16], 3, 4, 2, 64, 16)
    c.codes[:, :, :, 3] = 0x7f
    c.codes[:, :, :, 4] = 0xff
    sel, _ = c.call(9)
    assert (sel >= 0).all() and (sel < 40).all() and (np.diff(sel, axis=-1) > 0).all()


def test_without_scores_on_a_stream_and_captured():
    c = Case([700, 1203], 5, 10, 2, 128, 16)
    want, _ = c.call(8)
    a = (c.q.cuda(), torch.from_numpy(c.codes).cuda(), torch.from_numpy(c.scale).cuda(), torch.from_numpy(c.table).cuda(), i32(c.kv), 16, 8)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = eg.kv8_select(*a, stream=s)
    s.synchronize()
    assert (got.cpu().numpy() == want).all()
    ws, out = eg.Workspace("cuda"), torch.zeros_like(got)
    eg.kv8_select(*a, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.kv8_select(*a, out=out, workspace=ws)
    a[4].fill_(333)
    graph.replay()
    fresh = eg.kv8_select(*a)
    torch.cuda.synchronize()
    assert torch.equal(out, fresh) and not torch.equal(out, got)


def test_binding_refuses():
    c = Case([70], 2, 4, 2, 64, 16)
    q, codes, scale, table, kv = c.q.cuda(), torch.from_numpy(c.codes).cuda(), torch.from_numpy(c.scale).cuda(), torch.from_numpy(c.table).cuda(), i32([70])
    for bad in ((q.float(), codes, scale, table, kv), (q, codes.float(), scale, table, kv), (q, codes[:-1], scale, table, kv),
                (q, codes, scale.double(), table, kv), (q, codes, scale, table.long(), kv), (q, codes, scale, table, kv.cpu()),
                (q.transpose(1, 2), codes, scale, table, kv)):
        with pytest.raises(eg.EagleError):
            eg.kv8_select(*bad, 16, 4)
    for top, first, last in ((0, 0, 0), (2, 2, 1), (4, -1, 1)):
        with pytest.raises((eg.EagleError, RuntimeError)):
            eg.kv8_select(q, codes, scale, table, kv, 16, top, first, last)
