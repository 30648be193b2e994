"""Writes into the 8-bit paged cache on the GPU against the oracle.  Numbers
and scales are determined to the bit (the scale is the least power of two
that fits, dividing by it is exact, and one rounding to nearest even follows),
so everything is compared for equality."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv as okv
from oracle import kv8 as okv8

pytestmark = pytest.mark.gpu


def pool(rng, N, Hkv, P, dh):
    """Random finite numbers and scales."""
    codes = rng.integers(0, 256, (N, Hkv, P, dh)).astype(np.uint8)
    codes[(codes & 127) == 127] = 0x30
    return codes, 2.0 ** rng.integers(-9, -3, (N, Hkv)).astype(np.float64)


def on_gpu(codes, scale):
    return torch.from_numpy(codes.copy()).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scale).float().cuda()


def same(t, s, codes, scale):
    np.testing.assert_array_equal(s.double().cpu().numpy(), scale)
    np.testing.assert_array_equal(t.view(torch.uint8).cpu().numpy(), codes)


def place(rng, lens, firsts, P, spare=3):
    """Slots of sequences of `lens` new tokens whose first goes to row firsts[b] of a page."""
    need = [-(-(f + n) // P) for f, n in zip(firsts, lens)]
    order = iter(rng.permutation(sum(need) + spare).tolist())
    slots = []
    for n, f, m in zip(lens, firsts, need):
        pages = [next(order) for _ in range(m)]
        slots += [pages[(f + i) // P] * P + (f + i) % P for i in range(n)]
    return np.array(slots, dtype=np.int64), sum(need) + spare


def append(rng, lens, firsts, Hkv, dh, P, dtype, layout="tokens", spread=3, holes=()):
    slots, N = place(rng, lens, firsts, P)
    T = len(slots)
    x = torch.from_numpy(rng.standard_normal((2, T, Hkv, dh)) * 2.0 ** rng.integers(-spread, spread + 1, (2, T, Hkv, 1))).to(dtype)
    slots[list(holes)] = -1
    ck, sk = pool(rng, N, Hkv, P, dh)
    cv, sv = pool(rng, N, Hkv, P, dh)
    kp, ks = on_gpu(ck, sk)
    vp, vs = on_gpu(cv, sv)
    k, v = x[0].cuda(), x[1].cuda()
    if layout == "heads":                          # [Hkv, T, dh] in memory, as rope writes k_tree
        k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v))
    elif layout == "fused":
        both = torch.cat([k, v], 1)
        k, v = both[:, :Hkv], both[:, Hkv:]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.kv8_append(k, v, torch.from_numpy(slots).int().cuda(), kp, vp, ks, vs, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    okv8.append(x[0].double().numpy(), slots, ck, sk)
    okv8.append(x[1].double().numpy(), slots, cv, sv)
    same(kp, ks, ck, sk)
    same(vp, vs, cv, sv)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_prompts_begin_and_end_inside_pages(P, dtype):
    rng = np.random.default_rng(P)
    append(rng, [1, 2 * P, P + 5, 3], [0, 0, 3, P - 1], 2, 64, P, dtype)
    append(rng, [37, 1, P], [P - 1, P // 2, 1], 3, 128, P, dtype, layout="fused")


@pytest.mark.parametrize("dh", [16, 48, 64, 80, 128, 256, 512])
def test_head_dimensions(dh):
    append(np.random.default_rng(dh), [5, 33], [7, 0], 1, dh, 16, torch.bfloat16)


@pytest.mark.parametrize("layout", ["tokens", "heads", "fused"])
@pytest.mark.parametrize("lens,firsts", [([1], [0]), ([1], [9]), ([1] * 40, list(range(40))), ([300], [10]), ([100, 1, 1, 200], [1, 2, 3, 4])])
def test_layouts_and_lengths(layout, lens, firsts):
    append(np.random.default_rng(len(lens)), lens, [f % 32 for f in firsts], 5, 64, 32, torch.bfloat16, layout)


def test_large_prompt():
    append(np.random.default_rng(4), [5000, 1, 3001], [0, 5, 17], 8, 128, 64, torch.bfloat16)


def test_skipped_tokens_between_sequences():
    rng = np.random.default_rng(5)
    append(rng, [20, 16, 16], [0, 0, 0], 2, 64, 16, torch.bfloat16, holes=[*range(20, 36)])
    append(rng, [4, 4], [0, 3], 2, 64, 16, torch.bfloat16, holes=range(8))            # nothing at all


def test_wide_spread_grows_scales_and_reencodes():
    append(np.random.default_rng(6), [1] * 30, [15] * 30, 4, 64, 16, torch.float32, spread=12)


def test_extremes():
    """Zeros, the clamped scales, the ends of the range, and what is not finite."""
    P, dh, big = 16, 64, 448.0 * 2.0 ** 64
    rng = np.random.default_rng(7)
    ck, sk = pool(rng, 6, 1, P, dh)
    x = np.zeros((6, 1, dh), dtype=np.float32)
    x[1, 0, 5] = 448.0                              # exactly the largest at scale 1
    x[2, 0, 5] = np.nextafter(np.float32(448), np.float32(500))
    x[3, 0, 5], x[3, 0, 6] = 2.0 ** -80, -2.0 ** -72  # below the least scale's numbers, and its half step
    x[4, 0, 5], x[4, 0, 6] = -big, 1.0
    x[5, 0, 0] = -0.0
    slots = np.arange(6) * P
    kp, ks = on_gpu(ck, sk)
    vp, vs = on_gpu(ck, sk)
    t = torch.from_numpy(x).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.kv8_append(t, t, torch.from_numpy(slots).int().cuda(), kp, vp, ks, vs, status=status)
    okv8.append(x.astype(np.float64), slots, ck, sk)
    assert int(status) == 0
    same(kp, ks, ck, sk)
    x[1, 0, 7], x[2, 0, 7], x[4, 0, 7] = math.nan, -math.inf, 2 * big
    t = torch.from_numpy(x).cuda()
    eg.kv8_append(t, t, torch.from_numpy(slots).int().cuda(), kp, vp, ks, vs, status=status)
    okv8.append(x.astype(np.float64), slots, ck, sk)
    assert int(status) == -1
    same(kp, ks, ck, sk)


def test_broken_sequences_and_slots_past_the_pool():
    P, N = 16, 4
    rng = np.random.default_rng(8)
    ck, sk = pool(rng, N, 2, P, 64)
    x = torch.randn((6, 2, 64))
    kp, ks = on_gpu(ck, sk)
    vp, vs = on_gpu(ck, sk)
    slots = np.array([3, 4, 9, N * P, 2 * P, 2 ** 31 - 1])            # 9 does not follow 4; two slots past the pool
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.kv8_append(x.cuda(), x.cuda(), torch.from_numpy(slots).int().cuda(), kp, vp, ks, vs, status=status)
    assert int(status) == -1
    okv8.append(x.double().numpy(), np.array([3, 4, -1, -1, 2 * P, -1]), ck, sk)
    same(kp, ks, ck, sk)
    same(vp, vs, ck, sk)


def test_far_pages():
    """Offsets past 2^32 bytes."""
    Hkv, P, dh = 8, 64, 128
    N = (5 << 30) // (Hkv * P * dh)
    kp = torch.zeros((N, Hkv, P, dh), dtype=torch.uint8, device="cuda")
    ks = torch.ones((N, Hkv), device="cuda")
    vp, vs = torch.zeros_like(kp), torch.ones_like(ks)
    x = torch.randn((3, Hkv, dh)).to(torch.bfloat16)
    slots = torch.tensor([(N - 1) * P, (N - 1) * P + 1, (N - 2) * P], dtype=torch.int32)
    eg.kv8_append(x.cuda(), x.cuda(), slots.cuda(), kp, vp, ks, vs)
    codes, scale = np.zeros((2, Hkv, P, dh), np.uint8), np.ones((2, Hkv))
    okv8.append(x.double().numpy(), [P, P + 1, 0], codes, scale)
    for p, s in ((kp, ks), (vp, vs)):
        same(p[-2:], s[-2:], codes, scale)
        assert not p[:-2].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,Hkv,dh,P,D", [(1, 9, 1, 64, 16, 1), (4, 20, 3, 64, 16, 6), (3, 61, 40, 128, 64, 7), (2, 128, 2, 128, 16, 64),
                                            (70, 8, 8, 64, 32, 5)])
def test_commit(B, n, Hkv, dh, P, D, dtype):
    rng = np.random.default_rng(B * n)
    mp = 200 // P + 6
    N = B * mp + 3
    kv_len = rng.integers(1, 200, B)
    kv_len[0] = P                                   # the first accepted row opens a page
    acc = rng.integers(0, D + 1, B)
    acc[0] = D
    path = np.full((B, D + 1), -1)
    for b in range(B):
        path[b, 0] = 0
        path[b, 1:acc[b] + 1] = rng.permutation(np.arange(1, n))[:acc[b]] if acc[b] < n else rng.integers(1, n, acc[b])
    table = rng.permutation(N)[:B * mp].reshape(B, mp)
    tree = torch.from_numpy(rng.standard_normal((2, B, Hkv, n, dh)) * 2.0 ** rng.integers(-2, 3, (2, B, Hkv, n, 1))).to(dtype)
    ck, sk = pool(rng, N, Hkv, P, dh)
    cv, sv = pool(rng, N, Hkv, P, dh)
    kp, ks = on_gpu(ck, sk)
    vp, vs = on_gpu(cv, sv)
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x)).int().cuda()
    kl = i32(kv_len)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = eg.kv8_commit(tree[0].cuda(), tree[1].cuda(), i32(acc), i32(path), kp, vp, ks, vs, kl, i32(table), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert (kl.cpu().numpy() == kv_len + acc).all()
    assert (slots.cpu().numpy() == okv.slot_mapping(path, acc, kv_len, n)).all()
    for b in range(B):
        pos = kv_len[b] + np.arange(acc[b])
        where = table[b, pos // P] * P + pos % P
        nodes = path[b, 1:acc[b] + 1]
        for src, codes, scale in ((tree[0], ck, sk), (tree[1], cv, sv)):
            okv8.append(src[b].double().numpy()[:, nodes].transpose(1, 0, 2), where, codes, scale)
    same(kp, ks, ck, sk)
    same(vp, vs, cv, sv)


@pytest.mark.parametrize("fault", ["node 0", "node n", "accept", "length", "page", "full"])
def test_a_refused_commit_leaves_its_sequence_alone(fault):
    B, n, Hkv, dh, P, D, mp = 2, 6, 2, 64, 16, 3, 4
    rng = np.random.default_rng(11)
    ck, sk = pool(rng, 9, Hkv, P, dh)
    kp, ks = on_gpu(ck, sk)
    vp, vs = on_gpu(ck, sk)
    kv_len, acc = np.array([20, 20]), np.array([2, 2])
    path = np.array([[0, 1, 2, -1]] * 2)
    table = np.arange(8).reshape(2, 4)
    if fault == "node 0":
        path[0, 2] = 0
    elif fault == "node n":
        path[0, 1] = n
    elif fault == "accept":
        acc[0] = 4
    elif fault == "length":
        kv_len[0] = 0
    elif fault == "page":
        table[0, 1] = 9
    elif fault == "full":
        kv_len[0] = mp * P - 1
    x = torch.from_numpy(rng.standard_normal((B, Hkv, n, dh))).float()
    i32 = lambda t: torch.from_numpy(t).int().cuda()
    kl, status = i32(kv_len), torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.kv8_commit(x.cuda(), x.cuda(), i32(acc), i32(path), kp, vp, ks, vs, kl, i32(table), status=status)
    assert int(status) == -1
    assert kl.tolist() == [kv_len[0], 22]
    okv8.append(x[1].double().numpy()[:, [1, 2]].transpose(1, 0, 2), [table[1, 1] * P + 4, table[1, 1] * P + 5], ck, sk)
    same(kp, ks, ck, sk)


def test_captured_appends_follow_the_slots():
    rng = np.random.default_rng(12)
    ck, sk = pool(rng, 5, 2, 16, 64)
    kp, ks = on_gpu(ck, sk)
    vp, vs = on_gpu(ck, sk)
    x = torch.zeros((4, 2, 64), device="cuda")
    slots = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    eg.kv8_append(x, x, slots, kp, vp, ks, vs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eg.kv8_append(x, x, slots, kp, vp, ks, vs)
    for step in range(18):                          # single tokens through a page's end; one request is padding
        new = rng.standard_normal((4, 2, 64)).astype(np.float32) * (1 + step)
        at = np.array([step if step < 16 else 16 * 3 + step - 16, 32 + (step % 16) if step < 16 else -1, -1, -1])
        x.copy_(torch.from_numpy(new))
        slots.copy_(torch.from_numpy(at))
        g.replay()
        okv8.append(new.astype(np.float64), at, ck, sk)
    same(kp, ks, ck, sk)
    same(vp, vs, ck, sk)


def test_refused_by_the_binding():
    kp = torch.zeros((4, 2, 16, 64), dtype=torch.uint8, device="cuda")
    s = torch.ones((4, 2), device="cuda")
    k = torch.zeros((3, 2, 64), device="cuda")
    slots = torch.zeros(3, dtype=torch.int32, device="cuda")
    good = dict(k=k, v=k, slot_map=slots, k_pages=kp, v_pages=kp, k_scale=s, v_scale=s)
    for bad in (dict(v=k.bfloat16()), dict(v=k[:2]), dict(slot_map=slots.long()), dict(slot_map=slots[:2]), dict(k_scale=s[:3]),
                dict(v_pages=kp.view(torch.int8)), dict(k=k.half(), v=k.half()), dict(k=k[..., :32], v=k[..., :32]),
                dict(k=k[:1].expand(3, 2, 64), v=k[:1].expand(3, 2, 64)), dict(k_pages=kp.transpose(1, 2))):
        with pytest.raises(eg.EagleError):
            eg.kv8_append(**{**good, **bad})
