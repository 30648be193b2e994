"""Attention over the 8-bit cache with queries and keys near the ends of their
ranges: products that are 0 stay 0, whatever the factors beside them."""
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg

pytestmark = pytest.mark.gpu

# few rows, one M-tile (64 and 128 rows), two M-tiles with scales of groups and of tiles
SHAPES = [(3, 2, 64, 16), (20, 1, 128, 64), (61, 1, 128, 16), (61, 2, 128, 64), (61, 2, 64, 16), (61, 8, 64, 32), (61, 8, 64, 128),
          (61, 8, 128, 16), (61, 8, 128, 64)]


@pytest.mark.parametrize("n,G,dh,P", SHAPES)
@pytest.mark.parametrize("q_exp,ke,kt_exp", [(100, 64, 100), (120, 0, 119), (-100, -64, -90), (0, 64, 0)])
def test_orthogonal_queries_and_keys(n, G, dh, P, q_exp, ke, kt_exp):
    """Queries along one column, keys along others, values of +-1 and +-2: every
    score is 0 exactly, so a row is the mean of the values that it attends to, lse
    the logarithm of their number."""
    B, Hkv, L = 2, 2, 150
    pages = -(-L // P)
    g = torch.Generator().manual_seed(n)
    kp = torch.zeros((B * pages, Hkv, P, dh))
    kp[..., 1 + dh // 2:] = torch.tensor([448.0, -256.0, 1.0, -0.5])[torch.randint(0, 4, (B * pages, Hkv, P, dh - 1 - dh // 2), generator=g)]
    vp = torch.tensor([1.0, -1.0, 2.0, -2.0])[torch.randint(0, 4, (B * pages, Hkv, P, dh), generator=g)]
    q = torch.zeros((B, n, Hkv * G, dh))
    q[..., 3] = 2.0 ** q_exp
    kt = torch.zeros((B, Hkv, n, dh))
    kt[..., 4:] = 2.0 ** kt_exp
    vt = torch.tensor([1.0, -1.0, 2.0, -2.0])[torch.randint(0, 4, (B, Hkv, n, dh), generator=g)]
    bf = lambda t: t.to(torch.bfloat16).cuda()
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    mask = eg.tree_mask(torch.tensor([[-1] + list(range(n - 1))] * B, dtype=torch.int32, device="cuda"))
    ks = torch.full((B * pages, Hkv), 2.0 ** ke, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = eg.tree_attn_kv8(bf(q), kp.cuda().to(torch.float8_e4m3fn), vp.cuda().to(torch.float8_e4m3fn), ks, torch.ones_like(ks),
                                table, torch.full((B,), L, dtype=torch.int32, device="cuda"), bf(kt), bf(vt), mask, status=status)
    assert int(status) == 0
    V = vp.double().view(B, pages, Hkv, P, dh).transpose(1, 2).reshape(B, Hkv, pages * P, dh)[:, :, :L]
    total = V.sum(2)[:, :, None] + vt.double().cumsum(2)                       # a chain: node i and those before it
    count = L + 1.0 + torch.arange(n, dtype=torch.float64)
    want = (total / count[:, None]).transpose(1, 2).repeat_interleave(G, 2).cuda()
    # weights are one power of two and exact; the sums (whole numbers) too; 1 / l, the product and bf16 round
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -22).all()
    assert ((lse.double() - count.log().cuda()[None, :, None]).abs() <= 2.0 ** -21 * 6).all()


def test_a_workspace_of_another_device_is_refused():
    n, dh, P = 61, 128, 64
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")
    pool, scale, table = z(64, 8, P, dh, dtype=torch.uint8), z(64, 8, dtype=torch.float32), z(1, 64, dtype=torch.int32)
    args = (z(1, n, 8, dh), pool, pool, scale, scale, table, z(1, dtype=torch.int32), z(1, 8, n, dh), z(1, 8, n, dh),
            z(1, n, 1, dtype=torch.int64))
    with pytest.raises(eg.EagleError, match="workspace"):
        eg.tree_attn_kv8(*args, workspace=eg.Workspace("cpu"))
