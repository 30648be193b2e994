"""Attention over the 8-bit cache where one value is far larger than the others: an
outlier column sets its page's scale, and the weights of every other key are
rounded beside it.  The bound is the one that the header states, 2^-31 |v_k| 2^-e_k
max_j (p_j 2^e_j) for key k, element by element, so the columns without the outlier
are held to what the small pages leave them."""
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from test_gpu_kv8_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,G,dh,P", [(1, 8, 128, 64), (5, 2, 64, 16), (20, 1, 128, 32), (61, 1, 128, 16), (61, 2, 64, 64), (61, 2, 128, 16),
                                      (61, 8, 64, 64), (61, 8, 128, 32), (61, 8, 64, 128), (61, 8, 128, 64), (200, 2, 64, 256)])
@pytest.mark.parametrize("bits", [4, 12, 20, 26])
def test_an_outlier_column_on_one_page(n, G, dh, P, bits):
    c = Case([4 * P, 3 * P + 5], n, 2 * G, 2, dh, P, seed=bits)
    codes, scale = c.pools[1]
    for b, at in ((0, 2), (1, 0)):
        page = int(c.table[b, at])
        codes[page] = 0
        codes[page, :, ::3, 7] = 0x7e               # 448, in every third row
        scale[page] *= 2.0 ** bits
    c.run()


@pytest.mark.parametrize("n,G,dh,P", [(1, 8, 128, 64), (20, 1, 64, 32), (61, 1, 128, 16), (61, 2, 64, 64), (61, 8, 64, 64), (61, 8, 64, 128),
                                      (61, 8, 128, 64)])
def test_value_scales_2_to_the_100_apart_leave_lse_alone(n, G, dh, P):
    """lse does not depend on the values: pages of 2^50 and 2^-50, and tree values of
    2^-45, against the same keys with one scale, to the sums' rounding: a weight
    that float32 cannot hold beside the largest is below 2^-32 of the sum."""
    c = Case([4 * P, 3 * P + 5], n, 2 * G, 2, dh, P, seed=9)
    scale = c.pools[1][1]
    scale.fill_(1.0)
    c.vt = torch.ones_like(c.vt)
    _, want = eg.tree_attn_kv8(*c.args())
    used = c.table[c.table >= 0].long().cuda()
    scale[used] = 2.0 ** -50
    scale[used[::3]] = 2.0 ** 50
    c.vt = c.vt * 2.0 ** -45
    out, lse = eg.tree_attn_kv8(*c.args())
    # both are within (L + n) 2^-23 + 2^-20 and 2^-22 |lse| of the truth: ex2 and sums of one sign
    tol = 2 * ((4 * P + n) * 2.0 ** -23 + 2.0 ** -20) + 2.0 ** -21 * want.abs()
    assert ((lse - want).abs() <= tol).all() and torch.isfinite(out).all()
