"""Attention over lists of one or two sequences with many rows: the keys of a list are
split over CTAs for the longest list there can be, however short it turns out."""
import pytest
import torch

from test_gpu_kv8_pages_attn import Listed

pytestmark = pytest.mark.gpu


def spread(c, top, how):
    """The lists of c anew: the same pages for all nodes, pages of a node's own, or none but one node's."""
    B, n, Hkv, _ = c.sel.shape
    c.sel = torch.full_like(c.sel, -1)
    for b, L in enumerate(c.kv_len):
        live = -(-L // c.P)
        if how == "one":
            k = min(top, live)
            c.sel[b, n // 2, :, :k] = torch.arange(live - k, live, dtype=torch.int32)
            continue
        for i in range(n):
            pages = sorted({(p if how == "agree" else i * top + p) % live for p in range(top)}) if live else []
            c.sel[b, i, :, :len(pages)] = torch.tensor(pages, dtype=torch.int32)


@pytest.mark.parametrize("how", ["agree", "apart", "one"])
@pytest.mark.parametrize("n,Hq,Hkv,dh,P,top", [(49, 8, 1, 128, 16, 4), (61, 4, 4, 128, 16, 4), (70, 2, 2, 64, 16, 8), (256, 2, 2, 64, 16, 8),
                                               (33, 1, 1, 64, 256, 1), (40, 4, 2, 128, 128, 2)])
def test_few_sequences(n, Hq, Hkv, dh, P, top, how):
    c = Listed([n * top * P // 2 + 5], n, Hq, Hkv, dh, P, top)
    spread(c, top, how)
    c.run()
    c = Listed([1, 40], n, Hq, Hkv, dh, P, top, extra_pages=300)
    spread(c, top, how)
    c.run()
