"""grow() leaves every request's bounds true for the pages as they are: after rows
that nobody counted have changed a page's scale, and after a length was set back."""
import numpy as np
import pytest
import torch

from oracle import kv8 as okv8
from oracle import select as oselect
from tree_speculative_decoding_eagle_gb300.cache import KV8Cache

pytestmark = pytest.mark.gpu
B, HKV, DH, P, LAYERS = 3, 2, 64, 16, 2


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(lens, seed):
    g = torch.Generator().manual_seed(seed)
    cache = KV8Cache(B, HKV, DH, P, 40, 8, layers=LAYERS, bounds=True)
    add(cache, lens, g, 1.0)
    cache.grow(i32(lens))
    return cache, g


def add(cache, lens, g, size):
    """Rows of N(0, size^2) for lens[b] more tokens, appended in every layer and not counted."""
    slots = torch.empty(sum(lens), dtype=torch.int32, device="cuda")
    cache.reserve(i32(lens), slots)
    for layer in range(LAYERS):
        k, v = ((torch.randn((sum(lens), HKV, DH), generator=g) * size).bfloat16().cuda() for _ in range(2))
        cache.append(layer, k, v, slots)


def check(cache):
    table, lens = cache.block_table.tolist(), cache.kv_len.tolist()
    for layer in range(LAYERS):
        codes, bounds = (okv8.decode(t[layer].view(torch.uint8).cpu().numpy()) for t in (cache.k_pages, cache.k_bounds))
        for b in range(B):
            for p in range(-(-lens[b] // P)):
                page, rows = table[b][p], min(P, lens[b] - p * P)
                for g in range(HKV):
                    np.testing.assert_array_equal(bounds[page, g], np.stack(oselect.bounds(codes[page, g, :rows])))
    assert int(cache.status) == 0


@pytest.mark.parametrize("lens", [[21, 1, 40], [16, 47, 15]])
def test_rows_that_are_not_counted_may_change_a_page_s_scale(lens):
    cache, g = filled(lens, 1)
    check(cache)
    before = [s.clone() for s in cache.k_scale]
    add(cache, [5, 5, 5], g, 60.0)
    assert any(not torch.equal(s, t) for s, t in zip(before, cache.k_scale))
    cache.grow(i32([0, 0, 2]))                     # two of the first tokens were wanted after all
    check(cache)
    cache.grow(0)
    check(cache)


@pytest.mark.parametrize("to", [[19, 1, 33], [16, 17, 0], [0, 31, 48]])
def test_a_length_set_back(to):
    cache, g = filled([40, 33, 48], 2)
    cache.kv_len.copy_(i32(to))
    cache.trim()
    cache.grow(0)
    check(cache)
    add(cache, [3, 17, 1], g, 0.1)
    cache.grow(i32([3, 17, 1]))
    check(cache)


def test_a_step_that_accepts_nothing():
    """commit() without the root and with no node accepted, after uncounted rows."""
    cache, g = filled([21, 1, 40], 3)
    add(cache, [2, 2, 2], g, 60.0)
    trees = [torch.zeros((B, HKV, 3, DH), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
    cache.commit(trees, trees, i32([0, 0, 0]), i32([[0, -1, -1]] * B))
    check(cache)
