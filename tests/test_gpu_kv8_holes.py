"""Appends whose slot_map interrupts a page: what comes before the interruption is
written, what comes after it is skipped and reported, and every other page is as
the oracle has it, to the bit."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8 as okv8

pytestmark = pytest.mark.gpu
dh = 64


def check(slots, written, H, P, N, dtype, code):
    rng = np.random.default_rng(len(slots))
    x = torch.from_numpy(rng.standard_normal((2, len(slots), H, dh)) * 2.0 ** rng.integers(-3, 4, (2, len(slots), H, 1))).to(dtype)
    codes = [rng.integers(0, 0x70, (N, H, P, dh)).astype(np.uint8) for _ in range(2)]
    scale = [2.0 ** rng.integers(-9, -3, (N, H)).astype(np.float64) for _ in range(2)]
    gpu = [torch.from_numpy(c.copy()).cuda() for c in codes]
    gscale = [torch.from_numpy(s).float().cuda() for s in scale]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.kv8_append(x[0].cuda(), x[1].cuda(), torch.from_numpy(np.asarray(slots)).int().cuda(), *gpu, *gscale, status=status)
    assert int(status) == code
    for i in range(2):
        okv8.append(x[i].double().numpy(), np.where(written, slots, -1), codes[i], scale[i])
        np.testing.assert_array_equal(gscale[i].double().cpu().numpy(), scale[i])
        np.testing.assert_array_equal(gpu[i].cpu().numpy(), codes[i])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hole", [1, 5, 31, 32, 33, 64, 100, 1000, 1024])
@pytest.mark.parametrize("H,P,others", [(1, 16, 0), (2, 64, 7), (8, 16, 3000)])
def test_a_hole_inside_a_page(H, P, others, hole, dtype):
    """Seven tokens, `hole` skipped ones (one of them past the pool), the page's
    next rows, and the page after it; `others` tokens of other pages before."""
    pages = -(-others // P)
    N = pages + 4
    lead = list(range(2 * P + P // 2, 2 * P + P // 2 + 7))
    gap = [-1] * hole
    if hole > 2:
        gap[1] = N * P
    after = list(range(2 * P + P // 2 + 7, 2 * P + P // 2 + 8)) + list(range(3 * P, 3 * P + 5))
    front = [(4 + i // P) * P + i % P for i in range(others)]
    slots = np.array(front + lead + gap + after, dtype=np.int64)
    written = (slots >= 0) & (slots < N * P)
    written[len(front) + len(lead) + hole] = False
    check(slots, written, H, P, N, dtype, -1)


@pytest.mark.parametrize("H,others", [(2, 0), (8, 3000)])
def test_holes_between_sequences_are_as_before(H, others):
    """Padding after each of several requests, one of which goes on inside a page
    that is its own: nothing is refused."""
    P = 16
    N = 20 + -(-others // P)
    slots = [(20 + i // P) * P + i % P for i in range(others)]
    for r, (first, n) in enumerate([(0, 20), (5, 3), (15, 1), (9, 30), (0, 1), (3, 4)]):
        slots += [(3 * r) * P + first + i for i in range(n)] + [-1] * [40, 1, 700, 0, 33, 2000][r]
    slots = np.array(slots + [19 * P + 1])
    check(slots, slots >= 0, H, P, N, torch.bfloat16, 0)


def test_a_page_that_comes_again_near():
    """Tokens of two pages in turn: the first run of each is written."""
    slots = np.array([5, 6, 37, 7, 38, 39, -1, 8, 100])
    written = np.array([1, 1, 1, 0, 0, 0, 0, 0, 1], bool)
    check(slots, written, 2, 16, 8, torch.bfloat16, -1)
