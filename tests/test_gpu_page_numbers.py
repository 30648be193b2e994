"""Page numbers outside the pool, in the block table and in the free list: no
such number travels on, and the status tells."""
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("where", [0, 1023, 1024, 4095, 4096, 5499])
@pytest.mark.parametrize("bad", [-1, 9000, 2 ** 31 - 1, -2 ** 31])
def test_release_hands_on_no_bad_page(bad, where):
    """Request 1 gives back 5500 pages, one of which is none: nothing changes."""
    N, mp = 9000, 6000
    table = torch.full((3, mp), -1, dtype=torch.int32)
    table[0, :10] = torch.arange(10)
    table[1, :5505] = torch.arange(10, 5515)
    table[1, 5 + where] = bad
    count, free, fc = i32([10, 5505, 0]), torch.full((N,), -7, dtype=torch.int32, device="cuda"), i32([4])
    free[:4] = i32([8990, 8991, 8992, 8993])
    t, status = table.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    before = free.clone()
    eg.page_release(i32([-1, 5 * 16, 0]), t, count, free, fc, 16, status=status)
    assert int(status) == -1
    assert torch.equal(t.cpu(), table) and count.tolist() == [10, 5505, 0] and fc.item() == 4 and torch.equal(free, before)
    # with the number mended the same call gives the pages back, in order
    t[1, 5 + where] = 15 + where
    status.zero_()
    eg.page_release(i32([-1, 5 * 16, 0]), t, count, free, fc, 16, status=status)
    assert int(status) == 0 and count.tolist() == [10, 5, 0] and fc.item() == 5504
    assert free[:5504].tolist() == [8990, 8991, 8992, 8993] + list(range(5514, 14, -1))
    assert (t[1, 5:] == -1).all() and t[1, :5].tolist() == [10, 11, 12, 13, 14]


def test_a_bad_page_that_is_kept_does_not_matter():
    t, count, free, fc = i32([[-1, 3, 4]]), i32([3]), i32([-7] * 8), i32([0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.page_release(i32([16]), t, count, free, fc, 16, status=status)
    assert int(status) == 0 and t.tolist() == [[-1, -1, -1]] and fc.item() == 2 and free[:2].tolist() == [4, 3]


@pytest.mark.parametrize("bad", [-3, 8])
@pytest.mark.parametrize("slots", [True, False])
def test_map_takes_no_bad_page(bad, slots):
    t, count, free, fc = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), i32([0, 0]), i32([0, 1, bad, 3, 0, 0, 0, 0]), i32([4])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((40,), 9, dtype=torch.int32, device="cuda") if slots else None
    eg.page_map(i32([0, 0]), i32([20, 20]), t, count, free, fc, 16, slot_map=out, status=status)
    assert int(status) == -1
    assert t.tolist() == [[3, -1, -1, -1], [1, 0, -1, -1]] and count.tolist() == [2, 2] and fc.item() == 0
    if slots:
        assert out.tolist() == list(range(48, 64)) + [-1] * 4 + list(range(16, 32)) + list(range(4))
