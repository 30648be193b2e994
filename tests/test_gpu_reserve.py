"""Reservations that the free list cannot serve, in a loop that goes on without
looking at the status: nothing is written and nothing is counted."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import pages as opages
from tree_speculative_decoding_eagle_gb300.cache import KV8Cache

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,T", [(1, 2), (5, 150), (1500, 9000), (3, 40000)])
@pytest.mark.parametrize("why,code", [("pages", -6), ("length", -1), ("count", -1), ("free", -1), ("T", -1), (None, 0)])
def test_a_refusal_is_written_out(B, T, why, code):
    page, mp, N = 16, 3000, 4 * B + 4000
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 40, B)
    new = np.diff(np.concatenate([[0], np.sort(rng.integers(0, T + 1, B - 1)), [T]]))
    count = -(-kv // page)
    used = int(count.sum())
    order = rng.permutation(N)
    table = np.full((B, mp), -1)
    at = 0
    for b in range(B):
        table[b, :count[b]] = order[at:at + count[b]]
        at += count[b]
    free = np.concatenate([order[used:], np.full(used, -7)])
    fc, room = N - used, T
    if why == "pages":
        fc = int((np.maximum(count, -(-(kv + new) // page)) - count).sum()) - 1
        if fc < 0:
            kv[0], new[0], fc = count[0] * page, T, -(-T // page) - 1
            new[1:] = 0
    elif why == "length":
        kv[B // 2] = -1
    elif why == "count":
        count[0] = mp + 1
    elif why == "free":
        fc = N + 1
    elif why == "T":
        room = T - 1
    t, c, f, n = i32(table), i32(count), i32(free), i32([fc])
    slots, starts = torch.full((room,), 77, dtype=torch.int32, device="cuda"), torch.full((B + 1,), 77, dtype=torch.int32, device="cuda")
    granted, status = torch.full((1,), 77, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.page_map(i32(kv), i32(new), t, c, f, n, page, slot_map=slots, new_start=starts, status=status, granted=granted)
    assert int(status) == code
    if code:
        assert (slots == -1).all() and not starts.any() and granted.item() == 0
        assert t.tolist() == table.tolist() and c.tolist() == count.tolist() and n.item() == fc
    else:
        err, t_o, c_o, fc_o, slots_o, starts_o = opages.page_map(kv.tolist(), new.tolist(), table.tolist(), count.tolist(),
                                                                 free.tolist(), fc, page, N, T=room)
        assert err is None and granted.item() == 1
        assert slots.tolist() == slots_o and starts.tolist() == starts_o and t.tolist() == t_o and n.item() == fc_o
    assert f.tolist() == free.tolist()


def test_a_captured_loop_runs_out_of_pages_and_recovers():
    """Two requests decode one token a replay until the pool is empty: the slots
    of the last served step must not be written again, nor lengths grow."""
    B, H, dh, page = 2, 2, 64, 16
    c = KV8Cache(B, H, dh, page, 4, 4)
    one = i32([1, 1])
    slots = torch.empty(B, dtype=torch.int32, device="cuda")
    x = torch.zeros((2, B, H, dh), device="cuda")

    def step():
        c.reserve(one, slots)
        c.append(0, x[0], x[1], slots)
        c.grow(one)

    step()                                             # position 0 of both
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, 32):
        x.fill_(float(i))
        graph.replay()
    assert int(c.status) == 0 and c.kv_len.tolist() == [32, 32] and c.free_count.item() == 0
    held = [t.view(torch.uint8).clone() for t in (c.k_pages[0], c.v_pages[0])] + [c.k_scale[0].clone(), c.v_scale[0].clone()]
    x.fill_(384.0)
    for _ in range(3):                                 # nothing free: nothing happens
        graph.replay()
    assert int(c.status) == -6 and c.kv_len.tolist() == [32, 32]
    now = [t.view(torch.uint8) for t in (c.k_pages[0], c.v_pages[0])] + [c.k_scale[0], c.v_scale[0]]
    assert all(torch.equal(a, b) for a, b in zip(held, now))
    c.status.zero_()
    c.release(i32([0, -1]))
    c.kv_len[0] = 0
    graph.replay()                                     # both are served again
    assert int(c.status) == 0 and c.kv_len.tolist() == [1, 33] and (slots >= 0).all()
    page0 = int(c.block_table[0, 0])
    assert float(c.k_pages[0][page0, 0, 0, 0].float() * c.k_scale[0][page0, 0]) == 384.0


def test_grow_takes_numbers_and_tensors_and_counts_nothing_after_a_refusal():
    c = KV8Cache(2, 1, 64, 16, 2, 8)
    c.grow(3)                                          # before any reservation: as it is told
    assert c.kv_len.tolist() == [3, 3]
    c.kv_len.zero_()
    c.reserve(i32([5, 20]))                            # three pages of two
    c.grow(i32([5, 20]))
    assert int(c.status) == -6 and c.kv_len.tolist() == [0, 0]
    c.status.zero_()
    c.reserve(i32([5, 16]))
    c.grow(4)
    c.grow(torch.tensor([1, 12], device="cuda"))
    assert int(c.status) == 0 and c.kv_len.tolist() == [5, 16]
    c.reserve(i32([3, 0]))                             # two reservations, then what both were for
    c.reserve(i32([0, 0]))
    c.grow(i32([3, 0]))
    assert int(c.status) == 0 and c.kv_len.tolist() == [8, 16]
    c.grow(-2)
    assert c.kv_len.tolist() == [6, 14]
