"""eagle_page_map and eagle_page_release on the GPU against the oracle's loops:
whole numbers, so everything is compared for equality."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import pages as opages

pytestmark = pytest.mark.gpu


def state(seed, B, page, max_pages, kv_max, spare=8):
    rng = np.random.default_rng(seed)
    kv = rng.integers(0, kv_max + 1, B)
    count = -(-kv // page)
    N = B * max_pages + spare
    order = rng.permutation(N)
    table = np.full((B, max_pages), -1)
    used = 0
    for b in range(B):
        table[b, :count[b]] = order[used:used + count[b]]
        used += count[b]
    free = np.full(N, -7)
    free[:N - used] = order[used:]
    return rng, kv, count, table, free, N - used, N


def dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def map_on_gpu(kv, new, table, count, free, fc, page, T):
    t, c, f, n = dev(table), dev(count), dev(free), dev([fc])
    slots = torch.full((T,), -9, dtype=torch.int32, device="cuda") if T is not None else None
    starts = torch.full((len(kv) + 1,), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.page_map(dev(kv), dev(new), t, c, f, n, page, slot_map=slots, new_start=starts, status=status)
    torch.cuda.synchronize()
    return int(status), t, c, f, n, slots, starts


@pytest.mark.parametrize("B,page,new_max,extra", [(1, 16, 0, 3), (1, 16, 1, 0), (1, 64, 20000, 0), (3, 16, 7, 5), (33, 32, 40, 1),
                                                  (257, 16, 60, 100), (1025, 64, 30, 0), (4096, 128, 9, 3), (2, 4096, 9000, 2)])
def test_map_and_release(B, page, new_max, extra):
    kv_max = 300
    mp = (kv_max + new_max) // page + 1
    rng, kv, count, table, free, fc, N = state(B + page, B, page, mp, kv_max)
    new = rng.integers(0, new_max + 1, B)
    if B > 2:
        new[rng.integers(0, B, B // 3)] = 0                       # requests without new tokens, neighbours among them
    T = int(new.sum()) + extra
    err, t_o, c_o, fc_o, slots_o, starts_o = opages.page_map(kv.tolist(), new.tolist(), table.tolist(), count.tolist(),
                                                             free.tolist(), fc, page, N, T=T)
    assert err is None
    st, t, c, f, n, slots, starts = map_on_gpu(kv, new, table, count, free, fc, page, T)
    assert st == 0
    assert slots.tolist() == slots_o and starts.tolist() == starts_o
    assert t.tolist() == t_o and c.tolist() == c_o and n.item() == fc_o and f.tolist() == free.tolist()
    # trim to what is used now: everything is as before the map
    eg.page_release(dev(kv), t, c, f, n, page)
    assert t.tolist() == table.tolist() and c.tolist() == count.tolist()
    assert f.tolist() == free.tolist() and n.item() == fc
    # end some requests, leave some alone, trim others
    keep = np.where(rng.random(B) < 0.4, 0, np.where(rng.random(B) < 0.5, -1, kv // 2))
    t_o, c_o, f_o, fc_o = opages.page_release(keep.tolist(), table.tolist(), count.tolist(), free.tolist(), fc, page)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.page_release(dev(keep), t, c, f, n, page, status=status)
    assert int(status) == 0
    assert t.tolist() == t_o and c.tolist() == c_o and f.tolist() == f_o and n.item() == fc_o


def test_reserving_without_tokens_and_again():
    """No slot map: pages only; a second call for the same tokens takes none."""
    _, kv, count, table, free, fc, N = state(5, 7, 16, 30, 300)
    new = np.full(7, 40)
    st, t, c, f, n, _, starts = map_on_gpu(kv, new, table, count, free, fc, 16, None)
    assert st == 0 and starts.tolist()[-1] == 280
    assert c.tolist() == (-(-(kv + 40) // 16)).tolist()
    before = (t.clone(), c.clone(), n.clone())
    eg.page_map(dev(kv), dev(new), t, c, f, n, 16)
    assert torch.equal(t, before[0]) and torch.equal(c, before[1]) and torch.equal(n, before[2])


@pytest.mark.parametrize("case,code", [("pages", -6), ("negative kv", -1), ("negative new", -1), ("too long", -1),
                                       ("count", -1), ("free", -1), ("T", -1), ("far", -1)])
def test_a_refused_map_changes_nothing(case, code):
    _, kv, count, table, free, fc, N = state(6, 5, 16, 20, 100)
    new = np.full(5, 30)
    T = 150
    if case == "pages":
        fc = 3
    elif case == "negative kv":
        kv[3] = -1
    elif case == "negative new":
        new[0] = -4
    elif case == "too long":
        new[4] = 20 * 16 - kv[4] + 1
        T = 1000
    elif case == "count":
        count[2] = 21
    elif case == "free":
        fc = N + 1
    elif case == "T":
        T = 149
    elif case == "far":
        new[1] = 2 ** 31 - 1
    st, t, c, f, n, slots, starts = map_on_gpu(kv, new, table, count, free, fc, 16, T)
    assert st == code
    assert t.tolist() == table.tolist() and c.tolist() == count.tolist() and n.item() == fc
    assert (slots == -9).all() and (starts == -9).all()


def test_release_refused():
    _, kv, count, table, free, fc, N = state(8, 3, 16, 20, 100)
    for bad_fc, bad_count in ((-1, count), (N, count), (fc, np.array([1, 21, 0]))):
        t, c, f, n = dev(table), dev(bad_count), dev(free), dev([bad_fc])
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        eg.page_release(dev([0, 0, 0]), t, c, f, n, 16, status=status)
        assert int(status) == -1
        assert t.tolist() == table.tolist() and f.tolist() == free.tolist() and n.item() == bad_fc


def test_bad_page_numbers_give_no_slot():
    _, kv, count, table, free, fc, N = state(9, 2, 16, 20, 100)
    kv[:], count[:] = (20, 20), (2, 2)
    table[0, 1], free[fc - 1] = N, -3                              # in use by request 0; the next to be taken
    st, t, c, f, n, slots, _ = map_on_gpu(kv, np.array([13, 12]), table, count, free, fc, 16, 25)
    assert st == -1
    s = slots.tolist()
    assert s[:13] == [-1] * 13                                     # 20..31 on the bad page, 32 on the bad new page
    assert all(x >= 0 for x in s[13:])


def test_captured_and_replayed():
    """The graph keeps addresses only: lengths change between replays."""
    rng, kv, count, table, free, fc, N = state(10, 9, 16, 60, 100)
    new = rng.integers(1, 20, 9)
    kv_d, new_d, t, c, f, n = dev(kv), dev(new), dev(table), dev(count), dev(free), dev([fc])
    slots = torch.empty(200, dtype=torch.int32, device="cuda")
    eg.page_map(kv_d, new_d, t, c, f, n, 16, slot_map=slots)       # first calls outside the capture
    eg.page_release(kv_d, t, c, f, n, 16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        eg.page_map(kv_d, new_d, t, c, f, n, 16, slot_map=slots)
    tl, cl, fl, fcl = table.tolist(), count.tolist(), free.tolist(), fc
    for step in range(4):
        new = rng.integers(0, 20, 9)
        new_d.copy_(dev(new))
        g.replay()
        torch.cuda.synchronize()
        err, tl, cl, fcl, so, _ = opages.page_map(kv.tolist(), new.tolist(), tl, cl, fl, fcl, 16, N, T=200)
        assert err is None and slots.tolist() == so
        assert t.tolist() == tl and c.tolist() == cl and n.item() == fcl
        kv = kv + new
        kv_d.add_(new_d)
