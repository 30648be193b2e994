"""eagle_kv8_bounds on the GPU against the oracle: equal to the last bit of every
value (a bound is an e4m3 number)."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8, select

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    def __init__(self, kv, Hkv, dh, P, seed=0, extra=2, nan=0.0):
        rng = np.random.default_rng(seed)
        B = len(kv)
        self.kv, self.P = kv, P
        self.mp = max(1, max(-(-k // P) for k in kv)) + extra
        self.N = B * self.mp + 3
        self.codes = rng.integers(0, 256, (self.N, Hkv, P, dh)).astype(np.uint8)
        if nan < 1:
            bad = (self.codes & 127) == 127
            self.codes[bad & (rng.random(self.codes.shape) >= nan)] = 0x3a
        perm = rng.permutation(self.N)[:B * self.mp].reshape(B, self.mp)
        self.table = np.where(np.arange(self.mp)[None] < -(-np.array(kv)[:, None] // P), perm, -1).astype(np.int32)
        self.before = rng.integers(0, 127, (self.N, Hkv, 2, dh)).astype(np.uint8)

    def want(self, since):
        out = kv8.decode(self.before)
        for b, (lo, hi) in enumerate(zip(since, self.kv)):
            lo = max(lo, 0)
            if hi <= lo:
                continue
            for p in range(lo // self.P, -(-hi // self.P)):
                page = self.table[b, p]
                rows = min(self.P, hi - p * self.P)
                for g in range(self.codes.shape[1]):
                    out[page, g] = np.stack(select.bounds(kv8.decode(self.codes[page, g, :rows])))
        return out

    def run(self, since):
        got = torch.from_numpy(self.before.copy()).cuda()
        status = i32([0])
        eg.kv8_bounds(torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.table).cuda(), i32(since), i32(self.kv), got, status=status)
        torch.cuda.synchronize()
        assert int(status) == 0
        np.testing.assert_array_equal(kv8.decode(got.cpu().numpy()), self.want(since))


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 256])
def test_lengths_around_pages(dh, P):
    kv = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 130, 256, 257, 300]
    Pool(kv, 3, dh, P, seed=P).run([0] * len(kv))
    Pool(kv, 2, dh, P, seed=P + 1).run([max(0, k - 1) for k in kv])
    Pool(kv, 1, dh, P, seed=P + 2).run([k // 2 for k in kv])
    Pool(kv, 1, dh, P, seed=P + 2).run([k + (i % 3) - 1 for i, k in enumerate(kv)])    # some not grown, some shrunk, one negative


def test_nan_rows_widen_and_rows_past_the_length_do_not():
    Pool([1, 40, 64, 7], 2, 128, 32, nan=0.02).run([0, 0, 33, 5])
    Pool([1, 40, 64, 7], 2, 64, 32, nan=1.0).run([0, 0, 33, 5])
    p = Pool([5], 1, 64, 16)
    p.codes[p.table[0, 0], :, 5:] = 0x7f
    p.run([0])


def test_every_number_of_the_type():
    p = Pool([256], 1, 64, 256)
    p.codes[p.table[0, 0], 0, :, :] = np.arange(256, dtype=np.uint8)[:, None]
    p.codes[p.table[0, 0], 0, 127] = p.codes[p.table[0, 0], 0, 255] = 0
    for rows in (1, 2, 100, 127, 200):
        p.kv = [rows]
        p.run([0])


@pytest.mark.parametrize("B,Hkv", [(1, 1), (1, 40), (70, 2), (300, 1)])
def test_many_requests_and_long_ones(B, Hkv):
    rng = np.random.default_rng(B)
    kv = rng.integers(0, 90, B).tolist()
    kv[B // 2] = 3000
    Pool(kv, Hkv, 64, 16, seed=B).run([max(0, k - int(rng.integers(0, 40))) for k in kv])
    Pool(kv, Hkv, 128, 64, seed=B).run([0] * B)


def test_page_numbers_outside_the_pool_are_skipped_and_lengths_clamped():
    p = Pool([40, 33], 2, 64, 16, extra=0)
    p.table[0, 1], p.table[1, 0] = -7, p.N
    for bad in (i32([0]), None):
        got = torch.from_numpy(p.before.copy()).cuda()
        eg.kv8_bounds(torch.from_numpy(p.codes).cuda(), torch.from_numpy(p.table).cuda(), i32([0, 0]), i32([40, 10 ** 9]), got, status=bad)
        torch.cuda.synchronize()
        assert bad is None or int(bad) == -1
        want = kv8.decode(p.before)
        for b, lp in ((0, 0), (0, 2), (1, 1), (1, 2)):
            rows = 16 if b else min(16, 40 - 16 * lp)
            for g in range(2):
                want[p.table[b, lp], g] = np.stack(select.bounds(kv8.decode(p.codes[p.table[b, lp], g, :rows])))
        np.testing.assert_array_equal(kv8.decode(got.cpu().numpy()), want)


def test_the_largest_pages():
    Pool([4096 + 17], 1, 128, 4096, extra=0).run([4000])


def test_binding_refuses():
    p = Pool([20], 2, 64, 16)
    codes, table = torch.from_numpy(p.codes).cuda(), torch.from_numpy(p.table).cuda()
    good = torch.from_numpy(p.before).cuda()
    for bad in (good[:-1], good.float(), good.cpu(), good[..., ::2]):
        with pytest.raises(eg.EagleError):
            eg.kv8_bounds(codes, table, i32([0]), i32([20]), bad)
    with pytest.raises(eg.EagleError):
        eg.kv8_bounds(codes, table, i32([0, 0]), i32([20]), good)
    with pytest.raises(eg.EagleError):
        eg.kv8_bounds(codes.float(), table, i32([0]), i32([20]), good)
