"""The short bounded wait that every role of the 8-bit attention uses: it gives up
at its limit, and at once (a millisecond or so) when another role has given up."""
import ctypes

import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg

TIMEOUT = -5


def test_waits_that_do_not_exist_are_refused_on_the_host():
    from tree_speculative_decoding_eagle_gb300 import build
    build.build()
    lib = eg.load_library()
    for which in (-1, 2, 5):
        assert lib.eagle_selftest_wait(1_000_000, which, ctypes.c_void_p(0x1000), None, None) == -1


@pytest.mark.gpu
def test_it_gives_up_at_its_limit():
    for limit in (1_000_000, 20_000_000):
        status, waited = eg.selftest_wait(limit, 3)
        assert status == TIMEOUT
        assert limit <= waited < limit + 50_000_000
    assert float(torch.ones(4, device="cuda").sum()) == 4.0      # the context is as usable as before


@pytest.mark.gpu
def test_it_ends_early_when_another_role_gave_up():
    limit = 100_000_000
    status, waited = eg.selftest_wait(limit, 4)
    assert status == TIMEOUT and waited < limit // 2
