"""Refusals of the long-context entry points and of the head norms, on the host:
the argument checks run before anything is launched.  No GPU is needed."""
import ctypes

import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from test_serving_refusals import FAKE, INVALID, UNAL, UNSUPPORTED, lib, refuse  # noqa: F401

WORKSPACE = -4
F = ctypes.c_float


def test_qk_norm_rope(lib):  # noqa: F811
    #       q     k     v  dt B  n Hq Hkv dh  ldq  ldk  ldv  qw   kw    offset   eps      freq rot il factor base off shift
    good = [FAKE, FAKE, FAKE, 1, 2, 3, 4, 2, 64, 256, 128, 128, FAKE, FAKE, F(0.0), F(1e-6), FAKE, 64, 0, F(1.0), None, None, 0,
            ctypes.c_void_p(0x2000), FAKE, FAKE, None]
    fn = lib.eagle_qk_norm_rope
    for p in (0, 1, 16, 23, 24, 25):
        refuse(fn, good, INVALID, **{f"_{p}": None})
    for p in (0, 1, 2, 12, 13, 23, 24, 25):
        refuse(fn, good, INVALID, **{f"_{p}": UNAL})
    for p in (4, 5, 6, 7, 8):
        refuse(fn, good, INVALID, **{f"_{p}": 0})
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        refuse(fn, good, INVALID, _15=F(eps))
    for off in (float("nan"), float("inf"), float("-inf")):
        refuse(fn, good, INVALID, _14=F(off))
    for rot in (0, 3, 66, -2):
        refuse(fn, good, INVALID, _17=rot)
    refuse(fn, good, INVALID, _3=2)
    refuse(fn, good, INVALID, _9=255)
    refuse(fn, good, INVALID, _9=128)
    refuse(fn, good, UNSUPPORTED, _4=1 << 23)
    refuse(fn, good, UNSUPPORTED, _8=520, _9=4096, _10=4096, _11=4096)
    refuse(fn, good, INVALID, _0=FAKE, _23=FAKE, _9=512)   # in place with gaps between nodes


def test_kv8_bounds(lib):  # noqa: F811
    good = [FAKE, FAKE, 8, 16, 64, FAKE, FAKE, 2, 4, 64, FAKE, None, None]
    fn = lib.eagle_kv8_bounds
    for p in (0, 1, 5, 6, 10):
        refuse(fn, good, INVALID, **{f"_{p}": None})
    for p in (0, 10):
        refuse(fn, good, INVALID, **{f"_{p}": UNAL})
    for change in (dict(_2=0), dict(_3=8), dict(_3=48), dict(_3=8192), dict(_4=0), dict(_7=0), dict(_8=0), dict(_2=1 << 21)):
        refuse(fn, good, INVALID, **change)
    for change in (dict(_9=96), dict(_9=256), dict(_7=65536), dict(_4=1 << 30)):
        refuse(fn, good, UNSUPPORTED, **change)


def test_kv8_select(lib):  # noqa: F811
    #       q    dt bounds scale table mp  P  N   kv   B  n Hq Hkv dh top first last sel score status ws bytes
    good = [FAKE, 1, FAKE, FAKE, FAKE, 8, 16, 64, FAKE, 2, 3, 8, 2, 64, 4, 1, 1, FAKE, None, None, FAKE, 1 << 20, None]
    fn, size = lib.eagle_kv8_select, lib.eagle_kv8_select_workspace_size
    for p in (0, 2, 3, 4, 8, 17):
        refuse(fn, good, INVALID, **{f"_{p}": None})
    for p in (0, 2, 20):
        refuse(fn, good, INVALID, **{f"_{p}": UNAL})
    for change in (dict(_1=3), dict(_5=0), dict(_6=24), dict(_7=0), dict(_9=0), dict(_10=0), dict(_10=4097), dict(_11=7), dict(_12=0),
                   dict(_14=0), dict(_15=-1), dict(_16=-1), dict(_15=4), dict(_15=2, _16=3), dict(_15=2 ** 31 - 1, _16=2 ** 31 - 1)):
        refuse(fn, good, INVALID, **change)
    for change in (dict(_1=0), dict(_13=96), dict(_5=16385), dict(_14=16385), dict(_11=66), dict(_9=40000), dict(_7=1 << 30),
                   dict(_9=8192, _10=4096)):
        refuse(fn, good, UNSUPPORTED, **change)
    assert size(1, 2, 3, 8, 2, 64, 8, 16) == 2 * 3 * 2 * 8 * 4 and size(1, 1, 1, 1, 1, 128, 9, 16) == 16 * 4
    refuse(fn, good, WORKSPACE, _20=None)
    refuse(fn, good, WORKSPACE, _21=2 * 3 * 2 * 8 * 4 - 1)
    assert size(0, 2, 3, 8, 2, 64, 8, 16) == 0 and size(1, 2, 3, 8, 2, 64, 16385, 16) == 0 and size(1, 2, 3, 7, 2, 64, 8, 16) == 0


def test_tree_attn_kv8_pages(lib):  # noqa: F811
    good = [FAKE] * 6 + [8, 16, 64] + [FAKE] * 5 + [4, 1, 2, 3, 8, 2, 64, F(0.1), FAKE, None, None, None, 0, None]
    fn, size = lib.eagle_tree_attn_kv8_pages, lib.eagle_tree_attn_kv8_pages_workspace_size
    for p in (0, 1, 2, 3, 4, 5, 9, 10, 11, 12, 13, 22):
        refuse(fn, good, INVALID, **{f"_{p}": None})
    for p in (0, 1, 2, 10, 11, 22):
        refuse(fn, good, INVALID, **{f"_{p}": UNAL})
    for change in (dict(_6=0), dict(_7=8), dict(_8=0), dict(_14=0), dict(_14=(1 << 20) + 1), dict(_15=5), dict(_16=0), dict(_17=0),
                   dict(_17=4097), dict(_18=7), dict(_19=0), dict(_21=F(0.0)), dict(_21=F(float("nan")))):
        refuse(fn, good, INVALID, **change)
    for change in (dict(_15=0), dict(_20=96), dict(_16=40000), dict(_8=1 << 30), dict(_18=66), dict(_16=8192, _17=4096)):
        refuse(fn, good, UNSUPPORTED, **change)
    assert size(1, 2, 3, 66, 2, 64, 4, 8, 16) == 0 and size(0, 2, 3, 8, 2, 64, 4, 8, 16) == 0 and size(1, 2, 3, 8, 2, 64, 0, 8, 16) == 0


def test_binding_refuses_host_tensors_and_caches_without_bounds():
    from tree_speculative_decoding_eagle_gb300.cache import KV8Cache
    q = torch.zeros((1, 2, 4, 64))
    with pytest.raises(eg.EagleError, match="CUDA"):
        eg.qk_norm_rope(q, q, q, torch.zeros(32, dtype=torch.float64))
    i32 = dict(dtype=torch.int32)
    pages = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    with pytest.raises(eg.EagleError, match="CUDA"):
        eg.kv8_bounds(pages, torch.zeros((1, 4), **i32), torch.zeros(1, **i32), torch.zeros(1, **i32), pages[:, :, :2])
    with pytest.raises(eg.EagleError, match="CUDA"):
        eg.kv8_select(q.bfloat16(), pages[:, :, :2], torch.ones((4, 2)), torch.zeros((1, 4), **i32), torch.zeros(1, **i32), 16, 2)
    with pytest.raises(eg.EagleError, match="bounds"):
        KV8Cache(1, 2, 64, 16, 4, 4, device="cpu").select(0, q, 2)
