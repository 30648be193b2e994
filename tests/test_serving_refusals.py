"""Refusals of the serving loop's entry points, on the host: the C ABI's
argument checks run before anything is launched, and the binding checks
types, shapes and strides.  No GPU is needed."""
import ctypes

import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg

FAKE = ctypes.c_void_p(0x1000)     # never dereferenced: the checks come first
UNAL = ctypes.c_void_p(0x1008)
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_eagle_gb300 import build
    build.build()
    return eg.load_library()


def refuse(fn, good, code, **changes):
    """`good` with the named positions changed is refused with `code`."""
    args = list(good)
    for pos, value in changes.items():
        args[int(pos[1:])] = value
    assert fn(*args) == code, changes


def test_status_string(lib):
    assert lib.eagle_status_string(-6) == b"too few free pages"


def test_page_map(lib):
    good = [FAKE, FAKE, 4, 16, 8, 64, FAKE, FAKE, FAKE, FAKE, FAKE, 10, None, None, None]
    for p in (0, 1, 6, 7, 8, 9, 10):
        refuse(lib.eagle_page_map, good, INVALID, **{f"_{p}": None})
    refuse(lib.eagle_page_map, good, INVALID, _2=0)
    refuse(lib.eagle_page_map, good, UNSUPPORTED, _2=4097)
    for size in (8, 24, 8192, 0, -16):
        refuse(lib.eagle_page_map, good, INVALID, _3=size)
    refuse(lib.eagle_page_map, good, INVALID, _4=0)
    refuse(lib.eagle_page_map, good, INVALID, _4=(1 << 20) + 1)          # past 2^24 tokens
    refuse(lib.eagle_page_map, good, INVALID, _5=0)
    refuse(lib.eagle_page_map, good, INVALID, _5=1 << 27)                # slots past 31 bits
    refuse(lib.eagle_page_map, good, INVALID, _11=-1)
    refuse(lib.eagle_page_map, good, INVALID, _11=(1 << 30) + 1)
    good = [FAKE, 4, 16, 8, 64, FAKE, FAKE, FAKE, FAKE, None, None]
    for p in (0, 5, 6, 7, 8):
        refuse(lib.eagle_page_release, good, INVALID, **{f"_{p}": None})
    refuse(lib.eagle_page_release, good, INVALID, _1=0)
    refuse(lib.eagle_page_release, good, UNSUPPORTED, _1=5000)
    refuse(lib.eagle_page_release, good, INVALID, _2=17)


def test_rope(lib):
    #       q     k     v  dt B  n Hq Hkv dh  ldq  ldk  ldv  freq rot il  factor
    good = [FAKE, FAKE, FAKE, 1, 2, 3, 4, 2, 64, 256, 128, 128, FAKE, 64, 0, ctypes.c_float(1.0), None, None, 0, FAKE,
            FAKE, FAKE, None]
    good[19] = ctypes.c_void_p(0x2000)
    for p in (0, 1, 12, 19, 20, 21):
        refuse(lib.eagle_rope, good, INVALID, **{f"_{p}": None})
    for p in (0, 1, 2, 19, 20, 21):
        refuse(lib.eagle_rope, good, INVALID, **{f"_{p}": UNAL})
    refuse(lib.eagle_rope, good, INVALID, _3=2)
    for p in (4, 5, 6, 7, 8):
        refuse(lib.eagle_rope, good, INVALID, **{f"_{p}": 0})
    for rot in (0, 3, 66, -2):
        refuse(lib.eagle_rope, good, INVALID, _13=rot)
    refuse(lib.eagle_rope, good, INVALID, _9=255)          # row of 255 elements: not 16 bytes
    refuse(lib.eagle_rope, good, INVALID, _9=128)          # nodes overlap
    refuse(lib.eagle_rope, good, INVALID, _10=64)
    refuse(lib.eagle_rope, good, INVALID, _11=64)
    refuse(lib.eagle_rope, good, UNSUPPORTED, _4=1 << 23)
    refuse(lib.eagle_rope, good, UNSUPPORTED, _8=520, _13=64, _9=4096, _10=4096, _11=4096)
    refuse(lib.eagle_rope, good, INVALID, _0=FAKE, _19=FAKE, _9=512)   # in place with gaps between nodes


def test_kv8_append(lib):
    good = [FAKE, FAKE, 1, 5, 2, 64, 128, 64, FAKE, FAKE, FAKE, FAKE, FAKE, 16, 8, None, None]
    for p in (0, 1, 8, 9, 10, 11, 12):
        refuse(lib.eagle_kv8_append, good, INVALID, **{f"_{p}": None})
    for p in (0, 1, 9, 10):
        refuse(lib.eagle_kv8_append, good, INVALID, **{f"_{p}": UNAL})
    for change in (dict(_2=7), dict(_3=-1), dict(_3=(1 << 30) + 1), dict(_4=0), dict(_5=24), dict(_5=0), dict(_5=528), dict(_6=129), dict(_7=-64),
                   dict(_13=48), dict(_14=0), dict(_14=1 << 28)):
        refuse(lib.eagle_kv8_append, good, INVALID, **change)
    refuse(lib.eagle_kv8_append, good, UNSUPPORTED, _4=40000)
    refuse(lib.eagle_kv8_append, good, 0, _3=0)            # no tokens: nothing to do, nothing launched


def test_kv8_commit(lib):
    good = [FAKE, FAKE, 1, 2, 9, 2, 64, FAKE, FAKE, 6, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 16, 64, FAKE, None, None, None]
    for p in (0, 1, 7, 8, 10, 11, 12, 13, 14, 18):
        refuse(lib.eagle_kv8_commit, good, INVALID, **{f"_{p}": None})
    for change in (dict(_2=3), dict(_3=0), dict(_4=0), dict(_4=5000), dict(_5=0), dict(_6=40), dict(_9=0), dict(_9=65),
                   dict(_15=0), dict(_16=20), dict(_17=0), dict(_0=UNAL), dict(_10=UNAL)):
        refuse(lib.eagle_kv8_commit, good, INVALID, **change)
    refuse(lib.eagle_kv8_commit, good, UNSUPPORTED, _3=70000)


def test_tree_attn_kv8(lib):
    good = [FAKE] * 6 + [8, 16, 64] + [FAKE] * 4 + [1, 2, 3, 8, 2, 64, ctypes.c_float(0.1), FAKE, None, None, None, 0, None]
    for p in (0, 1, 2, 3, 4, 5, 9, 10, 11, 12, 20):
        refuse(lib.eagle_tree_attn_kv8, good, INVALID, **{f"_{p}": None})
    for p in (0, 1, 2, 10, 11, 20):
        refuse(lib.eagle_tree_attn_kv8, good, INVALID, **{f"_{p}": UNAL})
    for change in (dict(_6=0), dict(_7=8), dict(_7=100), dict(_8=0), dict(_13=5), dict(_14=0), dict(_15=0), dict(_15=4097),
                   dict(_16=7), dict(_17=0), dict(_19=ctypes.c_float(0.0)), dict(_19=ctypes.c_float(-1.0)),
                   dict(_19=ctypes.c_float(float("nan")))):
        refuse(lib.eagle_tree_attn_kv8, good, INVALID, **change)
    for change in (dict(_13=0), dict(_18=96), dict(_14=40000), dict(_8=1 << 30, _7=16, _17=4)):
        refuse(lib.eagle_tree_attn_kv8, good, UNSUPPORTED, **change)
    size = lib.eagle_tree_attn_kv8_workspace_size
    assert size(0, 2, 3, 8, 2, 64, 8, 16) == 0 and size(1, 0, 3, 8, 2, 64, 8, 16) == 0
    assert size(1, 2, 3, 7, 2, 64, 8, 16) == 0 and size(1, 2, 3, 8, 2, 80, 8, 16) == 0


def test_tree_attn_kv8_query_rows(lib):
    """Rows of a KV head past 2^23: the kernels count them in 32 bits."""
    good = [FAKE] * 6 + [8, 16, 64] + [FAKE] * 4 + [1, 2, 4096, 8, 2, 64, ctypes.c_float(0.1), FAKE, None, None, None, 0, None]
    refuse(lib.eagle_tree_attn_kv8, good, UNSUPPORTED, _16=2 * 2049)
    refuse(lib.eagle_tree_attn_kv8, good, UNSUPPORTED, _16=2 << 20)        # 2^32 rows
    assert lib.eagle_tree_attn_kv8_workspace_size(1, 2, 4096, 2 * 2049, 2, 64, 8, 16) == 0


def test_a_cache_keeps_the_workspaces_it_outgrows():
    """A captured graph holds the address of the workspace of its capture."""
    from tree_speculative_decoding_eagle_gb300.cache import KV8Cache
    cache = KV8Cache(1, 1, 64, 16, 2, 2, device="cpu")
    first = cache._ws.get(1000)[0]
    again = cache._ws.get(500)[0]
    larger = cache._ws.get(2000)[0]
    assert again is first and larger is not first and larger.numel() == 2000
    assert cache._ws._outgrown[0] is first and len(cache._ws._outgrown) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(eg.EagleError, match="CUDA"):
        eg.page_map(torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros((2, 4), **i32), torch.zeros(2, **i32),
                    torch.zeros(8, **i32), torch.zeros(1, **i32), 16)
    q = torch.zeros((1, 2, 4, 64))
    with pytest.raises(eg.EagleError):
        eg.rope(q, q, q, torch.zeros(32, dtype=torch.float64))
    with pytest.raises(eg.EagleError):
        eg.kv8_append(torch.zeros((3, 2, 64)), torch.zeros((3, 2, 64)), torch.zeros(3, **i32),
                      torch.zeros((4, 2, 16, 64), dtype=torch.uint8), torch.zeros((4, 2, 16, 64), dtype=torch.uint8),
                      torch.ones((4, 2)), torch.ones((4, 2)))
