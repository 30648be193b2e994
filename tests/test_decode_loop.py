"""The decoding loop's rule for the tree's root on the CPU: a restatement with
the oracles, and the host's refusals of the commit that stores the root."""
import ctypes

import numpy as np
import pytest

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import rope

FAKE, UNAL = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)


def attention(Q, K, W, live):
    s = np.where(live, Q @ K.T * Q.shape[1] ** -0.5, -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    return p @ W / p.sum(1, keepdims=True)


@pytest.mark.parametrize("accepted", [0, 2, 3])
def test_the_rule_gives_causal_attention_in_every_step(accepted):
    """kv_len counts the positions before the root; the root is node 0 at
    position kv_len; the commit stores it and the accepted path."""
    rng = np.random.default_rng(accepted)
    dh, V = 32, 100
    f, _ = rope.freqs(dh)
    q, k, v = rng.standard_normal((3, V, dh))
    rot = lambda x, p: rope.rotate(x[:, None, :], np.asarray(p), f)[:, 0]
    seq = rng.integers(0, V, 11).tolist()
    K, W = rot(k[seq], np.arange(11)), v[seq]
    for _ in range(4):
        tree, kv_len = rng.integers(0, V, 4).tolist(), len(K)
        pos = kv_len + np.arange(4)                   # a chain: node i at depth i
        kt, vt = rot(k[tree], pos), v[tree]
        live = np.hstack([np.ones((4, kv_len), bool), np.tril(np.ones((4, 4), bool))])
        got = attention(rot(q[tree], pos), np.vstack([K, kt]), np.vstack([W, vt]), live)
        every = seq + tree
        at = np.arange(len(every))
        want = attention(rot(q[every], at), rot(k[every], at), v[every], np.tril(np.ones((len(every),) * 2, bool)))[-4:]
        np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-14)
        K, W = np.vstack([K, kt[:accepted + 1]]), np.vstack([W, vt[:accepted + 1]])
        seq += tree[:accepted + 1]


def test_commit_root_refusals():
    from tree_speculative_decoding_eagle_gb300 import build
    build.build()
    lib = eg.load_library()
    good = [FAKE, FAKE, 1, 2, 9, 2, 64, FAKE, FAKE, 6, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 16, 64, FAKE, None, None, None]
    changes = [({p: None}, -1) for p in (0, 1, 7, 8, 10, 11, 12, 13, 14, 18)]
    changes += [(c, -1) for c in ({2: 3}, {3: 0}, {4: 0}, {4: 5000}, {5: 0}, {6: 40}, {9: 0}, {9: 65}, {15: 0}, {16: 20}, {17: 0},
                                  {0: UNAL}, {10: UNAL})] + [({3: 70000}, -2)]
    for change, code in changes:
        args = [change.get(i, a) for i, a in enumerate(good)]
        assert lib.eagle_kv8_commit_root(*args) == code, change


def test_page_reserve_refusals():
    from tree_speculative_decoding_eagle_gb300 import build
    build.build()
    lib = eg.load_library()
    good = [FAKE, FAKE, 4, 16, 8, 64, FAKE, FAKE, FAKE, FAKE, FAKE, 10, None, FAKE, None, None]
    changes = [({p: None}, -1) for p in (0, 1, 6, 7, 8, 9, 10, 13)]
    changes += [(c, -1) for c in ({2: 0}, {3: 24}, {4: 0}, {5: 0}, {5: 1 << 27}, {11: -1}, {11: (1 << 30) + 1})] + [({2: 4097}, -2)]
    for change, code in changes:
        args = [change.get(i, a) for i, a in enumerate(good)]
        assert lib.eagle_page_reserve(*args) == code, change


def test_tree_attn_kv8_refuses_a_workspace_off_its_boundary():
    """Partial results are stored as float4s."""
    from tree_speculative_decoding_eagle_gb300 import build
    build.build()
    lib = eg.load_library()
    size = lib.eagle_tree_attn_kv8_workspace_size(1, 1, 61, 8, 8, 128, 64, 64)
    assert size > 0
    args = [FAKE] * 6 + [64, 64, 64] + [FAKE] * 4 + [1, 1, 61, 8, 8, 128, ctypes.c_float(0.1), FAKE, None, None,
                                                    ctypes.c_void_p(0x1004), size, None]
    assert lib.eagle_tree_attn_kv8(*args) == -1
    args[-2] = size - 1
    args[-3] = FAKE
    assert lib.eagle_tree_attn_kv8(*args) == -4


def test_a_cache_names_its_device_once():
    from tree_speculative_decoding_eagle_gb300.cache import KV8Cache
    cache = KV8Cache(1, 1, 64, 16, 2, 2, device="cpu")
    assert cache._ws.device == cache.kv_len.device
