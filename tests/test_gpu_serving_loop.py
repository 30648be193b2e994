"""The serving loop's operators together, as a program uses them: prompts into
the 8-bit cache, then steps of reserve, draft, tree, rotary positions, attention
over the cache in two layers, verification, commit and trim, with a request
that ends and another that takes its place.  After every step the cache's values, lengths
and pages equal the oracle's and the attention is within its tolerance of fp64."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8 as okv8
from oracle import pages as opages
from oracle import rope as orope
from tree_speculative_decoding_eagle_gb300.cache import KV8Cache
from tree_speculative_decoding_eagle_gb300.step import TreeStep

B, D, k, m, V, Hq, Hkv, dh, P, LAYERS = 3, 3, 4, 15, 512, 4, 2, 64, 16, 2
N, MP = 40, 12
bf = torch.bfloat16


class Mirror:
    """The oracle's side of the cache."""

    def __init__(self):
        self.codes = np.zeros((LAYERS, 2, N, Hkv, P, dh), np.uint8)
        self.scale = np.ones((LAYERS, 2, N, Hkv))
        self.table = [[-1] * MP for _ in range(B)]
        self.count, self.free, self.fc = [0] * B, list(range(N - 1, -1, -1)), N
        self.kv = [0] * B

    def reserve(self, new):
        err, self.table, self.count, self.fc, slots, _ = opages.page_map(self.kv, new, self.table, self.count, self.free,
                                                                         self.fc, P, N)
        assert err is None
        return slots

    def release(self, keep):
        self.table, self.count, self.free, self.fc = opages.page_release(keep, self.table, self.count, self.free, self.fc, P)

    def write(self, layer, kv, rows, slots):
        okv8.append(rows, slots, self.codes[layer, kv], self.scale[layer, kv])

    def values(self, layer, kv, b):
        return okv8.gather(self.codes[layer, kv], self.scale[layer, kv], np.array(self.table[b]), self.kv[b])

    def same_as(self, c):
        assert int(c.status) == 0
        assert c.kv_len.tolist() == self.kv and c.page_count.tolist() == self.count
        assert c.block_table.tolist() == self.table and c.free_count.item() == self.fc
        assert c.free_pages.tolist()[:self.fc] == self.free[:self.fc]
        for layer in range(LAYERS):
            for i, (p, s) in enumerate(((c.k_pages, c.k_scale), (c.v_pages, c.v_scale))):
                np.testing.assert_array_equal(s[layer].double().cpu().numpy(), self.scale[layer, i])
                np.testing.assert_array_equal(p[layer].view(torch.uint8).cpu().numpy(), self.codes[layer, i])


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def prompt(cache, mirror, new, g, freqs):
    """new[b] prompt tokens a request, packed, through rope into the cache."""
    T = sum(new)
    slots, starts = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(B + 1, dtype=torch.int32, device="cuda")
    cache.reserve(i32(new), slots, starts)
    want = mirror.reserve(new)
    assert slots.tolist() == want
    pos = np.concatenate([np.arange(kv, kv + n) for kv, n in zip(mirror.kv, new)]) if T else np.zeros(0, int)
    for layer in range(LAYERS):
        qkv = torch.randn((1, T, Hq + 2 * Hkv, dh), generator=g).to(bf).cuda()
        q, kk, v = qkv.split([Hq, Hkv, Hkv], 2)
        _, kt, vt = eg.rope(q, kk, v, freqs, pos_off=i32(pos.reshape(1, -1).tolist()), interleaved=True)
        np.testing.assert_allclose(f64(kt[0]).transpose(1, 0, 2), orope.rotate(f64(kk[0]), pos, freqs.cpu().numpy(), 1.0, True),
                                   rtol=2 ** -7, atol=1e-5)
        cache.append(layer, kt[0].transpose(0, 1), vt[0].transpose(0, 1), slots)
        mirror.write(layer, 0, f64(kt[0]).transpose(1, 0, 2), want)
        mirror.write(layer, 1, f64(vt[0]).transpose(1, 0, 2), want)
    cache.grow(i32(new))
    mirror.kv = [a + b for a, b in zip(mirror.kv, new)]


def one_step(cache, mirror, step, g, freqs):
    cache.reserve(i32([D] * B))
    mirror.reserve([D] * B)
    draft = (torch.randn((B, D, k, V), generator=g) * 4).cuda()
    step.draft(draft)
    step.build()
    trees = []
    n = m + 1
    keep = np.array([[[bool((int(w) >> j) & 1) for j in range(n)] for w in row[:, 0]] for row in step.tree["mask"].cpu().numpy()])
    for layer in range(LAYERS):
        qkv = torch.randn((B, n, (Hq + 2 * Hkv) * dh), generator=g).to(bf).cuda()
        q, kk, v = (t.unflatten(2, (-1, dh)) for t in qkv.split([Hq * dh, Hkv * dh, Hkv * dh], 2))
        q, kt, vt = eg.rope(q, kk, v, freqs, pos_base=cache.kv_len, pos_off=step.tree["depth"], interleaved=True)
        out, lse = step.attend_kv8(cache, layer, q, kt, vt)
        trees.append((kt, vt))
        for b in range(B):
            K = np.concatenate([mirror.values(layer, 0, b), f64(kt[b])], 1)
            W = np.concatenate([mirror.values(layer, 1, b), f64(vt[b])], 1)
            live = np.concatenate([np.ones((n, mirror.kv[b]), bool), keep[b]], 1)
            for h in range(Hq):
                s = np.where(live, f64(q[b, :, h]) @ K[h // (Hq // Hkv)].T * dh ** -0.5, -np.inf)
                p = np.exp(s - s.max(1, keepdims=True))
                ref = p @ W[h // (Hq // Hkv)] / p.sum(1, keepdims=True)
                A = p @ np.abs(W[h // (Hq // Hkv)]) / p.sum(1, keepdims=True)
                # bf16's rounding, the weights' f16 (half a step is 2^-11), scores below 2^5 of 64 products in fp32, twice
                tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (2.0 ** -11 + 2 * 64 * 2.0 ** -23 * 2 ** 5) * A
                assert (np.abs(f64(out[b, :, h]) - ref) <= tol).all()
    # targets that follow the draft, so that some nodes are accepted
    row = step.tree["row"].cpu()
    flat = draft.cpu().view(B, D * k, V)
    target = torch.stack([torch.stack([flat[b, r] if r >= 0 else torch.randn(V, generator=g) for r in row[b].tolist()]) for b in range(B)])
    step.verify((target + 0.3 * torch.randn(target.shape, generator=g)).cuda())
    cache.commit([t[0] for t in trees], [t[1] for t in trees], step.accept_len, step.path_nodes)
    acc, path = step.accept_len.tolist(), step.path_nodes.tolist()
    for b in range(B):
        pos = [mirror.kv[b] + i for i in range(acc[b])]
        slots = [mirror.table[b][p // P] * P + p % P for p in pos]
        for layer, (kt, vt) in enumerate(trees):
            for i, t in enumerate((kt, vt)):
                mirror.write(layer, i, f64(t[b])[:, path[b][1:acc[b] + 1]].transpose(1, 0, 2), slots)
        mirror.kv[b] += acc[b]
    cache.trim()
    mirror.release(mirror.kv)
    assert int(step.status) == 0
    return sum(acc)


@pytest.mark.gpu
def test_prompts_steps_release_and_a_new_request():
    g = torch.Generator().manual_seed(77)
    cache, mirror = KV8Cache(B, Hkv, dh, P, N, MP, layers=LAYERS), Mirror()
    step = TreeStep(B, D, k, m, V, Hq, Hkv, dh, MP * P)
    freqs, _ = eg.rope_freqs(32, kind="bands", stretch=4.0, orig_len=64, low=1.0, high=4.0)
    prompt(cache, mirror, [37, 1, 64], g, freqs)
    mirror.same_as(cache)
    accepted = 0
    for _ in range(6):
        accepted += one_step(cache, mirror, step, g, freqs)
        mirror.same_as(cache)
    assert accepted > 0
    # request 2 ends, another one begins in its place with a prompt in two chunks
    cache.release(i32([-1, -1, 0]))
    mirror.release([-1, -1, 0])
    cache.kv_len[2] = 0
    mirror.kv[2] = 0
    prompt(cache, mirror, [0, 0, 21], g, freqs)
    prompt(cache, mirror, [0, 3, 30], g, freqs)
    mirror.same_as(cache)
    for _ in range(3):
        one_step(cache, mirror, step, g, freqs)
        mirror.same_as(cache)


@pytest.mark.gpu
def test_the_cache_part_of_a_step_in_a_graph():
    """reserve, attend, commit and trim captured once and replayed: the same as
    the calls made one by one on a second cache."""
    g = torch.Generator().manual_seed(5)
    caches = [KV8Cache(B, Hkv, dh, P, N, MP, layers=LAYERS) for _ in range(2)]
    n, new = 9, i32([20, 5, 31])
    x = torch.randn((2, LAYERS, 56, Hkv, dh), generator=g).to(bf).cuda()
    for c in caches:
        slots = torch.empty(56, dtype=torch.int32, device="cuda")
        c.reserve(new, slots)
        for layer in range(LAYERS):
            c.append(layer, x[0, layer], x[1, layer], slots)
        c.grow(new)
    tree = [torch.randn((LAYERS, B, Hkv, n, dh), generator=g).to(bf).cuda() for _ in range(2)]
    q = torch.randn((B, n, Hq, dh), generator=g).to(bf).cuda()
    mask = eg.tree_mask(i32([[-1] + list(range(n - 1))] * B))
    acc, path = i32([2, 0, 3]), i32([[0, 1, 2, -1], [0, -1, -1, -1], [0, 4, 5, 6]])
    need = i32([D] * B)
    out = [torch.empty_like(q) for _ in range(2)]
    lse = torch.empty((B, n, Hq), device="cuda")
    slots = torch.empty((B, n), dtype=torch.int32, device="cuda")

    def step(c, o):
        c.reserve(need)
        for layer in range(LAYERS):
            c.attend(layer, q, tree[0][layer], tree[1][layer], mask, out=o, lse=lse)
        c.commit(list(tree[0]), list(tree[1]), acc, path, slots)
        c.trim()

    step(caches[0], out[0])
    step(caches[1], out[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], out[0])
    for _ in range(5):
        graph.replay()
        step(caches[1], out[1])
        torch.cuda.synchronize()
        a, b = caches
        assert torch.equal(out[0], out[1])
        for name in ("kv_len", "page_count", "block_table", "free_count", "free_pages", "status"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        for name in ("k_pages", "v_pages"):
            assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(getattr(a, name), getattr(b, name)))
        assert all(torch.equal(s, t) for s, t in zip(a.k_scale + a.v_scale, b.k_scale + b.v_scale))
    assert int(caches[0].status) == 0 and caches[0].kv_len.tolist() == [20 + 12, 5, 31 + 18]


@pytest.mark.gpu
def test_a_captured_attend_outlives_a_larger_workspace():
    """A larger call grows the cache's workspace: the graph captured before it
    keeps its own, whatever is allocated and written afterwards."""
    g = torch.Generator().manual_seed(6)
    cache = KV8Cache(2, 2, 64, 16, 80, 40)
    new = i32([600, 333])
    slots = torch.empty(933, dtype=torch.int32, device="cuda")
    cache.reserve(new, slots)
    kv = torch.randn((2, 933, 2, 64), generator=g).to(bf).cuda()
    cache.append(0, kv[0], kv[1], slots)
    cache.grow(new)

    def inputs(n):
        return ([torch.randn(s, generator=g).to(bf).cuda() for s in ((2, n, 8, 64), (2, 2, n, 64), (2, 2, n, 64))]
                + [eg.tree_mask(i32([[-1] + list(range(n - 1))] * 2))])

    small, large = inputs(12), inputs(60)
    out, lse = torch.empty_like(small[0]), torch.empty((2, 12, 8), device="cuda")
    want, want_lse = cache.attend(0, *small)
    held = cache._ws.buf
    assert held is not None                      # the KV range is split
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(0, *small, out=out, lse=lse)
    cache.attend(0, *large)
    cache._ws.get(held.numel() + 1)              # what a call of more split rows asks for
    assert cache._ws.buf is not held
    size, address = held.numel(), held.data_ptr()
    del held
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(20)]
    assert all(t.data_ptr() != address for t in others)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert all(bool((t == 7).all()) for t in others)


@pytest.mark.gpu
def test_calls_on_a_given_stream():
    """`stream`: what a call allocates for itself belongs to that stream, so
    work of the current stream that follows does not touch it."""
    g = torch.Generator().manual_seed(7)
    cache = KV8Cache(2, 2, 64, 16, 80, 40)
    new = i32([600, 333])
    slots = torch.empty(933, dtype=torch.int32, device="cuda")
    cache.reserve(new, slots)
    kv = torch.randn((2, 933, 2, 64), generator=g).to(bf).cuda()
    cache.append(0, kv[0], kv[1], slots)
    cache.grow(new)
    n = 12
    x = [torch.randn((2, n, h, 64), generator=g).to(bf).cuda() for h in (8, 2, 2)]
    mask = eg.tree_mask(i32([[-1] + list(range(n - 1))] * 2))
    freqs, factor = eg.rope_freqs(64)

    def run(stream=None):
        q, k, v = eg.rope(*x, freqs, pos_base=cache.kv_len, factor=factor, stream=stream)
        return (q, k, v) + eg.tree_attn_kv8(q, *cache._pools(0), cache.block_table, cache.kv_len, k, v, mask, stream=stream)

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = run(side)
        junk = [torch.full((1 << 20,), 3, dtype=torch.uint8, device="cuda") for _ in range(8)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
    with pytest.raises(eg.EagleError):
        eg.rope(x[0], x[1][0, 0], None, freqs)


def test_a_cache_checks_its_arguments():
    with pytest.raises(eg.EagleError):
        KV8Cache(1, 1, 64, 16, 4, 4, layers=0, device="cpu")
    c = KV8Cache(1, 1, 64, 16, 4, 4, layers=2, device="cpu")
    with pytest.raises(eg.EagleError):
        c.commit([None], [None], None, None)
