"""The long-context operators together, as a program uses them: prompts into an
8-bit cache with bounds, then steps of reserve, draft, tree, norm and rotation,
selection and attention over the selected pages in two layers, verification, commit
(which renews the bounds) and trim.  After every step the bounds equal the oracle's
over the oracle's cache, the selected pages equal the oracle's, and the attention
is within its tolerance of fp64."""
import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8 as okv8
from oracle import select as oselect
from test_gpu_serving_loop import B, D, LAYERS, MP, Mirror, N, P, V, bf, dh, f64, Hkv, Hq, i32, k, m, prompt
from tree_speculative_decoding_eagle_gb300.cache import KV8Cache
from tree_speculative_decoding_eagle_gb300.step import TreeStep

pytestmark = pytest.mark.gpu
G = Hq // Hkv
TOP, FIRST, LAST = 3, 1, 1


def boxes(mirror, layer, b):
    """Bounds and key scales [pages, Hkv, ..] of a request's prefix by the oracle."""
    L = mirror.kv[b]
    pages = [mirror.table[b][p] for p in range(-(-L // P))]
    lo = np.zeros((len(pages), Hkv, dh))
    hi = np.zeros_like(lo)
    for p, page in enumerate(pages):
        rows = min(P, L - p * P)
        for g in range(Hkv):
            lo[p, g], hi[p, g] = oselect.bounds(okv8.decode(mirror.codes[layer, 0, page, g, :rows]))
    return pages, lo, hi, mirror.scale[layer, 0][pages]


def check_bounds(cache, mirror):
    for layer in range(LAYERS):
        got = okv8.decode(cache.k_bounds[layer].view(torch.uint8).cpu().numpy())
        for b in range(B):
            pages, lo, hi, _ = boxes(mirror, layer, b)
            np.testing.assert_array_equal(got[pages], np.stack([lo, hi], 2))


def norm_rope(qkv, freqs, w, **pos):
    q, kk, v = (t.unflatten(2, (-1, dh)) for t in qkv.split([Hq * dh, Hkv * dh, Hkv * dh], 2))
    return eg.qk_norm_rope(q, kk, v, freqs, *w, **pos)


def one_step(cache, mirror, step, g, freqs, w):
    n = m + 1
    cache.reserve(i32([D + 1] * B))
    mirror.reserve([D + 1] * B)
    draft = (torch.randn((B, D, k, V), generator=g) * 4).cuda()
    step.draft(draft)
    step.build()
    keep = np.array([[[bool((int(x) >> j) & 1) for j in range(n)] for x in row[:, 0]] for row in step.tree["mask"].cpu().numpy()])
    trees = []
    for layer in range(LAYERS):
        qkv = torch.randn((B, n, (Hq + 2 * Hkv) * dh), generator=g).to(bf).cuda()
        q, kt, vt = norm_rope(qkv, freqs, w, pos_base=cache.kv_len, pos_off=step.tree["depth"])
        out, lse = step.attend_kv8(cache, layer, q, kt, vt, top=TOP, first=FIRST, last=LAST)
        trees.append((kt, vt))
        sel = step.sels[TOP].tolist()
        qn = f64(q)
        for b in range(B):
            pages, lo, hi, scale = boxes(mirror, layer, b)
            K, W = (np.concatenate([mirror.values(layer, i, b), f64(t[b])], 1) for i, t in enumerate((kt, vt)))
            for i in range(n):
                for g_ in range(Hkv):
                    heads = slice(g_ * G, (g_ + 1) * G)
                    s = oselect.scores(qn[b, i, heads], lo[:, g_], hi[:, g_], scale[:, g_])
                    want = oselect.choose(s, TOP, FIRST, LAST)
                    assert sel[b][i][g_] == want + [-1] * (TOP - len(want))
                    live = np.concatenate([np.isin(np.arange(mirror.kv[b]) // P, want), keep[b, i]])
                    x = qn[b, i, heads] @ K[g_][live].T * dh ** -0.5
                    p = np.exp(x - x.max(1, keepdims=True))
                    p /= p.sum(1, keepdims=True)
                    ref, A = p @ W[g_][live], p @ np.abs(W[g_][live])
                    # bf16's rounding, the weights' f16 (half a step is 2^-11), scores below 2^5 of 64 products in fp32, twice
                    tol = 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) + (2.0 ** -11 + 2 * 64 * 2.0 ** -23 * 2 ** 5) * A
                    assert (np.abs(f64(out[b, i, heads]) - ref) <= tol).all()
    row = step.tree["row"].cpu()
    flat = draft.cpu().view(B, D * k, V)
    target = torch.stack([torch.stack([flat[b, r] if r >= 0 else torch.randn(V, generator=g) for r in row[b].tolist()]) for b in range(B)])
    step.verify((target + 0.3 * torch.randn(target.shape, generator=g)).cuda())
    step.commit_kv8(cache, [t[0] for t in trees], [t[1] for t in trees])
    acc, path = step.accept_len.tolist(), step.path_nodes.tolist()
    for b in range(B):
        pos = [mirror.kv[b] + i for i in range(acc[b] + 1)]
        slots = [mirror.table[b][p // P] * P + p % P for p in pos]
        for layer, pair in enumerate(trees):
            for i, t in enumerate(pair):
                mirror.write(layer, i, f64(t[b])[:, path[b][:acc[b] + 1]].transpose(1, 0, 2), slots)
        mirror.kv[b] += acc[b] + 1
    cache.trim()
    mirror.release(mirror.kv)
    assert int(step.status) == 0


def test_prompts_steps_and_a_new_request():
    g = torch.Generator().manual_seed(78)
    cache, mirror = KV8Cache(B, Hkv, dh, P, N, MP, layers=LAYERS, bounds=True), Mirror()
    step = TreeStep(B, D, k, m, V, Hq, Hkv, dh, MP * P)
    freqs, _ = eg.rope_freqs(dh)
    w = [(1 + 0.3 * torch.randn(dh, generator=g)).to(bf).cuda() for _ in range(2)]
    prompt(cache, mirror, [85, 1, 64], g, freqs[:16])
    check_bounds(cache, mirror)
    for _ in range(5):
        one_step(cache, mirror, step, g, freqs, w)
        mirror.same_as(cache)
        check_bounds(cache, mirror)
    # request 2 ends, another one begins in its place with a prompt in two chunks
    cache.release(i32([-1, -1, 0]))
    mirror.release([-1, -1, 0])
    cache.kv_len[2] = 0
    mirror.kv[2] = 0
    prompt(cache, mirror, [0, 0, 21], g, freqs[:16])
    prompt(cache, mirror, [0, 3, 30], g, freqs[:16])
    check_bounds(cache, mirror)
    for _ in range(2):
        one_step(cache, mirror, step, g, freqs, w)
        mirror.same_as(cache)
        check_bounds(cache, mirror)
    # a reservation that is refused: nothing grows, the bounds stay
    before = [t.view(torch.uint8).clone() for t in cache.k_bounds]
    cache.reserve(i32([0, 0, 10 ** 6]), torch.empty(4, dtype=torch.int32, device="cuda"))
    cache.grow(i32([0, 0, 4]))
    assert all(torch.equal(a, t.view(torch.uint8)) for a, t in zip(before, cache.k_bounds)) and cache.kv_len.tolist() == mirror.kv


def test_a_node_of_the_tree_is_what_decoding_its_tokens_gives():
    """A path of the tree verified in one pass, and its tokens decoded one by one
    over a second cache: the same pages, outputs within their tolerance."""
    g = torch.Generator().manual_seed(9)
    caches = [KV8Cache(1, Hkv, dh, P, N, MP, bounds=True) for _ in range(2)]
    new = i32([100])
    x = torch.randn((2, 100, Hkv, dh), generator=g).to(bf).cuda()
    for c in caches:
        slots = torch.empty(100, dtype=torch.int32, device="cuda")
        c.reserve(new, slots)
        c.append(0, x[0], x[1], slots)
        c.grow(new)
    n = 4
    q = torch.randn((1, n, Hq, dh), generator=g).to(bf).cuda()
    kt, vt = (torch.randn((1, Hkv, n, dh), generator=g).to(bf).cuda() for _ in range(2))
    mask = eg.tree_mask(i32([[-1, 0, 1, 2]]))
    # three pages by score: the tokens of the path lie in the last, forced page
    tree_sel = caches[0].select(0, q, 4)
    tree_out, tree_lse = caches[0].attend_pages(0, q, kt, vt, mask, tree_sel)
    one, slot = i32([1]), torch.empty(1, dtype=torch.int32, device="cuda")
    alone = eg.tree_mask(i32([[-1]]))
    for i in range(n):
        c = caches[1]
        sel = c.select(0, q[:, i:i + 1].contiguous(), 4)
        assert torch.equal(sel[0, 0], tree_sel[0, i])
        out, lse = c.attend_pages(0, q[:, i:i + 1].contiguous(), kt[:, :, i:i + 1].contiguous(), vt[:, :, i:i + 1].contiguous(), alone, sel)
        # the earlier nodes' keys and values are in e4m3 by now: 2^-4 of each, on a score below 2^3 of them
        assert (out[0, 0] - tree_out[0, i]).abs().max() < 0.5 and (lse[0, 0] - tree_lse[0, i]).abs().max() < 0.5
        if i == 0:
            assert torch.equal(out[0, 0], tree_out[0, 0]) or (out[0, 0].float() - tree_out[0, 0].float()).abs().max() <= 2.0 ** -7 * tree_out[0, 0].float().abs().max()
        c.reserve(one, slot)
        c.append(0, kt[:, :, i].contiguous(), vt[:, :, i].contiguous(), slot)
        c.grow(one)
    assert int(caches[1].status) == 0


def test_a_step_in_a_graph():
    """select, attend, commit (with the bounds) and trim captured once and replayed:
    the same as the calls made one by one on a second cache."""
    g = torch.Generator().manual_seed(6)
    caches = [KV8Cache(B, Hkv, dh, P, N, MP, layers=LAYERS, bounds=True) for _ in range(2)]
    n, new = 9, i32([70, 5, 51])
    x = torch.randn((2, LAYERS, 126, Hkv, dh), generator=g).to(bf).cuda()
    for c in caches:
        slots = torch.empty(126, dtype=torch.int32, device="cuda")
        c.reserve(new, slots)
        for layer in range(LAYERS):
            c.append(layer, x[0, layer], x[1, layer], slots)
        c.grow(new)
    tree = [torch.randn((LAYERS, B, Hkv, n, dh), generator=g).to(bf).cuda() for _ in range(2)]
    q = torch.randn((B, n, Hq, dh), generator=g).to(bf).cuda()
    mask = eg.tree_mask(i32([[-1] + list(range(n - 1))] * B))
    acc, path = i32([2, 0, 3]), i32([[0, 1, 2, -1], [0, -1, -1, -1], [0, 4, 5, 6]])
    need = i32([D + 1] * B)
    out = [torch.empty_like(q) for _ in range(2)]
    sel = [torch.empty((B, n, Hkv, TOP), dtype=torch.int32, device="cuda") for _ in range(2)]
    lse = torch.empty((B, n, Hq), device="cuda")
    slots = torch.empty((B, n), dtype=torch.int32, device="cuda")

    def step(c, o, s):
        c.reserve(need)
        for layer in range(LAYERS):
            c.select(layer, q, TOP, out=s)
            c.attend_pages(layer, q, tree[0][layer], tree[1][layer], mask, s, out=o, lse=lse)
        c.commit(list(tree[0]), list(tree[1]), acc, path, slots, root=True)
        c.trim()

    step(caches[0], out[0], sel[0])
    step(caches[1], out[1], sel[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], out[0], sel[0])
    for _ in range(5):
        graph.replay()
        step(caches[1], out[1], sel[1])
        torch.cuda.synchronize()
        a, b = caches
        assert torch.equal(out[0], out[1]) and torch.equal(sel[0], sel[1])
        for name in ("kv_len", "page_count", "block_table", "free_count", "free_pages", "status"):
            assert torch.equal(getattr(a, name), getattr(b, name)), name
        for name in ("k_pages", "v_pages", "k_bounds"):
            assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(getattr(a, name), getattr(b, name)))
    assert int(caches[0].status) == 0 and caches[0].kv_len.tolist() == [70 + 18, 5 + 6, 51 + 24]


def test_two_calls_at_once():
    """Selection and attention of two layers on two streams, a workspace each: what
    one after the other gives."""
    g = torch.Generator().manual_seed(11)
    cache = KV8Cache(2, 2, 128, 16, 700, 330, layers=2, bounds=True)
    new = i32([5000, 3333])
    slots = torch.empty(8333, dtype=torch.int32, device="cuda")
    cache.reserve(new, slots)
    for layer in range(2):
        kv = torch.randn((2, 8333, 2, 128), generator=g).to(bf).cuda()
        cache.append(layer, kv[0], kv[1], slots)
    cache.grow(new)
    for n, heads in ((1, 8), (40, 8), (40, 32)):
        q, kt, vt = (torch.randn(s, generator=g).to(bf).cuda() for s in ((2, n, heads, 128), (2, 2, n, 128), (2, 2, n, 128)))
        mask = eg.tree_mask(i32([[-1] + list(range(n - 1))] * 2))

        def run(layer, ws, out, lse):
            sel = cache.select(layer, q, 12, workspace=ws)
            return cache.attend_pages(layer, q, kt, vt, mask, sel, out=out, lse=lse, workspace=ws)

        spaces = [eg.Workspace("cuda") for _ in range(2)]
        want = [tuple(t.clone() for t in run(layer, spaces[layer], None, None)) for layer in range(2)]
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in range(2)]
        outs = [(torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])) for _ in range(2)]
        for _ in range(20):
            for layer in range(2):
                with torch.cuda.stream(side[layer]):
                    run(layer, spaces[layer], *outs[layer])
        torch.cuda.synchronize()
        for layer in range(2):
            assert torch.equal(outs[layer][0], want[layer][0]) and torch.equal(outs[layer][1], want[layer][1])
    assert int(cache.status) == 0


def test_bounds_after_a_cut():
    """kv_len set back: the last page's bounds stay wider until the request grows."""
    g = torch.Generator().manual_seed(12)
    cache = KV8Cache(1, 1, 64, 16, 8, 8, bounds=True)
    x = torch.randn((40, 1, 64), generator=g).to(bf).cuda()
    slots = torch.empty(40, dtype=torch.int32, device="cuda")
    cache.reserve(i32([40]), slots)
    cache.append(0, x, x, slots)
    cache.grow(40)
    cache.kv_len.fill_(19)
    cache.trim()
    slot = torch.empty(1, dtype=torch.int32, device="cuda")
    cache.reserve(i32([1]), slot)
    cache.append(0, x[:1] * 3, x[:1], slot)
    cache.grow(1)
    page = int(cache.block_table[0, 1])
    rows = okv8.decode(cache.k_pages[0].view(torch.uint8).cpu().numpy()[page, 0, :4])
    got = okv8.decode(cache.k_bounds[0].view(torch.uint8).cpu().numpy()[page, 0])
    np.testing.assert_array_equal(got, np.stack(oselect.bounds(rows)))


def test_a_cache_with_bounds_checks_its_head_dimension():
    with pytest.raises(eg.EagleError):
        KV8Cache(1, 1, 80, 16, 4, 4, bounds=True)


def test_steps_of_two_sizes_keep_their_lists():
    """attend_kv8 with another `top` does not take the list of a captured one away."""
    g = torch.Generator().manual_seed(13)
    cache = KV8Cache(B, Hkv, dh, P, N, MP, bounds=True)
    slots = torch.empty(150, dtype=torch.int32, device="cuda")
    cache.reserve(i32([50] * B), slots)
    x = torch.randn((150, Hkv, dh), generator=g).to(bf).cuda()
    cache.append(0, x, x, slots)
    cache.grow(50)
    step = TreeStep(B, D, k, m, V, Hq, Hkv, dh, MP * P)
    step.draft((torch.randn((B, D, k, V), generator=g) * 4).cuda())
    step.build()
    q, kt, vt = (torch.randn(s, generator=g).to(bf).cuda() for s in ((B, m + 1, Hq, dh), (B, Hkv, m + 1, dh), (B, Hkv, m + 1, dh)))
    want = [t.clone() for t in step.attend_kv8(cache, 0, q, kt, vt, top=2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.attend_kv8(cache, 0, q, kt, vt, top=2)
    step.attend_kv8(cache, 0, q, kt, vt, top=4)
    assert step.sels[2].shape[-1] == 2 and step.sels[4].shape[-1] == 4
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.attn_out, want[0]) and torch.equal(step.lse, want[1])
