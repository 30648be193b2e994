"""The decoding loop over the 8-bit cache against causal attention.

Each token has fixed raw q, k and v (a layer's tables), so what a tree row must
give is known without any cache: causal attention in fp64 over the tokens that
are committed and the row's ancestors, at their positions.  k and v are
multiples of 1/4 up to 2, which e4m3 holds exactly at every scale that such
numbers get, and the rotations are quarter turns, so the cache rounds nothing
and the attention's own tolerance is all that is allowed:
  2^-8 |o| (1 + 2^-8) bf16's rounding, (2^-11 + w) A with w = 2 (dh 2^-23 smax +
  2^-21) + 2 N 2^-24 for f16 weights, fp32 scores, ex2 and sums (A: the weighted
  sum of |v|, smax: the row's largest sum of |q k| scale), and f16's subnormal
  weights: 2^-31 |v_k| 2^(max e - e_k) for each of N keys, |v| <= 2 and blocks of
  such v within 2^5 of one another: N 2^-25."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_eagle_gb300 as eg
from oracle import kv8 as okv8
from oracle import rope as orope
from tree_speculative_decoding_eagle_gb300.cache import KV8Cache
from tree_speculative_decoding_eagle_gb300.step import TreeStep

pytestmark = pytest.mark.gpu
D, k, m, V, Hq, Hkv, dh, P, LAYERS = 3, 4, 15, 512, 4, 2, 64, 16, 2
MP = 12
bf = torch.bfloat16
FREQS = (math.pi / 2) * (np.arange(16) % 4 + 1.0)     # quarter turns: 1, 2, 3, 4 of them a position


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


class Model:
    """Raw q, k and v of every token, a table for each layer."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        draw = lambda h: torch.randint(-8, 9, (LAYERS, V, h, dh), generator=g).float() / 4
        self.q, self.k, self.v = draw(Hq), draw(Hkv), draw(Hkv)

    def qkv(self, layer, tok):
        t = torch.as_tensor(tok).long()
        return (x[layer][t].to(bf).cuda() for x in (self.q, self.k, self.v))

    def check(self, out, layer, seq, tok, parent, weights=2.0 ** -11, half=2.0 ** -8):
        """Every node's row against causal attention over seq and its ancestors;
        `weights`, `half`: half a step of the types that weights and outputs are rounded to."""
        n, L = len(tok), len(seq)
        live = np.zeros((n, n), bool)
        depth = np.zeros(n, int)
        for i in range(n):
            if i:
                live[i] = live[parent[i]]
                depth[i] = depth[parent[i]] + 1
            live[i, i] = True
        at = lambda x, t, p: orope.rotate(x[layer][t].double().numpy(), p, FREQS)
        every = list(seq) + list(tok)
        pos = np.concatenate([np.arange(L), L + depth])
        Q, K, W = at(self.q, list(tok), L + depth), at(self.k, every, pos), self.v[layer][every].double().numpy()
        live = np.hstack([np.ones((n, L), bool), live])
        for h in range(Hq):
            key, val = K[:, h // (Hq // Hkv)], W[:, h // (Hq // Hkv)]
            s = np.where(live, Q[:, h] @ key.T * dh ** -0.5, -np.inf)
            smax = (np.abs(Q[:, h]) @ np.abs(key).T * dh ** -0.5).max(1, keepdims=True)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            ref, A = p @ val, p @ np.abs(val)
            w = 2 * (dh * 2.0 ** -23 * smax + 2.0 ** -21) + 2 * (L + n) * 2.0 ** -24
            tol = half * np.abs(ref) * (1 + half) + (weights + w) * A + (L + n) * 2.0 ** -25
            assert (np.abs(out[:, h] - ref) <= tol).all(), (layer, L, float((np.abs(out[:, h] - ref) / tol).max()))


class Loop:
    """Requests that decode: their committed tokens and their next root."""

    def __init__(self, lens, seed, rule):
        self.g = torch.Generator().manual_seed(seed)
        self.rule, self.B, self.model = rule, len(lens), Model(seed)
        self.cache = KV8Cache(self.B, Hkv, dh, P, self.B * MP, MP, layers=LAYERS)
        self.step = TreeStep(self.B, D, k, m, V, Hq, Hkv, dh, MP * P)
        self.freqs = torch.from_numpy(FREQS).cuda()
        self.seqs = [torch.randint(0, V, (n,), generator=self.g).tolist() for n in lens]
        self.roots = torch.randint(0, V, (self.B,), generator=self.g).tolist()
        self.prompts(lens)

    def prompts(self, lens):
        c, toks = self.cache, sum(self.seqs, [])
        slots = torch.empty(len(toks), dtype=torch.int32, device="cuda")
        c.reserve(i32(lens), slots)
        pos = i32([[p for n in lens for p in range(n)]])
        for layer in range(LAYERS):
            q, kk, v = (t[None] for t in self.model.qkv(layer, toks))
            _, kt, vt = eg.rope(q, kk, v, self.freqs, pos_off=pos)
            c.append(layer, kt[0].transpose(0, 1), vt[0].transpose(0, 1), slots)
        c.grow(i32(lens))

    def one(self):
        c, step, B = self.cache, self.step, self.B
        c.reserve(i32([D + 1] * B))
        draft = (torch.randn((B, D, k, V), generator=self.g) * 4).cuda()
        step.draft(draft)
        step.build(i32(self.roots))
        tok, parent, row = (step.tree[x].tolist() for x in ("tok", "parent", "row"))
        trees = []
        for layer in range(LAYERS):
            q, kk, v = self.model.qkv(layer, tok)
            q, kt, vt = eg.rope(q, kk, v, self.freqs, pos_base=c.kv_len, pos_off=step.tree["depth"])
            out, _ = step.attend_kv8(c, layer, q, kt, vt)
            trees.append((kt, vt))
            for b in range(B):
                self.model.check(f64(out[b]), layer, self.seqs[b], tok[b], parent[b])
        flat = draft.cpu().view(B, D * k, V)
        target = torch.stack([torch.stack([flat[b, r] if r >= 0 else torch.randn(V, generator=self.g) for r in row[b]])
                              for b in range(B)])
        step.verify((target + 0.3 * torch.randn(target.shape, generator=self.g)).cuda())
        kts, vts = [t[0] for t in trees], [t[1] for t in trees]
        if self.rule == "commit stores the root":
            step.commit_kv8(c, kts, vts)
        else:                                          # the caller stores it, then the path after it
            slots = torch.empty(B, dtype=torch.int32, device="cuda")
            c.reserve(i32([1] * B), slots)
            for layer in range(LAYERS):
                c.append(layer, kts[layer][:, :, 0], vts[layer][:, :, 0], slots)
            c.grow(i32([1] * B))
            c.commit(kts, vts, step.accept_len, step.path_nodes)
        c.trim()
        acc, path, new = step.accept_len.tolist(), step.path_nodes.tolist(), step.out_tokens.tolist()
        for b in range(B):
            self.seqs[b] += [tok[b][i] for i in path[b][:acc[b] + 1]]
            self.roots[b] = new[b][acc[b]]
        assert c.kv_len.tolist() == [len(s) for s in self.seqs]
        assert c.page_count.tolist() == [-(-len(s) // P) for s in self.seqs]
        assert int(c.status) == 0 and int(step.status) == 0
        return sum(acc)


@pytest.mark.parametrize("rule", ["commit stores the root", "the caller stores the root"])
def test_every_row_of_every_step_is_causal_attention(rule):
    loop = Loop([37, 0, 64], 3, rule)
    assert sum(loop.one() for _ in range(8)) > 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,n,heads,d,page,depth", [(1, 1, 1, 64, 16, 1), (4, 20, 3, 64, 16, 6), (3, 61, 40, 128, 64, 7),
                                                    (2, 128, 2, 128, 16, 64), (70, 8, 8, 64, 32, 5)])
def test_commit_with_the_root(B, n, heads, d, page, depth, dtype):
    rng = np.random.default_rng(B * n)
    mp = 200 // page + 6
    N = B * mp + 3
    kv_len = rng.integers(0, 200, B)
    kv_len[0] = page - 1                              # the root fills a page
    kv_len[-1] = 0                                    # nothing before the root
    acc = rng.integers(0, min(depth, n - 1) + 1, B)
    acc[0] = min(depth, n - 1)
    path = np.full((B, depth + 1), -1)
    for b in range(B):
        path[b, 0] = 0
        path[b, 1:acc[b] + 1] = 1 + rng.permutation(n - 1)[:acc[b]]
    table = rng.permutation(N)[:B * mp].reshape(B, mp)
    tree = torch.from_numpy(rng.standard_normal((2, B, heads, n, d)) * 2.0 ** rng.integers(-2, 3, (2, B, heads, n, 1))).to(dtype)
    codes = [rng.integers(0, 0x70, (N, heads, page, d)).astype(np.uint8) for _ in range(2)]
    scale = [2.0 ** rng.integers(-9, -3, (N, heads)).astype(np.float64) for _ in range(2)]
    gpu = [torch.from_numpy(c.copy()).cuda().view(torch.float8_e4m3fn) for c in codes]
    gscale = [torch.from_numpy(s).float().cuda() for s in scale]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).int().cuda()
    kl, status = dev(kv_len), torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = eg.kv8_commit(tree[0].cuda(), tree[1].cuda(), dev(acc), dev(path), *gpu, *gscale, kl, dev(table), status=status,
                          root=True)
    assert int(status) == 0
    assert kl.tolist() == (kv_len + acc + 1).tolist()
    want = np.full((B, n), -1)
    for b in range(B):
        pos = kv_len[b] + np.arange(acc[b] + 1)
        nodes = path[b, :acc[b] + 1]
        want[b, nodes] = pos
        where = table[b, pos // page] * page + pos % page
        for src, c, s in zip(tree, codes, scale):
            okv8.append(src[b].double().numpy()[:, nodes].transpose(1, 0, 2), where, c, s)
    assert slots.tolist() == want.tolist()
    for t, s, c, w in zip(gpu, gscale, codes, scale):
        np.testing.assert_array_equal(s.double().cpu().numpy(), w)
        np.testing.assert_array_equal(t.view(torch.uint8).cpu().numpy(), c)


@pytest.mark.parametrize("fault", ["root", "node 0", "node n", "accept", "length", "page", "full"])
def test_a_refused_commit_with_the_root_leaves_its_sequence_alone(fault):
    n, mp, page = 6, 4, 16
    kv_len, acc, path = np.array([30, 20]), np.array([2, 2]), np.array([[0, 1, 2, -1]] * 2)
    table = np.arange(8).reshape(2, 4)
    if fault == "root":
        path[0, 0] = 3
    elif fault == "node 0":
        path[0, 2] = 0
    elif fault == "node n":
        path[0, 1] = n
    elif fault == "accept":
        acc[0] = -1
    elif fault == "length":
        kv_len[0] = -1
    elif fault == "page":
        table[0, 2] = 9                               # positions 30, 31 are mapped, 32 is not
    elif fault == "full":
        kv_len[0] = mp * page - 2
    dev = lambda t: torch.from_numpy(t).int().cuda()
    pool = lambda: torch.full((9, 2, page, 64), 7, dtype=torch.uint8, device="cuda")
    kp, vp, ks, vs = pool(), pool(), torch.ones((9, 2), device="cuda"), torch.ones((9, 2), device="cuda")
    x = torch.randn((2, 2, n, 64), device="cuda")
    kl, status = dev(kv_len), torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.kv8_commit(x, x, dev(acc), dev(path), kp, vp, ks, vs, kl, dev(table), status=status, root=True)
    assert int(status) == -1 and kl.tolist() == [int(kv_len[0]), 23]
    mine = int(table[1, 1])
    others = [p for p in range(9) if p != mine]
    assert (kp[others] == 7).all() and (vp[others] == 7).all() and (ks[others] == 1).all() and (kp[mine, :, 7:] == 7).all()
    assert not (kp[mine, :, 4:7] == 7).all()


def test_the_loop_in_a_graph():
    """reserve, attend, commit with the root and trim captured once and
    replayed: the same as the calls made one by one on a second cache."""
    B, n = 2, 9
    g = torch.Generator().manual_seed(5)
    caches = [KV8Cache(B, Hkv, dh, P, 40, MP, layers=LAYERS) for _ in range(2)]
    tree = [torch.randn((LAYERS, B, Hkv, n, dh), generator=g).to(bf).cuda() for _ in range(2)]
    q = torch.randn((B, n, Hq, dh), generator=g).to(bf).cuda()
    mask = eg.tree_mask(i32([[-1] + list(range(n - 1))] * B))
    acc, path, need = i32([2, 0]), i32([[0, 1, 2, -1], [0, -1, -1, -1]]), i32([D + 1] * B)
    out = [torch.empty_like(q) for _ in range(2)]
    lse, slots = torch.empty((B, n, Hq), device="cuda"), torch.empty((B, n), dtype=torch.int32, device="cuda")

    def step(c, o):
        c.reserve(need)
        for layer in range(LAYERS):
            c.attend(layer, q, tree[0][layer], tree[1][layer], mask, out=o, lse=lse)
        c.commit(list(tree[0]), list(tree[1]), acc, path, slots, root=True)
        c.trim()

    step(caches[0], out[0])
    step(caches[1], out[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0], out[0])
    for _ in range(9):
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
    assert int(caches[0].status) == 0 and caches[0].kv_len.tolist() == [30, 10]


@pytest.mark.parametrize("paged", [False, True])
def test_the_16_bit_loop_follows_the_same_rule(paged):
    """eagle_tree_attn(_paged) with the positions before the root; the caller
    stores the root's row; eagle_kv_commit with one position more."""
    B, n, Lmax = 2, 6, 64
    model, g = Model(11), torch.Generator().manual_seed(11)
    dtype = bf if paged else torch.float32
    parent = [-1, 0, 0, 1, 3, 2]
    path = i32([[0, 1, 3, 4]] * B)
    mask, depth = eg.tree_mask(i32([parent] * B)), i32([[0, 1, 1, 2, 3, 2]] * B)
    freqs = torch.from_numpy(FREQS).cuda()
    shape = (B * Lmax // P, Hkv, P, dh) if paged else (B, Hkv, Lmax, dh)
    kc, vc = (torch.full(shape, 7.0, dtype=dtype, device="cuda") for _ in range(2))
    table = torch.randperm(B * Lmax // P, generator=g).view(B, -1).int().cuda() if paged else None
    seqs, kv_len = [[], []], torch.zeros(B, dtype=torch.int32, device="cuda")
    for step in range(7):
        tok = torch.randint(0, V, (B, n), generator=g)
        q, kk, v = (t.to(dtype) for t in model.qkv(0, tok))
        q, kt, vt = eg.rope(q, kk, v, freqs, pos_base=kv_len, pos_off=depth)
        if paged:
            out, _ = eg.tree_attn_paged(q, kc, vc, table, kv_len, kt, vt, mask)
        else:
            out, _ = eg.tree_attn(q, kc, vc, kv_len, kt, vt, mask)
        acc = [step % 4, (step + 2) % 4]
        for b in range(B):
            model.check(f64(out[b]), 0, seqs[b], tok[b].tolist(), parent, weights=2.0 ** -8 if paged else 0.0, half=2.0 ** -8 if paged else 2.0 ** -24)
            at = int(kv_len[b])
            for c, t in ((kc, kt), (vc, vt)):
                if paged:
                    c[int(table[b, at // P]), :, at % P] = t[b, :, 0]
                else:
                    c[b, :, at] = t[b, :, 0]
            seqs[b] += [int(tok[b, i]) for i in [0, 1, 3, 4][:acc[b] + 1]]
        kv_len += 1
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        eg.kv_commit(kt, vt, i32(acc), path, kc, vc, kv_len, block_table=table, status=status)
        assert int(status) == 0 and kv_len.tolist() == [len(s) for s in seqs]
