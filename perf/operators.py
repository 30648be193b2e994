"""The serving step over a paged cache in 8 bits: its operators' cases, their plain forms and what they cost.

    pages   the pages that new tokens need are mapped from a free list and the slot of every new token is listed; then the
            pages past each request's length are given back, as after a step that accepted none of its draft
    rope    rotary positions of q and k, into the layouts that the tree attention reads
    write   keys and values into pages of e4m3 numbers with one power-of-two scale for each page and head: a prompt's or
            single tokens by their slots ("append"), or the accepted path of a draft tree ("commit")
    attend  tree-masked attention of draft nodes (or of single tokens) over that cache

With `own` the calls are the framework's, without it elementary torch operations in 32 bits (angles in 64).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
E_MIN, E_MAX = -64, 64          # exponents that a block's scale may take


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # one request's step: room for a path of 6 accepted tokens and the bonus; launch latency is all there is
        {"name": "pages one request", "kind": "pages", "B": 1, "page": 16, "kv_max": 2048, "new_max": 7, "T": 7},
        # a scheduler's mixed batch: many requests decoding, others with a chunk of their prompt
        {"name": "pages 512 requests", "kind": "pages", "B": 512, "page": 16, "kv_max": 4096, "new_max": 127, "T": 32768},
        # the tree of llama2-7b-b1: 61 nodes, every head with its own keys
        {"name": "rope llama2-7b-b1", "kind": "rope", "B": 1, "n": 61, "Hq": 32, "Hkv": 32, "dh": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "dtype": "bf16", "kv_max": 2048},
        # the trees of gpt-oss-20b-b64: grouped heads, frequencies stretched for long contexts, far positions
        {"name": "rope gpt-oss-20b-b64", "kind": "rope", "B": 64, "n": 61, "Hq": 64, "Hkv": 8, "dh": 64, "rot": 64,
         "interleaved": False, "scaling": "yarn", "dtype": "bf16", "kv_max": 131072},
        # a prompt of odd length, interleaved pairs, a quarter of the head rotated, in 32 bits
        {"name": "rope prompt f32", "kind": "rope", "B": 1, "n": 8191, "Hq": 40, "Hkv": 40, "dh": 128, "rot": 32,
         "interleaved": True, "scaling": "linear", "dtype": "f32", "kv_max": 0},
        # the accepted paths of llama2-13b-b8's trees
        {"name": "write commit 13b-b8", "kind": "write", "form": "commit", "B": 8, "n": 51, "D": 6, "Hkv": 40, "dh": 128,
         "page": 16, "kv_max": 4096, "T": 0, "dtype": "bf16"},
        # one token of each of 64 requests (plain decoding)
        {"name": "write tokens 64", "kind": "write", "form": "append", "B": 64, "n": 0, "D": 0, "Hkv": 8, "dh": 64,
         "page": 64, "kv_max": 1024, "T": 64, "dtype": "bf16"},
        # the prompts of llama2-70b-b16, whole
        {"name": "write prompts 70b-b16", "kind": "write", "form": "append", "B": 16, "n": 0, "D": 0, "Hkv": 8, "dh": 128,
         "page": 64, "kv_max": 0, "T": 65536, "dtype": "bf16"},
        # the framework's headline workload: one sequence, 61 nodes, all heads with their own keys, small pages
        {"name": "attend llama2-7b-b1", "kind": "attend", "B": 1, "n": 61, "Hq": 32, "Hkv": 32, "dh": 128, "page": 16,
         "L": 2048, "L_min": 2048},
        # grouped queries, 8 to a KV head: arithmetic counts
        {"name": "attend llama2-70b-b16", "kind": "attend", "B": 16, "n": 49, "Hq": 64, "Hkv": 8, "dh": 128, "page": 64,
         "L": 4096, "L_min": 4096},
        # the largest: 64 sequences of 8192 tokens, head dimension 64
        {"name": "attend gpt-oss-20b-b64", "kind": "attend", "B": 64, "n": 61, "Hq": 64, "Hkv": 8, "dh": 64, "page": 128,
         "L": 8192, "L_min": 8192},
        # single tokens of 64 requests with ragged lengths: the cache's bytes are all that counts
        {"name": "attend tokens 64", "kind": "attend", "B": 64, "n": 1, "Hq": 64, "Hkv": 8, "dh": 128, "page": 64,
         "L": 8192, "L_min": 1024},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["pages", "rope", "write", "write", "attend", "attend", "attend"])
    if kind == "pages":
        B = _log(rng, 1, 512)
        new_max = _log(rng, 1, 127)
        return {"kind": kind, "B": B, "page": rng.choice([16, 32, 64, 128, 256]), "kv_max": _log(rng, 1, 4096),
                "new_max": new_max, "T": min(32768, B * new_max)}
    if kind == "rope":
        B = _log(rng, 1, 64)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        dh = rng.choice([64, 128])
        Hkv, G = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 4, 5, 8])
        Hq = min(64, Hkv * G) // Hkv * Hkv
        most = 80e6 / (B * (Hq + 2 * Hkv) * dh * (4 if dtype == "f32" else 2))
        return {"kind": kind, "B": B, "n": _log(rng, 1, max(1, min(8191, int(most)))), "Hq": Hq, "Hkv": Hkv, "dh": dh,
                "rot": rng.choice([dh, dh, dh // 2, dh // 4, 20]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "yarn", "bands"]), "dtype": dtype, "kv_max": _log(rng, 1, 131072)}
    if kind == "write":
        form = rng.choice(["append", "append", "commit"])
        B, Hkv, dh = _log(rng, 1, 64), rng.choice([1, 2, 4, 8, 16, 40]), rng.choice([64, 128])
        c = {"kind": kind, "form": form, "B": B, "n": 0, "D": 0, "Hkv": Hkv, "dh": dh, "page": rng.choice([16, 32, 64, 128, 256]),
             "kv_max": _log(rng, 1, 1024), "T": 0, "dtype": rng.choice(["bf16", "bf16", "f32"])}
        if form == "commit":
            c["n"], c["D"] = rng.randint(8, 61), rng.randint(1, 7)
        else:
            c["T"] = max(B, _log(rng, B, max(B + 1, int(3e7 / (Hkv * dh)))))
        return c
    dh = rng.choice([64, 128])
    Hkv, G = rng.choice([1, 2, 4, 8, 32, 40]), rng.choice([1, 1, 2, 4, 5, 8])
    Hq = min(64, Hkv * G) // Hkv * Hkv
    n = rng.choice([1, 1, _log(rng, 2, 16), rng.randint(17, 128)])
    B = _log(rng, 1, 64)
    L = _log(rng, 1, 8192)
    while B * L * n * Hq * dh > 64 * 8192 * 61 * 64 * 64 * 0.5 or B * L * Hkv * dh > 64 * 8192 * 8 * 128:
        L = max(1, L // 2)
        B = max(1, B - B // 4)
    return {"kind": kind, "B": B, "n": n, "Hq": Hq, "Hkv": Hkv, "dh": dh, "page": rng.choice([16, 32, 64, 128, 256]),
            "L": L, "L_min": rng.choice([0, L, (L + 1) // 2])}


# ---- what a program has in hand -------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(g, lo, hi, size):
    """Whole numbers of lo..hi."""
    return torch.randint(lo, hi + 1, size, generator=g, device=DEV, dtype=torch.int32)


def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _block_exponent(amax):
    """The least e with amax <= 448 * 2^e, within E_MIN..E_MAX."""
    m, e = torch.frexp(amax)                       # amax = m * 2^e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)            # 448 = 0.875 * 2^9
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _random_pool(g, num_pages, Hkv, page, dh):
    """Pages of N(0, 1) rows times a magnitude of the page and head, in e4m3 with their scales."""
    x = torch.randn((num_pages, Hkv, page, dh), generator=g, device=DEV)
    x = x * torch.exp2(torch.randn((num_pages, Hkv, 1, 1), generator=g, device=DEV) * 0.5)
    scale = torch.exp2(_block_exponent(x.abs().amax((2, 3))).float())
    return (x / scale[:, :, None, None]).to(torch.float8_e4m3fn), scale


def _tree_mask(g, B, n):
    """Ancestor masks [B, n, ceil(n/64)] of random trees (parent before child): uint64 words as int64."""
    keep = torch.eye(n, dtype=torch.bool, device=DEV).repeat(B, 1, 1)
    up = torch.rand((B, n), generator=g, device=DEV)
    for i in range(1, n):
        lo = max(0, i - 8)
        parent = (lo + (up[:, i] * (i - lo)).long()).clamp(max=i - 1)
        keep[:, i] |= keep[torch.arange(B, device=DEV), parent]
    W = (n + 63) // 64
    bits = torch.zeros((B, n, W * 64), dtype=torch.int64, device=DEV)
    bits[:, :, :n] = keep.long()
    return (bits.view(B, n, W, 64) << torch.arange(64, device=DEV)).sum(3).contiguous(), keep


def _tables(g, kv_len, page, max_pages, num_pages):
    B = kv_len.shape[0]
    perm = torch.randperm(num_pages, generator=g, device=DEV)[:B * max_pages].to(torch.int32).view(B, max_pages)
    used = (kv_len[:, None] + page - 1) // page > torch.arange(max_pages, device=DEV)[None]
    return torch.where(used, perm, torch.full_like(perm, -1)).contiguous()


def _prepare_pages(case, g):
    B, page = case["B"], case["page"]
    kv = _ints(g, 0, case["kv_max"], (B,))
    new = _ints(g, 1, case["new_max"], (B,))
    over = torch.cumsum(new, 0) - case["T"]                       # the batch's token budget
    new = (new - over.clamp(min=0)).clamp(min=0).to(torch.int32)
    max_pages = (case["kv_max"] + case["new_max"] + page - 1) // page
    count = ((kv + page - 1) // page).to(torch.int32)
    num_pages = B * max_pages + 8
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = order[:B * max_pages].view(B, max_pages)
    mapped = torch.arange(max_pages, device=DEV)[None] < count[:, None]
    used = torch.zeros(num_pages, dtype=torch.bool, device=DEV)
    used[table[mapped].long()] = True
    free = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    rest = order[~used[order.long()]]
    free[:rest.shape[0]] = rest
    return {"kv_len": kv, "new_len": new, "table": torch.where(mapped, table, torch.full_like(table, -1)).contiguous(),
            "count": count, "free": free, "free_count": torch.tensor([rest.shape[0]], dtype=torch.int32, device=DEV),
            "slots": torch.empty(case["T"], dtype=torch.int32, device=DEV),
            "starts": torch.empty(B + 1, dtype=torch.int32, device=DEV),
            "status": torch.zeros(1, dtype=torch.int32, device=DEV)}


def _frequencies(case):
    """inv_freq [rot/2] in 64 bits and the factor on cos and sin."""
    rot, theta = case["rot"], 10000.0
    f = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    turns = 4096 * f / (2 * math.pi)               # turns over the context that the model was trained on
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "bands":                 # wave lengths past the trained context stretched, short ones kept
        return f / 8.0 + (f - f / 8.0) * np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1), 1.0
    if case["scaling"] == "yarn":                  # the ramp is linear in the pair's index
        at = lambda r: rot * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / 32.0 * ramp + f * (1 - ramp), 0.1 * math.log(32.0) + 1.0
    return f, 1.0


def _prepare_rope(case, g):
    B, n, Hq, Hkv, dh = (case[k] for k in ("B", "n", "Hq", "Hkv", "dh"))
    qkv = torch.randn((B, n, (Hq + 2 * Hkv) * dh), generator=g, device=DEV).to(_type(case))    # one fused projection
    f, factor = _frequencies(case)
    kv = _ints(g, 1, max(1, case["kv_max"]), (B,))
    depth = None
    if case["kv_max"]:                             # a tree: positions from the nodes' depths; a prompt: 0, 1, 2 ...
        depth = torch.sort(_ints(g, 0, 6, (B, n)), dim=1).values.to(torch.int32)
        depth[:, 0] = 0
    else:
        kv = torch.ones_like(kv)
    q, k, v = qkv.split([Hq * dh, Hkv * dh, Hkv * dh], dim=2)
    return {"q": q.unflatten(2, (Hq, dh)), "k": k.unflatten(2, (Hkv, dh)), "v": v.unflatten(2, (Hkv, dh)), "kv_len": kv,
            "depth": depth, "inv_freq": torch.from_numpy(f).to(DEV), "factor": factor,
            "interleaved": case["interleaved"], "q_out": torch.empty((B, n, Hq, dh), dtype=qkv.dtype, device=DEV),
            "k_out": torch.empty((B, Hkv, n, dh), dtype=qkv.dtype, device=DEV),
            "v_out": torch.empty((B, Hkv, n, dh), dtype=qkv.dtype, device=DEV)}


def _prepare_write(case, g):
    B, Hkv, dh, page, T = (case[k] for k in ("B", "Hkv", "dh", "page", "T"))
    t = _type(case)
    s = {"form": case["form"], "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if case["form"] == "commit":
        n, D = case["n"], case["D"]
        kv = _ints(g, 1, case["kv_max"], (B,))
        s["accept"] = _ints(g, 0, D, (B,))
        path = 1 + torch.argsort(torch.rand((B, n - 1), generator=g, device=DEV), dim=1)[:, :D]
        path = torch.cat([torch.zeros((B, 1), dtype=path.dtype, device=DEV), torch.sort(path, dim=1).values], 1)
        past = torch.arange(D + 1, device=DEV)[None] > s["accept"][:, None]
        s["path"] = torch.where(past, torch.full_like(path, -1), path).to(torch.int32).contiguous()
        new = torch.full((B,), D, dtype=torch.int32, device=DEV)
        s["k"], s["v"] = (torch.randn((B, Hkv, n, dh), generator=g, device=DEV).to(t) for _ in range(2))
        s["slots"] = torch.empty((B, n), dtype=torch.int32, device=DEV)
        most = case["kv_max"] + D
    else:
        kv = _ints(g, 0, case["kv_max"], (B,))
        # the budget shared out: one token for each, the rest by random shares (whole prompts of like lengths)
        share = torch.rand(B, generator=g, device=DEV) + 1.0
        new = (share / share.sum() * (T - B)).to(torch.int32) + 1
        new[0] += T - new.sum()
        most = int((kv + new).max())
        s["k"], s["v"] = (torch.randn((T, Hkv, dh), generator=g, device=DEV).to(t) for _ in range(2))
    max_pages = (most + page - 1) // page
    need = (kv + new + page - 1) // page
    num_pages = T // page + B * ((case["kv_max"] + case["D"]) // page + 2) + 8
    ends = torch.cumsum(need, 0)
    at = (ends - need)[:, None] + torch.arange(max_pages, device=DEV)[None]
    perm = torch.randperm(num_pages, generator=g, device=DEV)
    table = torch.where(at < ends[:, None], perm[at.clamp(max=num_pages - 1)], torch.full_like(at, -1)).to(torch.int32)
    s["table"] = table.contiguous()
    s["kp"], s["ks"] = _random_pool(g, num_pages, Hkv, page, dh)
    s["vp"], s["vs"] = _random_pool(g, num_pages, Hkv, page, dh)
    if case["form"] == "commit":
        s["kv_len0"], s["kv_len"] = kv, kv.clone()
    else:
        starts = torch.cumsum(new, 0) - new
        b = torch.repeat_interleave(torch.arange(B, device=DEV), new.long(), output_size=T)
        pos = (kv[b] + torch.arange(T, device=DEV) - starts[b]).long()
        s["slots"] = (table[b, pos // page].long() * page + pos % page).to(torch.int32)
    return s


def _prepare_attend(case, g):
    B, n, Hq, Hkv, dh, page = (case[k] for k in ("B", "n", "Hq", "Hkv", "dh", "page"))
    kv = _ints(g, case["L_min"], case["L"], (B,))
    max_pages = (case["L"] + page - 1) // page
    num_pages = B * max_pages + 4
    s = {"kv_len": kv, "table": _tables(g, kv, page, max_pages, num_pages), "L": case["L"]}
    s["kp"], s["ks"] = _random_pool(g, num_pages, Hkv, page, dh)
    s["vp"], s["vs"] = _random_pool(g, num_pages, Hkv, page, dh)
    # queries strong enough for a peaked softmax, as a trained model's are
    s["q"] = (torch.randn((B, n, Hq, dh), generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    s["kt"], s["vt"] = (torch.randn((B, Hkv, n, dh), generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    s["mask"], s["keep"] = _tree_mask(g, B, n)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((B, n, Hq), dtype=torch.float32, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    s["scratch"] = {}                              # where a program keeps the operator's workspace
    return s


_PREPARE = {"pages": _prepare_pages, "rope": _prepare_rope, "write": _prepare_write, "attend": _prepare_attend}


def prepare(case, seed):
    s = _PREPARE[case["kind"]](case, _gen(seed))
    s["kind"], s["page"] = case["kind"], case.get("page")
    return s


# ---- one pass -------------------------------------------------------------------

def _plain_pages(s):
    P, kv, new, count, table, free, fc = s["page"], s["kv_len"], s["new_len"], s["count"], s["table"], s["free"], s["free_count"]
    B, cols = table.shape
    col = torch.arange(cols, device=DEV)[None]
    need = torch.maximum((kv + new + P - 1) // P, count)
    add = need - count
    at = fc - 1 - ((torch.cumsum(add, 0) - add)[:, None] + col - count[:, None])
    fresh = (col >= count[:, None]) & (col < need[:, None])
    table = torch.where(fresh, free[torch.where(fresh, at, torch.zeros_like(at)).long()], table)
    fc = fc - add.sum()
    ends = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32)
    t = torch.arange(s["slots"].shape[0], device=DEV)
    b = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    pos = (kv[b] + t - starts[b]).clamp(min=0)
    slots = torch.where(t < ends[-1], table[b, (pos // P).clamp(max=cols - 1)] * P + pos % P, torch.full_like(t, -1)).to(torch.int32)
    # the pages past each request's length go back, the last taken first
    keep = torch.minimum((kv + P - 1) // P, need)
    drop = (col >= keep[:, None]) & (col < need[:, None])
    rank = torch.cumsum(drop.reshape(-1).long(), 0) - 1
    total = drop.sum()
    to = torch.where(drop.reshape(-1), fc + total - 1 - rank, torch.full_like(rank, free.shape[0]))
    free = torch.cat([free, free[:1]]).scatter(0, to, table.reshape(-1))[:-1]
    table = torch.where(drop, torch.full_like(table, -1), table)
    return {"slots": slots, "starts": starts, "table": table, "count": keep.to(torch.int32), "free": free,
            "free_count": (fc + total).to(torch.int32)}


def _plain_rope(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, n, Hq, dh = q.shape
    half = s["inv_freq"].shape[0]
    off = s["depth"] if s["depth"] is not None else torch.arange(n, device=DEV)[None]
    pos = (s["kv_len"][:, None] - 1 + off).double()
    angle = pos[:, :, None, None] * s["inv_freq"]
    c, d = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()

    def turned(x):
        y = x.float()
        r, rest = y[..., :2 * half], y[..., 2 * half:]
        a, b = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else (r[..., :half], r[..., half:])
        a, b = a * c - b * d, b * c + a * d
        r = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1).to(x.dtype)

    return {"q": turned(q), "k": turned(k).transpose(1, 2).contiguous(), "v": v.transpose(1, 2).contiguous()}


def _plain_rows(x, pool, scale, page, row, live):
    """Rows x [T, Hkv, dh] into row `row` of page `page` where `live`; a page whose first new row is not its row 0 keeps its
    earlier rows, at a scale that has room for both."""
    N, Hkv, P, dh = pool.shape
    x = x.float()
    at = torch.where(live, page, torch.full_like(page, N))
    amax = torch.zeros((N + 1, Hkv), device=DEV).index_reduce(0, at, x.abs().amax(2), "amax")[:N]
    first = torch.full((N + 1,), P, device=DEV, dtype=torch.long).scatter_reduce(0, at, row, "amin")[:N]
    e_old = torch.frexp(scale)[1] - 1
    e = _block_exponent(amax)
    e = torch.where((first > 0)[:, None], torch.maximum(e, e_old), e)
    e = torch.where((first < P)[:, None], e, e_old)
    before = torch.arange(P, device=DEV)[None, :] < first[:, None]          # all rows of a page that is not written to
    codes = (pool.float() * torch.where(before[:, None, :], torch.exp2((e_old - e).float())[:, :, None], torch.ones((), device=DEV))[..., None])
    y = (x / torch.exp2(e.float())[at.clamp(max=N - 1)][:, :, None]).to(torch.float8_e4m3fn)
    codes = codes.to(torch.float8_e4m3fn).view(torch.uint8).transpose(1, 2).reshape(N * P, Hkv, dh)
    codes = torch.cat([codes, codes[:1]]).index_copy(0, torch.where(live, page * P + row, torch.full_like(page, N * P)), y.view(torch.uint8))[:-1]
    pool.view(torch.uint8).copy_(codes.view(N, P, Hkv, dh).transpose(1, 2))
    scale.copy_(torch.exp2(e.float()))


def _plain_write(s):
    P = s["page"]
    if s["form"] == "append":
        slots = s["slots"].long()
        page, row, live = slots // P, slots % P, slots >= 0
        k, v = s["k"], s["v"]
    else:
        s["kv_len"].copy_(s["kv_len0"])
        B, Hkv, n, dh = s["k"].shape
        D = s["path"].shape[1] - 1
        step = torch.arange(1, D + 1, device=DEV)[None]
        live = step <= s["accept"][:, None]
        node = s["path"][:, 1:].clamp(min=0).long()
        pos = (s["kv_len"][:, None] + step - 1).long()
        page = s["table"].gather(1, pos // P).long().reshape(-1)
        row = (pos % P).reshape(-1)
        k, v = (x.gather(2, node[:, None, :, None].expand(B, Hkv, D, dh)).transpose(1, 2).reshape(B * D, Hkv, dh) for x in (s["k"], s["v"]))
        slots = torch.full((B, n + 1), -1, dtype=torch.int32, device=DEV)
        slots[:, 0] = s["kv_len"] - 1
        s["slots"].copy_(slots.scatter(1, torch.where(live, node, torch.full_like(node, n)), pos.int())[:, :n])
        s["kv_len"].add_(s["accept"])
        live = live.reshape(-1)
    _plain_rows(k, s["kp"], s["ks"], page, row, live)
    _plain_rows(v, s["vp"], s["vs"], page, row, live)


def _plain_attend(s):
    q, kp, P = s["q"], s["kp"], s["page"]
    B, n, Hq, dh = q.shape
    Hkv, L = kp.shape[1], s["L"]
    at = s["table"].clamp(min=0).long()
    keys, values = ((pool[at].float() * sc[at][..., None, None]).transpose(2, 1).reshape(B, Hkv, -1, dh)[:, :, :L]
                    for pool, sc in ((kp, s["ks"]), (s["vp"], s["vs"])))
    there = torch.arange(L, device=DEV)[None] < s["kv_len"][:, None]
    keys = torch.cat([keys, s["kt"].float()], 2)
    values = torch.cat([torch.where(there[:, None, :, None], values, torch.zeros((), device=DEV)), s["vt"].float()], 2)
    qg = q.float().view(B, n, Hkv, Hq // Hkv, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, dh)
    x = torch.matmul(qg, keys.transpose(2, 3)) * dh ** -0.5
    keep = torch.cat([there[:, None, :].expand(B, n, L), s["keep"]], 2)
    x = x.view(B, Hkv, Hq // Hkv, n, L + n).masked_fill(~keep[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(B, Hkv, -1, L + n), values).view(B, Hkv, Hq // Hkv, n, dh) / total
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, dh).to(q.dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, n, Hq)}


def _own(s):
    import tree_speculative_decoding_eagle_gb300 as eg
    if s["kind"] == "pages":
        eg.page_map(s["kv_len"], s["new_len"], s["table"], s["count"], s["free"], s["free_count"], s["page"],
                    slot_map=s["slots"], new_start=s["starts"], status=s["status"])
        eg.page_release(s["kv_len"], s["table"], s["count"], s["free"], s["free_count"], s["page"], status=s["status"])
        return {k: s[k] for k in ("slots", "starts", "table", "count", "free", "free_count")}
    if s["kind"] == "rope":
        q, k, v = eg.rope(s["q"], s["k"], s["v"], s["inv_freq"], pos_base=s["kv_len"], pos_off=s["depth"], shift=-1,
                          factor=s["factor"], interleaved=s["interleaved"], q_out=s["q_out"], k_tree=s["k_out"],
                          v_tree=s["v_out"])
        return {"q": q, "k": k, "v": v}
    if s["kind"] == "write":
        pools = (s["kp"], s["vp"], s["ks"], s["vs"])
        if s["form"] == "append":
            eg.kv8_append(s["k"], s["v"], s["slots"], *pools, status=s["status"])
        else:
            s["kv_len"].copy_(s["kv_len0"])        # the same step again: the commit adds to kv_len
            eg.kv8_commit(s["k"], s["v"], s["accept"], s["path"], *pools, s["kv_len"], s["table"],
                          slot_mapping=s["slots"], status=s["status"])
        return None
    if "ws" not in s["scratch"]:
        s["scratch"]["ws"] = eg.Workspace(DEV)
    out, lse = eg.tree_attn_kv8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["kv_len"], s["kt"], s["vt"],
                                s["mask"], out=s["out"], lse=s["lse"], workspace=s["scratch"]["ws"], status=s["status"])
    return {"out": out, "lse": lse}


_PLAIN = {"pages": _plain_pages, "rope": _plain_rope, "write": _plain_write, "attend": _plain_attend}


def run(state):
    got = _own(state) if own else _PLAIN[state["kind"]](state)
    if state["kind"] == "write":                   # a cache value is its e4m3 number times its block's scale
        got = {k: state[k] for k in ("kp", "ks", "vp", "vs")}
        if state["form"] == "commit":
            got |= {"slots": state["slots"], "kv_len": state["kv_len"]}
    return got


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    B, size = case["B"], 4 if case.get("dtype") == "f32" else 2
    if case["kind"] == "pages":
        taken = B + case["T"] // case["page"]      # about: pages that the new tokens begin
        return {"bytes": 4.0 * (5 * B + case["T"] + 4 * taken), "flops": 4.0 * (B + case["T"])}
    if case["kind"] == "rope":
        n, Hq, Hkv, dh = (case[k] for k in ("n", "Hq", "Hkv", "dh"))
        return {"bytes": 2.0 * B * n * (Hq + 2 * Hkv) * dh * size + 4.0 * B * n, "flops": 3.0 * B * n * (Hq + Hkv) * case["rot"]}
    if case["kind"] == "write":
        rows = case["T"] if case["form"] == "append" else B * case["D"] / 2
        touched = rows / case["page"] + B
        return {"bytes": 2.0 * rows * case["Hkv"] * case["dh"] * (size + 1) + 2 * 4.0 * touched * case["Hkv"] + 4.0 * rows,
                "flops": 4.0 * rows * case["Hkv"] * case["dh"]}
    n, Hq, Hkv, dh = (case[k] for k in ("n", "Hq", "Hkv", "dh"))
    L = (case["L"] + case["L_min"]) / 2
    return {"bytes": B * (2.0 * L * Hkv * (dh + 4.0 / case["page"]) + 4.0 * n * Hkv * dh + 4.0 * n * Hq * dh + 4.0 * n * Hq),
            "flops": 4.0 * B * n * Hq * dh * (L + min(n, 6))}


# ---- the definitions in 64 bits ---------------------------------------------------

def _e4m3(y):
    """Nearest e4m3 number, ties to even, in 64 bits (|y| <= 448)."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > y.abs().clamp(min=2.0 ** -6), e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= y.abs(), e + 1, e)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _exact_rope(case, s):
    half, p = case["rot"] // 2, s["kv_len"].double()[:, None] - 1
    p = p + (s["depth"].double() if s["depth"] is not None else torch.arange(case["n"], device=DEV, dtype=torch.float64)[None])
    j = torch.arange(half, device=DEV)
    first, second = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
    turn = torch.polar(torch.full((), s["factor"], device=DEV, dtype=torch.float64), p[..., None] * s["inv_freq"].double())

    def one(x):
        x = x.double().clone()
        z = torch.complex(x[..., first], x[..., second]) * turn[:, :, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    return {"q": one(s["q"]), "k": one(s["k"]).movedim(2, 1).contiguous(), "v": s["v"].double().movedim(2, 1).contiguous()}


def _exact_write(case, s):
    P = case["page"]
    if case["form"] == "append":
        slots = s["slots"].tolist()
        where = [(t, sl // P, sl % P) for t, sl in enumerate(slots) if sl >= 0]
        rows = {"k": s["k"].double(), "v": s["v"].double()}
    else:
        where, pick = [], []
        for b in range(case["B"]):
            for a in range(int(s["accept"][b])):
                at = int(s["kv_len0"][b]) + a
                where.append((len(pick), int(s["table"][b, at // P]), at % P))
                pick.append((b, int(s["path"][b, a + 1])))
        bs, ns = ([x[i] for x in pick] for i in (0, 1))
        rows = {"k": s["k"][bs, :, ns].double(), "v": s["v"][bs, :, ns].double()}
    runs = {}
    for t, page, row in where:
        runs.setdefault(page, []).append((t, row))
    out = {}
    order = sorted(runs)
    fresh = torch.tensor([min(r for _, r in runs[p]) == 0 for p in order], device=DEV)
    first = torch.tensor([min(r for _, r in runs[p]) for p in order], device=DEV)
    idx = torch.tensor(order, device=DEV)
    which = {p: i for i, p in enumerate(order)}
    ts, ps, rs = (torch.tensor([x[i] for x in where], device=DEV, dtype=torch.long) for i in (0, 1, 2))
    group = torch.tensor([which[int(p)] for p in ps.tolist()], device=DEV, dtype=torch.long)
    for name, pool, scale in (("k", "kp", "ks"), ("v", "vp", "vs")):
        codes, sc = s[pool].double(), s[scale].double()
        if order:
            x = rows[name][ts]
            top = torch.zeros((len(order), x.shape[1]), dtype=torch.float64, device=DEV).index_reduce(0, group, x.abs().amax(2), "amax")
            least = torch.exp2(torch.ceil(torch.log2((top / E4M3_MAX).clamp(min=2.0 ** E_MIN))).clamp(E_MIN, E_MAX))
            least = torch.where(least * E4M3_MAX < top, least * 2, least)
            grown = torch.where(fresh[:, None], least, torch.maximum(least, sc[idx]))
            old = _e4m3(codes[idx] * (sc[idx] / grown)[:, :, None, None])
            codes[idx] = torch.where((torch.arange(P, device=DEV)[None] < first[:, None])[:, None, :, None], old, codes[idx])
            codes[ps, :, rs] = _e4m3(x / grown[group][:, :, None])
            sc[idx] = grown
        out[pool], out[scale] = codes, sc
    return out


def _exact_attend(case, s):
    n, Hq, Hkv, dh, P = (case[k] for k in ("n", "Hq", "Hkv", "dh", "page"))
    if case["B"] * (case["L"] + n) * n * Hq * dh > 3e11:
        return None                                # too long in 64 bits
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        L = int(s["kv_len"][b])
        pages = s["table"][b, :(L + P - 1) // P].long()
        for g in range(Hkv):
            K, V = (torch.cat([(pool[pages, g].double() * sc[pages, g].double()[:, None, None]).reshape(-1, dh)[:L], tree[b, g].double()])
                    for pool, sc, tree in ((s["kp"], s["ks"], s["kt"]), (s["vp"], s["vs"], s["vt"])))
            heads = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            x = torch.einsum("ihd,ld->ihl", s["q"][b, :, heads].double(), K) / math.sqrt(dh)
            x[:, :, L:].masked_fill_(~s["keep"][b][:, None], -math.inf)
            lse[b, :, heads] = torch.logsumexp(x, -1)
            out[b, :, heads] = torch.einsum("ihl,ld->ihd", torch.softmax(x, -1), V)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["kind"] == "pages":
        return None                                # whole numbers
    return {"rope": _exact_rope, "write": _exact_write, "attend": _exact_attend}[case["kind"]](case, prepare(case, seed))
