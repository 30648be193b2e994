"""Long contexts over the paged 8-bit cache: its operators' cases, their plain forms and what they cost.

    norm    each head's root mean square taken out of q and k, a learned weight, and the rotary position, into the layouts
            that the attention reads
    bounds  the least and the greatest number of each column over the keys of a page, for the pages that new tokens touched
    select  for each query and KV head the pages whose bounds allow the greatest product with the query
    attend  attention of draft nodes (or of single tokens) over the selected pages and the tree

One decoding step is norm, attend with what select chose, and bounds once the accepted tokens are in the cache.  With `own` the
calls are the framework's, without it elementary torch operations in 32 bits (angles in 64).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ---- cases --------------------------------------------------------------------

def listed():
    return [
        # the tree of llama2-7b-b1: 61 nodes, every head with its own keys; launch latency counts
        {"name": "norm llama2-7b-b1", "kind": "norm", "B": 1, "n": 61, "Hq": 32, "Hkv": 32, "dh": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "dtype": "bf16", "kv_max": 2048},
        # the trees of gpt-oss-20b-b64: grouped heads, frequencies stretched for long contexts, far positions
        {"name": "norm gpt-oss-20b-b64", "kind": "norm", "B": 64, "n": 61, "Hq": 64, "Hkv": 8, "dh": 64, "rot": 64,
         "interleaved": False, "scaling": "yarn", "dtype": "bf16", "kv_max": 131072},
        # a prompt of odd length, interleaved pairs, a quarter of the head rotated, in 32 bits
        {"name": "norm prompt f32", "kind": "norm", "B": 1, "n": 8191, "Hq": 40, "Hkv": 40, "dh": 128, "rot": 32,
         "interleaved": True, "scaling": "linear", "dtype": "f32", "kv_max": 0},
        # one more token of each of 64 requests: the page that it ends up in
        {"name": "bounds tokens 64", "kind": "bounds", "B": 64, "Hkv": 8, "dh": 64, "page": 64, "kv_max": 8192, "new": 1},
        # the prompts of llama2-70b-b16, whole
        {"name": "bounds prompts 70b-b16", "kind": "bounds", "B": 16, "Hkv": 8, "dh": 128, "page": 64, "kv_max": 0, "new": 4096},
        # one request far into its context, one token: small pages, every head with its own keys
        {"name": "select one request", "kind": "select", "B": 1, "n": 1, "Hq": 32, "Hkv": 32, "dh": 128, "page": 16,
         "L": 32768, "L_min": 32768, "top": 64, "first": 1, "last": 2},
        # single tokens of 64 requests with ragged long contexts: the bounds' bytes are all that counts
        {"name": "select tokens 64", "kind": "select", "B": 64, "n": 1, "Hq": 64, "Hkv": 8, "dh": 128, "page": 64,
         "L": 131072, "L_min": 32768, "top": 32, "first": 1, "last": 1},
        # the trees of llama2-70b-b16 after a longer context: products count
        {"name": "select 70b-b16 trees", "kind": "select", "B": 16, "n": 49, "Hq": 64, "Hkv": 8, "dh": 128, "page": 64,
         "L": 32768, "L_min": 32768, "top": 16, "first": 1, "last": 1},
        # one token of one request
        {"name": "attend one request", "kind": "attend", "B": 1, "n": 1, "Hq": 32, "Hkv": 32, "dh": 128, "page": 16,
         "L": 32768, "L_min": 32768, "top": 64},
        # single tokens of 64 requests with ragged contexts: the selected pages' bytes
        {"name": "attend tokens 64", "kind": "attend", "B": 64, "n": 1, "Hq": 64, "Hkv": 8, "dh": 128, "page": 64,
         "L": 16384, "L_min": 1024, "top": 32},
        # the trees of llama2-70b-b16
        {"name": "attend 70b-b16 trees", "kind": "attend", "B": 16, "n": 49, "Hq": 64, "Hkv": 8, "dh": 128, "page": 64,
         "L": 8192, "L_min": 4096, "top": 16},
        # the largest: the trees of gpt-oss-20b-b64
        {"name": "attend gpt-oss-20b-b64 trees", "kind": "attend", "B": 64, "n": 61, "Hq": 64, "Hkv": 8, "dh": 64, "page": 128,
         "L": 8192, "L_min": 8192, "top": 8},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm", "bounds", "select", "select", "attend", "attend"])
    dh = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "norm":
        B = _log(rng, 1, 64)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        Hkv, G = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 2, 4, 5, 8])
        Hq = min(64, Hkv * G) // Hkv * Hkv
        most = 80e6 / (B * (Hq + 2 * Hkv) * dh * (4 if dtype == "f32" else 2))
        return {"kind": kind, "B": B, "n": _log(rng, 1, max(1, min(8191, int(most)))), "Hq": Hq, "Hkv": Hkv, "dh": dh,
                "rot": rng.choice([dh, dh, dh // 2, dh // 4, 20]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice(["none", "linear", "yarn"]), "dtype": dtype, "kv_max": _log(rng, 1, 131072)}
    if kind == "bounds":
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 4, 8, 40])
        most = 6e7 / (B * Hkv * dh)
        new = _log(rng, 1, max(1, min(8192, int(most))))
        return {"kind": kind, "B": B, "Hkv": Hkv, "dh": dh, "page": page, "new": new,
                "kv_max": _log(rng, 1, max(1, min(8192, int(2.5 * most))))}
    Hkv, G = rng.choice([1, 2, 4, 8, 32]), rng.choice([1, 1, 2, 4, 5, 8])
    Hq = min(64, Hkv * G) // Hkv * Hkv
    n = rng.choice([1, 1, _log(rng, 2, 16), rng.randint(17, 64)])
    B, L = _log(rng, 1, 64), _log(rng, 1, 131072 if kind == "select" else 16384)
    top = rng.randint(2, 64)
    c = {"kind": kind, "B": B, "n": n, "Hq": Hq, "Hkv": Hkv, "dh": dh, "page": page, "top": top}
    if kind == "select":
        pages = lambda: (L + page - 1) // page
        while B * pages() * Hkv * dh > 64 * 2048 * 8 * 128 * 0.7 or B * n * Hq * pages() * dh > 16 * 49 * 64 * 512 * 128 * 0.7:
            L, B = max(1, L // 2), max(1, B - B // 4)
        return c | {"B": B, "L": L, "L_min": rng.choice([0, L, (L + 1) // 2]), "first": rng.randint(0, 1), "last": rng.randint(0, 1)}
    while B * n * Hkv * top * page * dh > 64 * 61 * 8 * 1024 * 64 * 0.7 or B * L * Hkv * dh > 64 * 16384 * 8 * 128:
        top, L, B = max(1, top // 2), max(1, L * 3 // 4), max(1, B - B // 4)
    return c | {"B": B, "L": L, "L_min": rng.choice([0, L, (L + 1) // 2]), "top": top}


# ---- what a program has in hand -------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(g, lo, hi, size):
    """Whole numbers of lo..hi."""
    return torch.randint(lo, hi + 1, size, generator=g, device=DEV, dtype=torch.int32)


def _randn(g, *size):
    return torch.randn(size, generator=g, device=DEV)


def _random_pool(g, num_pages, Hkv, page, dh):
    """Pages of N(0, 1) rows times a magnitude of the page and head, in e4m3 with the least power of two that fits."""
    x = _randn(g, num_pages, Hkv, page, dh)
    x *= torch.exp2(_randn(g, num_pages, Hkv, 1, 1) * 0.5)
    scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / E4M3_MAX)))
    scale = torch.where(scale * E4M3_MAX < x.abs().amax((2, 3)), scale * 2, scale)
    x /= scale[:, :, None, None]
    return x.to(torch.float8_e4m3fn), scale


def _tables(g, kv_len, page, max_pages, num_pages):
    B = kv_len.shape[0]
    perm = torch.randperm(num_pages, generator=g, device=DEV)[:B * max_pages].to(torch.int32).view(B, max_pages)
    used = (kv_len[:, None] + page - 1) // page > torch.arange(max_pages, device=DEV)[None]
    return torch.where(used, perm, torch.full_like(perm, -1)).contiguous()


def _frequencies(case):
    """inv_freq [rot/2] in 64 bits and the factor on cos and sin."""
    rot, theta = case["rot"], 10000.0
    f = theta ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "yarn":                  # the ramp is linear in the pair's index
        at = lambda r: rot * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f / 32.0 * ramp + f * (1 - ramp), 0.1 * math.log(32.0) + 1.0
    return f, 1.0


def _prepare_norm(case, g):
    B, n, Hq, Hkv, dh = (case[k] for k in ("B", "n", "Hq", "Hkv", "dh"))
    t = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    # one fused projection, of heads of unlike magnitudes
    qkv = (_randn(g, B, n, Hq + 2 * Hkv, dh) * torch.exp2(_randn(g, Hq + 2 * Hkv, 1))).to(t).view(B, n, -1)
    f, factor = _frequencies(case)
    kv = _ints(g, 1, max(1, case["kv_max"]), (B,))
    depth = None
    if case["kv_max"]:                             # a tree: positions from the nodes' depths; a prompt: 0, 1, 2 ...
        depth = torch.sort(_ints(g, 0, 6, (B, n)), dim=1).values.to(torch.int32)
        depth[:, 0] = 0
    else:
        kv = torch.zeros_like(kv)
    q, k, v = qkv.split([Hq * dh, Hkv * dh, Hkv * dh], dim=2)
    return {"q": q.unflatten(2, (Hq, dh)), "k": k.unflatten(2, (Hkv, dh)), "v": v.unflatten(2, (Hkv, dh)), "kv_len": kv,
            "depth": depth, "inv_freq": torch.from_numpy(f).to(DEV), "factor": factor, "interleaved": case["interleaved"],
            "eps": 1e-6, "qw": (1 + 0.2 * _randn(g, dh)).to(t), "kw": (1 + 0.2 * _randn(g, dh)).to(t),
            "q_out": torch.empty((B, n, Hq, dh), dtype=t, device=DEV),
            "k_out": torch.empty((B, Hkv, n, dh), dtype=t, device=DEV),
            "v_out": torch.empty((B, Hkv, n, dh), dtype=t, device=DEV)}


def _prepare_bounds(case, g):
    B, Hkv, dh, page, new = (case[k] for k in ("B", "Hkv", "dh", "page", "new"))
    before = _ints(g, 0, case["kv_max"], (B,))
    # prompts come whole and alike, pieces of them ragged
    add = torch.full((B,), new, dtype=torch.int32, device=DEV) if new == 1 or not case["kv_max"] else _ints(g, 0, new, (B,))
    max_pages = (case["kv_max"] + new + page - 1) // page
    num_pages = B * max_pages + 4
    kv = before + add
    kp, ks = _random_pool(g, num_pages, Hkv, page, dh)
    return {"kp": kp, "from": before, "kv_len": kv, "table": _tables(g, kv, page, max_pages, num_pages), "window": new // page + 2,
            "bounds": torch.zeros((num_pages, Hkv, 2, dh), device=DEV).to(torch.float8_e4m3fn),
            "status": torch.zeros(1, dtype=torch.int32, device=DEV)}


def _prepare_select(case, g):
    B, n, Hq, Hkv, dh, page = (case[k] for k in ("B", "n", "Hq", "Hkv", "dh", "page"))
    kv = _ints(g, case["L_min"], case["L"], (B,))
    max_pages = (case["L"] + page - 1) // page
    num_pages = B * max_pages + 4
    # a page's columns: a middle and a width about it, in units where its largest number is below 448
    middle, width = _randn(g, num_pages, Hkv, 1, dh) * 48, 60 + 60 * torch.rand((num_pages, Hkv, 1, dh), generator=g, device=DEV)
    x = torch.cat([middle - width, middle + width], 2).clamp(-E4M3_MAX, E4M3_MAX)
    return {"q": (_randn(g, B, n, Hq, dh) * 1.5).to(torch.bfloat16), "kv_len": kv,
            "bounds": (torch.round(2 * x) / 2).to(torch.float8_e4m3fn),
            "ks": torch.exp2(_ints(g, -8, -6, (num_pages, Hkv)).float()),
            "table": _tables(g, kv, page, max_pages, num_pages), "top": case["top"], "first": case["first"], "last": case["last"],
            "sel": torch.empty((B, n, Hkv, case["top"]), dtype=torch.int32, device=DEV),
            "score": torch.empty((B, n, Hkv, case["top"]), dtype=torch.float32, device=DEV),
            "status": torch.zeros(1, dtype=torch.int32, device=DEV), "scratch": {}}


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


def _prepare_attend(case, g):
    B, n, Hq, Hkv, dh, page, top = (case[k] for k in ("B", "n", "Hq", "Hkv", "dh", "page", "top"))
    kv = _ints(g, case["L_min"], case["L"], (B,))
    max_pages = (case["L"] + page - 1) // page
    num_pages = B * max_pages + 4
    s = {"kv_len": kv, "table": _tables(g, kv, page, max_pages, num_pages)}
    s["kp"], s["ks"] = _random_pool(g, num_pages, Hkv, page, dh)
    s["vp"], s["vs"] = _random_pool(g, num_pages, Hkv, page, dh)
    # queries strong enough for a peaked softmax, as a trained model's are
    s["q"] = (_randn(g, B, n, Hq, dh) * 1.5).to(torch.bfloat16)
    s["kt"], s["vt"] = (_randn(g, B, Hkv, n, dh).to(torch.bfloat16) for _ in range(2))
    s["mask"], s["keep"] = _tree_mask(g, B, n)
    # the pages of a node: those of its tree for the most part, the first and the last among them
    live = (kv + page - 1) // page
    col = torch.arange(max_pages, device=DEV)
    want = _randn(g, B, 1, Hkv, max_pages) + 0.5 * _randn(g, B, n, Hkv, max_pages)
    want = torch.where((col == 0) | (col == live[:, None, None, None] - 1), torch.full_like(want, 100.0), want)
    want = torch.where(col < live[:, None, None, None], want, torch.full_like(want, -100.0))
    best = torch.sort(want, dim=-1, descending=True, stable=True)
    sel = torch.where(best.values > -100.0, best.indices, torch.full_like(best.indices, max_pages))[..., :top]
    sel = torch.sort(sel, dim=-1).values
    sel = torch.where(sel < max_pages, sel, torch.full_like(sel, -1)).to(torch.int32)
    s["sel"] = torch.full((B, n, Hkv, top), -1, dtype=torch.int32, device=DEV)
    s["sel"][..., :sel.shape[-1]] = sel            # fewer pages than `top`: -1 behind them
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((B, n, Hq), dtype=torch.float32, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    s["scratch"] = {}                              # where a program keeps the operator's workspace
    return s


_PREPARE = {"norm": _prepare_norm, "bounds": _prepare_bounds, "select": _prepare_select, "attend": _prepare_attend}


def prepare(case, seed):
    s = _PREPARE[case["kind"]](case, _gen(seed))
    s["kind"], s["page"] = case["kind"], case.get("page")
    return s


# ---- one pass -------------------------------------------------------------------

def _plain_norm(s):
    n, half = s["q"].shape[1], s["inv_freq"].shape[0]
    off = s["depth"] if s["depth"] is not None else torch.arange(n, device=DEV)[None]
    angle = (s["kv_len"][:, None] + off).double()[:, :, None, None] * s["inv_freq"]
    c, d = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()

    def turned(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        r, rest = y[..., :2 * half], y[..., 2 * half:]
        a, b = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else (r[..., :half], r[..., half:])
        a, b = a * c - b * d, b * c + a * d
        r = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([r, rest], -1).to(x.dtype)

    return {"q": turned(s["q"], s["qw"]), "k": turned(s["k"], s["kw"]).transpose(1, 2).contiguous(),
            "v": s["v"].transpose(1, 2).contiguous()}


def _plain_bounds(s):
    P, kp, table = s["page"], s["kp"], s["table"]
    N = kp.shape[0]
    # the pages from the first new token's to the last one's, at most `window` of them
    col = (s["from"] // P)[:, None] + torch.arange(s["window"], device=DEV)[None]
    live = (col * P < s["kv_len"][:, None]) & (s["kv_len"] > s["from"])[:, None]
    page = table.gather(1, col.clamp(max=table.shape[1] - 1).long()).long().clamp(min=0)
    there = (col * P)[..., None] + torch.arange(P, device=DEV) < s["kv_len"][:, None, None]
    x = kp[page].float()
    there = there[:, :, None, :, None]
    hi = torch.ceil(2 * x.masked_fill(~there, -math.inf).amax(3)) / 2
    lo = torch.floor(2 * x.masked_fill(~there, math.inf).amin(3)) / 2
    got = torch.stack([lo, hi], 3).flatten(0, 1).to(torch.float8_e4m3fn).view(torch.uint8)
    all_pages = torch.cat([s["bounds"].view(torch.uint8), got[:1]])
    s["bounds"].view(torch.uint8).copy_(all_pages.index_copy(0, torch.where(live, page, torch.full_like(page, N)).flatten(), got)[:-1])
    return {"bounds": s["bounds"]}


def _plain_select(s):
    q, P, top = s["q"].float(), s["page"], s["top"]
    B, n, Hq, dh = q.shape
    N, Hkv = s["bounds"].shape[:2]
    Np, G = s["table"].shape[1], Hq // Hkv
    amax = q.abs().amax(-1, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 7, torch.zeros_like(amax, dtype=torch.int32)).clamp(-32, 32)
    whole = torch.round(q * torch.exp2(-e.float())).clamp(-128, 128)
    rows = lambda x: x.view(B, n, Hkv, G, -1).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, -1)
    at = s["table"].clamp(min=0).long()
    b = s["bounds"].float()[at].permute(0, 2, 3, 4, 1)                    # [B, Hkv, 2, dh, Np]
    w = rows(whole)
    u = torch.matmul(w.clamp(max=0), b[:, :, 0]) + torch.matmul(w.clamp(min=0), b[:, :, 1])
    score = u * torch.exp2(rows(e.float())) * s["ks"][at].transpose(1, 2)[:, :, None]
    score = score.view(B, Hkv, n, G, Np).amax(3).transpose(1, 2)          # [B, n, Hkv, Np]
    live = ((s["kv_len"] + P - 1) // P)[:, None, None, None]
    col = torch.arange(Np, device=DEV)
    want = score.masked_fill((col < s["first"]) | (col >= live - s["last"]), math.inf).masked_fill(col >= live, -math.inf)
    best = torch.sort(want, dim=-1, descending=True, stable=True).indices[..., :top]
    best = torch.sort(torch.where(best < live, best, torch.full_like(best, Np)), dim=-1).values
    s["sel"].fill_(-1)
    s["sel"][..., :best.shape[-1]] = torch.where(best < Np, best, torch.full_like(best, -1)).to(torch.int32)
    s["score"].fill_(-math.inf)
    s["score"][..., :best.shape[-1]] = score.gather(-1, best.clamp(max=Np - 1)).masked_fill(best >= Np, -math.inf)
    return {"sel": s["sel"], "score": s["score"]}


def _plain_attend(s):
    q, P, sel = s["q"].float(), s["page"], s["sel"].long()
    B, n, Hq, dh = q.shape
    Hkv, top = s["kp"].shape[1], sel.shape[-1]
    col = sel.clamp(min=0)
    page = s["table"].clamp(min=0).long()[torch.arange(B, device=DEV)[:, None, None, None], col]
    block = page * Hkv + torch.arange(Hkv, device=DEV)[:, None]           # [B, n, Hkv, top]
    keys, values = ((pool.view(torch.uint8).flatten(0, 1)[block].view(torch.float8_e4m3fn).float() * sc.flatten()[block][..., None, None]).flatten(3, 4)
                    for pool, sc in ((s["kp"], s["ks"]), (s["vp"], s["vs"])))
    there = ((col * P)[..., None] + torch.arange(P, device=DEV) < s["kv_len"][:, None, None, None, None]) & (sel >= 0)[..., None]
    there = there.flatten(3, 4)
    qg = q.view(B, n, Hkv, Hq // Hkv, dh)
    x = torch.matmul(qg, keys.transpose(3, 4)).masked_fill(~there[:, :, :, None], -math.inf)
    y = torch.matmul(qg.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, dh), s["kt"].float().transpose(2, 3))
    y = y.view(B, Hkv, n, -1, n).masked_fill(~s["keep"][:, None, :, None], -math.inf).transpose(1, 2)
    x = torch.cat([x, y], -1) * dh ** -0.5
    most = x.amax(-1, keepdim=True)
    x = torch.exp(x - most)
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x[..., :top * P], values)
    y = x[..., top * P:].transpose(1, 2).reshape(B, Hkv, -1, n)
    out = (out + torch.matmul(y, s["vt"].float()).view(B, Hkv, n, -1, dh).transpose(1, 2)) / total
    return {"out": out.reshape(B, n, Hq, dh).to(s["q"].dtype), "lse": (most + torch.log(total)).reshape(B, n, Hq)}


def _own(s):
    import tree_speculative_decoding_eagle_gb300 as eg
    if s["kind"] == "norm":
        q, k, v = eg.qk_norm_rope(s["q"], s["k"], s["v"], s["inv_freq"], s["qw"], s["kw"], eps=s["eps"], pos_base=s["kv_len"],
                                  pos_off=s["depth"], factor=s["factor"], interleaved=s["interleaved"], q_out=s["q_out"],
                                  k_tree=s["k_out"], v_tree=s["v_out"])
        return {"q": q, "k": k, "v": v}
    if s["kind"] == "bounds":
        eg.kv8_bounds(s["kp"], s["table"], s["from"], s["kv_len"], s["bounds"], status=s["status"])
        return {"bounds": s["bounds"]}
    if "ws" not in s["scratch"]:
        s["scratch"]["ws"] = eg.Workspace(DEV)
    if s["kind"] == "select":
        sel = eg.kv8_select(s["q"], s["bounds"], s["ks"], s["table"], s["kv_len"], s["page"], s["top"], first=s["first"],
                            last=s["last"], out=s["sel"], score=s["score"], workspace=s["scratch"]["ws"], status=s["status"])
        return {"sel": sel, "score": s["score"]}
    out, lse = eg.tree_attn_kv8_pages(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["kv_len"], s["kt"], s["vt"],
                                      s["mask"], s["sel"], out=s["out"], lse=s["lse"], workspace=s["scratch"]["ws"],
                                      status=s["status"])
    return {"out": out, "lse": lse}


_PLAIN = {"norm": _plain_norm, "bounds": _plain_bounds, "select": _plain_select, "attend": _plain_attend}


def run(state):
    return _own(state) if own else _PLAIN[state["kind"]](state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    B = case["B"]
    if case["kind"] == "norm":
        n, Hq, Hkv, dh = (case[k] for k in ("n", "Hq", "Hkv", "dh"))
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2.0 * B * n * (Hq + 2 * Hkv) * dh * size + 4.0 * B * n,
                "flops": B * n * (Hq + Hkv) * (4.0 * dh + 3.0 * case["rot"])}
    if case["kind"] == "bounds":
        rows = case["new"] if case["new"] == 1 or not case["kv_max"] else case["new"] / 2
        # the page of the first new token is looked at from its start
        rows, pages = rows + (case["page"] / 2 if case["kv_max"] else 0), rows / case["page"] + 1
        return {"bytes": B * case["Hkv"] * case["dh"] * (rows + 2.0 * pages) + 4.0 * B * pages,
                "flops": 2.0 * B * case["Hkv"] * case["dh"] * rows}
    n, Hq, Hkv, dh, P, top = (case[k] for k in ("n", "Hq", "Hkv", "dh", "page", "top"))
    L = (case["L"] + case["L_min"]) / 2
    if case["kind"] == "select":
        pages = max(1.0, L / P)
        return {"bytes": B * (pages * Hkv * (2.0 * dh + 4) + 4.0 * pages + 2.0 * n * Hq * dh + 8.0 * n * Hkv * top),
                "flops": 2.0 * B * n * Hq * pages * dh}
    keys = min(L, top * P)                         # of a node; its tree reads at least these
    return {"bytes": B * (2.0 * keys * Hkv * (dh + 4.0 / P) + 4.0 * n * Hkv * dh + 4.0 * n * Hq * dh + 4.0 * n * Hq + 4.0 * n * Hkv * top),
            "flops": 4.0 * B * n * Hq * dh * (keys + min(n, 6))}


# ---- the definitions in 64 bits ---------------------------------------------------

def _exact_norm(case, s):
    half, p = case["rot"] // 2, s["kv_len"].double()[:, None]
    p = p + (s["depth"].double() if s["depth"] is not None else torch.arange(case["n"], device=DEV, dtype=torch.float64)[None])
    j = torch.arange(half, device=DEV)
    first, second = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
    turn = torch.polar(torch.full((), s["factor"], device=DEV, dtype=torch.float64), p[..., None] * s["inv_freq"].double())

    def one(x, w):
        x = x.double()
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["dh"] + s["eps"]) * w.double()
        z = torch.complex(x[..., first], x[..., second]) * turn[:, :, None]
        x[..., first], x[..., second] = z.real, z.imag
        return x

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"]).movedim(2, 1).contiguous(), "v": s["v"].double().movedim(2, 1).contiguous()}


def _exact_bounds(case, s):
    P, got = case["page"], s["bounds"].double()
    for b in range(case["B"]):
        lo, hi = int(s["from"][b]), int(s["kv_len"][b])
        if hi <= lo:
            continue
        full = torch.arange(lo // P, hi // P, device=DEV)
        rest = [(full, P)] if len(full) else []
        if hi % P:
            rest.append((torch.tensor([hi // P], device=DEV), hi % P))
        for cols, rows in rest:
            pages = s["table"][b, cols].long()
            x = s["kp"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()[:, :, :rows]
            got[pages] = torch.stack([torch.floor(x.amin(2) * 2) / 2, torch.ceil(x.amax(2) * 2) / 2], 2)
    return {"bounds": got}


def _exact_select(case, s):
    B, n, Hq, Hkv, P, top = (case[k] for k in ("B", "n", "Hq", "Hkv", "page", "top"))
    score = torch.full((B, n, Hkv, top), -math.inf, dtype=torch.float64, device=DEV)
    q = s["q"].double()
    size = q.abs().amax(-1)
    size = size.clamp(min=2.0 ** -26)
    step = torch.exp2(torch.floor(torch.log2(size)) - 6)
    step = torch.where(step * 128 <= size, step * 2, step)                # the logarithm of a power of two may end below it
    q = torch.round(q / step[..., None]) * step[..., None]
    codes = s["bounds"].view(torch.uint8)
    for b in range(B):
        Np = (int(s["kv_len"][b]) + P - 1) // P
        if Np == 0:
            continue
        pages = s["table"][b, :Np].long()
        b_of = codes[pages].view(torch.float8_e4m3fn).double() * s["ks"][pages].double()[..., None, None]
        for g in range(Hkv):
            x = q[b, :, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)]
            up = torch.einsum("ihd,pd->ihp", x * (x > 0), b_of[:, g, 1]) + torch.einsum("ihd,pd->ihp", x * (x < 0), b_of[:, g, 0])
            up = up.max(1).values
            order = up.clone()
            order[:, :case["first"]] = math.inf
            if case["last"]:
                order[:, max(0, Np - case["last"]):] = math.inf
            keep = min(top, Np)
            took = torch.argsort(order, dim=-1, descending=True, stable=True)[:, :keep].sort(-1).values
            score[b, :, g, :keep] = up.gather(1, took)
    return {"sel": None, "score": score}


def _exact_attend(case, s):
    n, Hq, Hkv, dh, P = (case[k] for k in ("n", "Hq", "Hkv", "dh", "page"))
    if case["B"] * Hkv > 2600 or case["B"] * n * Hkv * case["top"] * P * dh > 3e9:
        return None                                # too long in 64 bits
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    G = Hq // Hkv
    kp, vp = s["kp"].view(torch.uint8), s["vp"].view(torch.uint8)
    for b in range(case["B"]):
        L = int(s["kv_len"][b])
        for g in range(Hkv):
            cols = s["sel"][b, :, g].long()
            pages = s["table"][b].long()[cols.clamp(min=0)].clamp(min=0)
            K, V = ((pool[pages, g].view(torch.float8_e4m3fn).double() * sc[pages, g].double()[..., None, None]).reshape(n, -1, dh)
                    for pool, sc in ((kp, s["ks"]), (vp, s["vs"])))
            where = (cols * P)[..., None] + torch.arange(P, device=DEV)
            gone = ((where >= L) | (cols < 0)[..., None]).reshape(n, 1, -1)
            heads = slice(g * G, (g + 1) * G)
            Q = s["q"][b, :, heads].double()
            x = torch.cat([torch.einsum("ihd,ild->ihl", Q, K).masked_fill(gone, -math.inf),
                           torch.einsum("ihd,jd->ihj", Q, s["kt"][b, g].double()).masked_fill(~s["keep"][b][:, None], -math.inf)], -1)
            x = x / math.sqrt(dh)
            lse[b, :, heads] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            out[b, :, heads] = torch.einsum("ihl,ild->ihd", p[..., :-n], V) + torch.einsum("ihj,jd->ihd", p[..., -n:], s["vt"][b, g].double())
    return {"out": out, "lse": lse}


def exact(case, seed):
    return {"norm": _exact_norm, "bounds": _exact_bounds, "select": _exact_select, "attend": _exact_attend}[case["kind"]](case, prepare(case, seed))
