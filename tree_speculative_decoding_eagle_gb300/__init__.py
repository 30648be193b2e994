"""Python binding of libeagle.so, the sm_103a implementation of one EAGLE-2
tree-speculative decoding step.

Each function below marshals torch CUDA tensors into the C ABI declared in
include/eagle.h and calls it on the current CUDA stream; every step of the
computation runs in the library's kernels.  There is no fallback: if the
library is missing or a call reports an error, an exception is raised.

    draft_topk  -> eagle_draft_topk   (softmax statistics + top-k per draft row)
    tree_build  -> eagle_tree_build   (global scores, expansion, rerank, mask;
                   eagle_tree_build_variant for the ablation flags)
    static_tree -> eagle_static_tree  (EAGLE-1 static tree from a template)
    tree_mask   -> eagle_tree_mask    (ancestor-only attention mask)
    tree_attn   -> eagle_tree_attn    (tree-masked attention over the KV prefix)
    tree_attn_paged -> eagle_tree_attn_paged (the same over a paged prefix)
    kv_commit   -> eagle_kv_commit    (accepted path's K/V into the cache)
    verify      -> eagle_verify       (greedy / speculative-sampling walk)
    verify_noalloc -> eagle_verify_noalloc (the same without a caller workspace)
    verify_draft -> eagle_verify_draft (sampling walk against draft distributions q)
    selftest_wait -> eagle_selftest_wait (a bounded device wait that must give up)
    page_map / page_release -> eagle_page_map, eagle_page_reserve,
                   eagle_page_release (pages of a free list to requests and
                   back; slots of new tokens)
    rope        -> eagle_rope         (rotary positions, into the attention's layouts;
                   rope_freqs -> eagle_rope_freqs)
    qk_norm_rope -> eagle_qk_norm_rope (norms of the heads of q and k before them)
    kv8_append / kv8_commit -> eagle_kv8_append, eagle_kv8_commit,
                   eagle_kv8_commit_root (keys and values into the paged cache
                   of e4m3 numbers)
    tree_attn_kv8 -> eagle_tree_attn_kv8 (tree attention over that cache)
    kv8_bounds / kv8_select / tree_attn_kv8_pages -> eagle_kv8_bounds,
                   eagle_kv8_select, eagle_tree_attn_kv8_pages (the same over
                   the pages that each query's score selects)
    run_step / StepGraph -> eagle_step, eagle_step_graph_* (the four stages
                   in one call, or recorded once as a graph and replayed)
"""
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libeagle.so")

F32, BF16 = 0, 1
GREEDY, SAMPLE = 0, 1
TREE_CONFIDENCE_ONLY, TREE_NO_RERANK = 1, 2
ROPE_KINDS = {"plain": 0, "linear": 1, "bands": 2, "yarn": 3}

EXPORTED = (
    "eagle_status_string", "eagle_version", "eagle_selftest_wait",
    "eagle_draft_topk_workspace_size", "eagle_draft_topk",
    "eagle_tree_build", "eagle_tree_build_variant", "eagle_static_tree", "eagle_tree_mask",
    "eagle_tree_attn_workspace_size", "eagle_tree_attn_kernel_count", "eagle_tree_attn",
    "eagle_tree_attn_paged_workspace_size", "eagle_tree_attn_paged", "eagle_kv_commit",
    "eagle_verify_workspace_size", "eagle_verify", "eagle_verify_noalloc", "eagle_verify_draft",
    "eagle_page_map", "eagle_page_reserve", "eagle_page_release", "eagle_rope", "eagle_rope_freqs",
    "eagle_kv8_append", "eagle_kv8_commit", "eagle_kv8_commit_root", "eagle_tree_attn_kv8_workspace_size", "eagle_tree_attn_kv8",
    "eagle_qk_norm_rope", "eagle_kv8_bounds", "eagle_kv8_select_workspace_size", "eagle_kv8_select",
    "eagle_tree_attn_kv8_pages_workspace_size", "eagle_tree_attn_kv8_pages",
    "eagle_step_workspace_size", "eagle_step", "eagle_step_graph_create", "eagle_step_graph_launch",
    "eagle_step_graph_destroy",
)

_lib = None


class EagleError(RuntimeError):
    pass


_P, _I, _I64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


class StepArgs(ctypes.Structure):
    """eagle_step_args: every buffer of the four stage calls (device
    pointers) and the step's shapes, field for field as include/eagle.h
    declares them."""
    _fields_ = [
        ("dtype", _I), ("B", _I), ("D", _I), ("k", _I), ("m", _I), ("V", _I),
        ("Hq", _I), ("Hkv", _I), ("dh", _I), ("Lmax", _I),
        ("mode", _I), ("temperature", _F), ("scale", _F),
        ("draft_logits", _P), ("draft_ld", _I64),
        ("tok", _P), ("conf", _P), ("stats", _P),
        ("root_tok", _P), ("node_tok", _P), ("node_parent", _P), ("node_depth", _P),
        ("node_score", _P), ("node_src", _P), ("node_row", _P), ("mask", _P),
        ("q", _P), ("k_cache", _P), ("v_cache", _P), ("kv_len", _P), ("k_tree", _P), ("v_tree", _P),
        ("attn_out", _P), ("lse", _P),
        ("target", _P), ("target_ld", _I64), ("uniforms", _P),
        ("accept_len", _P), ("path_nodes", _P), ("out_tokens", _P),
        ("status", _P),
    ]


def load_library(path=LIB_PATH):
    """Load libeagle.so (built by tree_speculative_decoding_eagle_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise EagleError(f"{path} is missing: run `python -m tree_speculative_decoding_eagle_gb300.build`")
    lib = ctypes.CDLL(path)
    P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "eagle_status_string": (ctypes.c_char_p, [I]),
        "eagle_version": (I, []),
        "eagle_selftest_wait": (I, [ctypes.c_uint64, I, P, P, P]),
        "eagle_draft_topk_workspace_size": (SZ, [I, I, I, I]),
        "eagle_draft_topk": (I, [P, I, I, I, I, I, I64, P, P, P, P, P, SZ, P]),
        "eagle_tree_build": (I, [P, P, I, I, I, I, P, P, P, P, P, P, P, P, P, P]),
        "eagle_tree_build_variant": (I, [P, P, I, I, I, I, I, P, P, P, P, P, P, P, P, P, P]),
        "eagle_static_tree": (I, [P, P, I, I, I, P, P, I, P, P, P, P, P, P, P, P, P, P]),
        "eagle_tree_mask": (I, [P, I, I, P, P]),
        "eagle_tree_attn_workspace_size": (SZ, [I, I, I, I, I, I, I]),
        "eagle_tree_attn_kernel_count": (I, [I, I, I, I, I, I, I]),
        "eagle_tree_attn": (I, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, P, SZ, P]),
        "eagle_tree_attn_paged_workspace_size": (SZ, [I, I, I, I, I, I, I, I]),
        "eagle_tree_attn_paged": (I, [P, P, P, P, I, I, I, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, SZ, P]),
        "eagle_kv_commit": (I, [P, P, I, I, I, I, I, P, P, I, P, P, I, P, I, I, I, P, P, P, P]),
        "eagle_verify_workspace_size": (SZ, [I, I, I]),
        "eagle_verify": (I, [P, I, I64, P, P, I, I, I, I, I, F, P, P, P, P, P, P, SZ, P]),
        "eagle_verify_noalloc": (I, [P, I, I64, P, P, I, I, I, I, I, F, P, P, P, P, P, P]),
        "eagle_verify_draft": (I, [P, P, I, I64, I64, P, P, P, I, I, I, I, I, F, P, P, P, P, P, P]),
        "eagle_page_map": (I, [P, P, I, I, I, I, P, P, P, P, P, I, P, P, P]),
        "eagle_page_reserve": (I, [P, P, I, I, I, I, P, P, P, P, P, I, P, P, P, P]),
        "eagle_page_release": (I, [P, I, I, I, I, P, P, P, P, P, P]),
        "eagle_rope": (I, [P, P, P, I, I, I, I, I, I, I64, I64, I64, P, I, I, F, P, P, I, P, P, P, P]),
        "eagle_rope_freqs": (I, [I, ctypes.c_double, I, ctypes.c_double, I, ctypes.c_double, ctypes.c_double, P, P]),
        "eagle_kv8_append": (I, [P, P, I, I, I, I, I64, I64, P, P, P, P, P, I, I, P, P]),
        "eagle_kv8_commit": (I, [P, P, I, I, I, I, I, P, P, I, P, P, P, P, P, I, I, I, P, P, P, P]),
        "eagle_kv8_commit_root": (I, [P, P, I, I, I, I, I, P, P, I, P, P, P, P, P, I, I, I, P, P, P, P]),
        "eagle_tree_attn_kv8_workspace_size": (SZ, [I, I, I, I, I, I, I, I]),
        "eagle_tree_attn_kv8": (I, [P, P, P, P, P, P, I, I, I, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, SZ, P]),
        "eagle_qk_norm_rope": (I, [P, P, P, I, I, I, I, I, I, I64, I64, I64, P, P, F, F, P, I, I, F, P, P, I, P, P, P, P]),
        "eagle_kv8_bounds": (I, [P, P, I, I, I, P, P, I, I, I, P, P, P]),
        "eagle_kv8_select_workspace_size": (SZ, [I, I, I, I, I, I, I, I]),
        "eagle_kv8_select": (I, [P, I, P, P, P, I, I, I, P, I, I, I, I, I, I, I, I, P, P, P, P, SZ, P]),
        "eagle_tree_attn_kv8_pages_workspace_size": (SZ, [I, I, I, I, I, I, I, I, I]),
        "eagle_tree_attn_kv8_pages": (I, [P, P, P, P, P, P, I, I, I, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, P, SZ, P]),
        "eagle_step_workspace_size": (SZ, [ctypes.POINTER(StepArgs)]),
        "eagle_step": (I, [ctypes.POINTER(StepArgs), P, SZ, P]),
        "eagle_step_graph_create": (I, [ctypes.POINTER(StepArgs), P, SZ, ctypes.POINTER(P)]),
        "eagle_step_graph_launch": (I, [P, P]),
        "eagle_step_graph_destroy": (I, [P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise EagleError(f"unsupported dtype {t.dtype}")


def _check(rc, what):
    if rc != 0:
        msg = load_library().eagle_status_string(rc).decode()
        raise EagleError(f"{what} failed: {msg} ({rc})")


def _cuda(t, name):
    if not t.is_cuda:
        raise EagleError(f"{name} must be a CUDA tensor")
    return t


class Workspace:
    """Zero-initialised device scratch, grown on demand and reused."""

    def __init__(self, device=None):
        self.device = device
        self.buf = None

    def get(self, nbytes):
        if nbytes == 0:
            return None, 0
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=self.device or "cuda")
        return self.buf, self.buf.numel()


def draft_topk(logits, k, tok=None, conf=None, stats=None, workspace=None, status=None,
               stream=None):
    """logits [B, D, k, V(ld)] -> tok int32 [B,D,k,k], conf f32, stats f32 [B,D,k,2]."""
    lib = load_library()
    _cuda(logits, "logits")
    B, D, kk, V = logits.shape
    if kk != k or logits.stride(-1) != 1:
        raise EagleError("logits must be [B, D, k, V] with unit stride in V")
    ld = logits.stride(2)
    if logits.stride(1) != k * ld or logits.stride(0) != D * k * ld:
        raise EagleError("logits rows must be evenly spaced")
    dev = logits.device
    tok = tok if tok is not None else torch.empty((B, D, k, k), dtype=torch.int32, device=dev)
    conf = conf if conf is not None else torch.empty((B, D, k, k), dtype=torch.float32, device=dev)
    stats = stats if stats is not None else torch.empty((B, D, k, 2), dtype=torch.float32, device=dev)
    ws = workspace or Workspace(dev)
    wbuf, wbytes = ws.get(lib.eagle_draft_topk_workspace_size(B, D, k, V))
    _check(lib.eagle_draft_topk(_ptr(logits), _dtype_code(logits), B, D, k, V, ld, _ptr(tok),
                                _ptr(conf), _ptr(stats), _ptr(status), _ptr(wbuf), wbytes,
                                _stream(stream)),
           "eagle_draft_topk")
    return tok, conf, stats


def tree_build(tok, conf, m, root_tok=None, with_mask=True, out=None, status=None, stream=None, flags=0):
    """tok/conf [B, D, k, k] -> dict of node arrays [B, m+1] (+ mask [B, m+1, W]).

    flags: 0 for the method, or TREE_CONFIDENCE_ONLY | TREE_NO_RERANK for the
    ablation variants (eagle_tree_build_variant)."""
    lib = load_library()
    _cuda(tok, "tok")
    B, D, k, _ = tok.shape
    n = m + 1
    dev = tok.device
    W = (n + 63) // 64
    o = out or {}
    o.setdefault("tok", torch.empty((B, n), dtype=torch.int32, device=dev))
    o.setdefault("parent", torch.empty((B, n), dtype=torch.int32, device=dev))
    o.setdefault("depth", torch.empty((B, n), dtype=torch.int32, device=dev))
    o.setdefault("score", torch.empty((B, n), dtype=torch.float32, device=dev))
    o.setdefault("src", torch.empty((B, n), dtype=torch.int32, device=dev))
    o.setdefault("row", torch.empty((B, n), dtype=torch.int32, device=dev))
    if with_mask:
        o.setdefault("mask", torch.empty((B, n, W), dtype=torch.int64, device=dev))
    if flags:
        _check(lib.eagle_tree_build_variant(_ptr(tok), _ptr(conf), B, D, k, m, int(flags), _ptr(root_tok),
                                            _ptr(o["tok"]), _ptr(o["parent"]), _ptr(o["depth"]),
                                            _ptr(o["score"]), _ptr(o["src"]), _ptr(o["row"]),
                                            _ptr(o.get("mask")), _ptr(status), _stream(stream)),
               "eagle_tree_build_variant")
    else:
        _check(lib.eagle_tree_build(_ptr(tok), _ptr(conf), B, D, k, m, _ptr(root_tok), _ptr(o["tok"]),
                                    _ptr(o["parent"]), _ptr(o["depth"]), _ptr(o["score"]),
                                    _ptr(o["src"]), _ptr(o["row"]), _ptr(o.get("mask")),
                                    _ptr(status), _stream(stream)), "eagle_tree_build")
    return o


def static_tree(tok, conf, tree_parent, tree_rank, root_tok=None, with_mask=True, out=None, status=None,
                stream=None):
    """EAGLE-1 static tree: tok/conf [B, D, k, k] and a template (tree_parent,
    tree_rank int32 [n] on the device) -> node arrays [B, n] (+ mask)."""
    lib = load_library()
    _cuda(tok, "tok")
    B, D, k, _ = tok.shape
    n = int(tree_parent.shape[0])
    dev = tok.device
    W = (n + 63) // 64
    o = out or {}
    for key, dt in (("tok", torch.int32), ("parent", torch.int32), ("depth", torch.int32),
                    ("score", torch.float32), ("src", torch.int32), ("row", torch.int32)):
        o.setdefault(key, torch.empty((B, n), dtype=dt, device=dev))
    if with_mask:
        o.setdefault("mask", torch.empty((B, n, W), dtype=torch.int64, device=dev))
    _check(lib.eagle_static_tree(_ptr(tok), _ptr(conf), B, D, k, _ptr(tree_parent), _ptr(tree_rank), n,
                                 _ptr(root_tok), _ptr(o["tok"]), _ptr(o["parent"]), _ptr(o["depth"]),
                                 _ptr(o["score"]), _ptr(o["src"]), _ptr(o["row"]), _ptr(o.get("mask")),
                                 _ptr(status), _stream(stream)), "eagle_static_tree")
    return o


def tree_mask(node_parent, mask=None, stream=None):
    """node_parent int32 [B, n] -> mask int64 (uint64 bit pattern) [B, n, W]."""
    lib = load_library()
    _cuda(node_parent, "node_parent")
    B, n = node_parent.shape
    W = (n + 63) // 64
    mask = mask if mask is not None else torch.empty((B, n, W), dtype=torch.int64, device=node_parent.device)
    _check(lib.eagle_tree_mask(_ptr(node_parent), B, n, _ptr(mask), _stream(stream)), "eagle_tree_mask")
    return mask


def tree_attn(q, k_cache, v_cache, kv_len, k_tree, v_tree, mask, scale=None, out=None,
              lse=None, workspace=None, status=None, stream=None):
    """q [B,n,Hq,dh], caches [B,Hkv,Lmax,dh], tree KV [B,Hkv,n,dh] -> out, lse."""
    lib = load_library()
    for t, nm in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (k_tree, "k_tree"),
                  (v_tree, "v_tree"), (kv_len, "kv_len"), (mask, "mask")):
        _cuda(t, nm)
        if not t.is_contiguous():
            raise EagleError(f"{nm} must be contiguous")
    B, n, Hq, dh = q.shape
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    dt = _dtype_code(q)
    scale = dh ** -0.5 if scale is None else scale
    out = out if out is not None else torch.empty_like(q)
    lse = lse if lse is not None else torch.empty((B, n, Hq), dtype=torch.float32, device=q.device)
    ws = workspace or Workspace(q.device)
    wbuf, wbytes = ws.get(lib.eagle_tree_attn_workspace_size(dt, B, n, Hq, Hkv, dh, Lmax))
    _check(lib.eagle_tree_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), _ptr(k_tree),
                               _ptr(v_tree), _ptr(mask), dt, B, n, Hq, Hkv, dh, Lmax,
                               ctypes.c_float(scale), _ptr(out), _ptr(lse), _ptr(status),
                               _ptr(wbuf), wbytes, _stream(stream)), "eagle_tree_attn")
    return out, lse


def verify(target, node_tok, node_parent, D, mode, temperature=1.0, uniforms=None,
           accept_len=None, path_nodes=None, out_tokens=None, status=None, workspace=None,
           stream=None):
    """target [B, m+1, V] -> accept_len [B], path_nodes [B, D+1], out_tokens [B, D+1]."""
    lib = load_library()
    _cuda(target, "target")
    B, n, V = target.shape
    if target.stride(-1) != 1 or target.stride(0) != n * target.stride(1):
        raise EagleError("target must be [B, m+1, V] with evenly spaced rows")
    ld = target.stride(1)
    m = n - 1
    dev = target.device
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    path_nodes = path_nodes if path_nodes is not None else torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    ws = workspace or Workspace(dev)
    wbuf, wbytes = ws.get(lib.eagle_verify_workspace_size(B, m, V))
    mode_code = GREEDY if mode in ("greedy", GREEDY) else SAMPLE
    _check(lib.eagle_verify(_ptr(target), _dtype_code(target), ld, _ptr(node_tok), _ptr(node_parent),
                            B, m, D, V, mode_code, ctypes.c_float(temperature), _ptr(uniforms),
                            _ptr(accept_len), _ptr(path_nodes), _ptr(out_tokens), _ptr(status),
                            _ptr(wbuf), wbytes, _stream(stream)), "eagle_verify")
    return accept_len, path_nodes, out_tokens


def verify_noalloc(target, node_tok, node_parent, D, mode, temperature=1.0, uniforms=None,
                   accept_len=None, path_nodes=None, out_tokens=None, status=None, stream=None):
    """verify() for callers that cannot allocate device memory for a workspace
    (eagle_verify_noalloc): the chunk records live in a fixed array inside the
    library, so calls that overlap on the GPU race.  Same results as verify()."""
    lib = load_library()
    _cuda(target, "target")
    B, n, V = target.shape
    if target.stride(-1) != 1 or target.stride(0) != n * target.stride(1):
        raise EagleError("target must be [B, m+1, V] with evenly spaced rows")
    dev = target.device
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    path_nodes = path_nodes if path_nodes is not None else torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    mode_code = GREEDY if mode in ("greedy", GREEDY) else SAMPLE
    _check(lib.eagle_verify_noalloc(_ptr(target), _dtype_code(target), target.stride(1), _ptr(node_tok),
                                    _ptr(node_parent), B, n - 1, D, V, mode_code, ctypes.c_float(temperature),
                                    _ptr(uniforms), _ptr(accept_len), _ptr(path_nodes), _ptr(out_tokens),
                                    _ptr(status), _stream(stream)), "eagle_verify_noalloc")
    return accept_len, path_nodes, out_tokens


def verify_draft(target, draft, node_tok, node_parent, node_row, D, temperature, uniforms, accept_len=None,
                 path_nodes=None, out_tokens=None, status=None, stream=None):
    """Speculative-sampling verification against the draft distributions:
    target [B, m+1, V] and draft [B, D, k, V] logits (same dtype), node
    arrays [B, m+1] -> (accept_len [B], path_nodes [B, D+1], out_tokens [B, D+1])."""
    lib = load_library()
    _cuda(target, "target")
    B, n, V = target.shape
    k = draft.shape[2]
    assert draft.shape[0] == B and draft.shape[1] == D and draft.dtype == target.dtype
    dev = target.device
    accept_len = accept_len if accept_len is not None else torch.empty(B, dtype=torch.int32, device=dev)
    path_nodes = path_nodes if path_nodes is not None else torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    out_tokens = out_tokens if out_tokens is not None else torch.empty((B, D + 1), dtype=torch.int32, device=dev)
    _check(lib.eagle_verify_draft(_ptr(target), _ptr(draft), _dtype_code(target), target.stride(1),
                                  draft.stride(2), _ptr(node_tok), _ptr(node_parent), _ptr(node_row), B, n - 1,
                                  D, k, V, ctypes.c_float(temperature), _ptr(uniforms), _ptr(accept_len),
                                  _ptr(path_nodes), _ptr(out_tokens), _ptr(status), _stream(stream)),
           "eagle_verify_draft")
    return accept_len, path_nodes, out_tokens


def tree_attn_paged(q, k_pages, v_pages, block_table, kv_len, k_tree, v_tree, mask, scale=None, out=None,
                    lse=None, workspace=None, status=None, stream=None):
    """Tree attention over a paged prefix: k_pages/v_pages [num_pages, Hkv,
    page_size, dh], block_table int32 [B, max_pages]; else as tree_attn."""
    lib = load_library()
    _cuda(q, "q")
    B, n, Hq, dh = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    max_pages = block_table.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    out = out if out is not None else torch.empty_like(q)
    lse = lse if lse is not None else torch.empty((B, n, Hq), dtype=torch.float32, device=q.device)
    ws = workspace or Workspace(q.device)
    dt = _dtype_code(q)
    wbuf, wbytes = ws.get(lib.eagle_tree_attn_paged_workspace_size(dt, B, n, Hq, Hkv, dh, max_pages, page_size))
    _check(lib.eagle_tree_attn_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), max_pages,
                                     page_size, num_pages, _ptr(kv_len), _ptr(k_tree), _ptr(v_tree), _ptr(mask),
                                     dt, B, n, Hq, Hkv, dh, ctypes.c_float(scale), _ptr(out), _ptr(lse),
                                     _ptr(status), _ptr(wbuf), wbytes, _stream(stream)), "eagle_tree_attn_paged")
    return out, lse


def kv_commit(k_tree, v_tree, accept_len, path_nodes, k_cache, v_cache, kv_len, block_table=None,
              slot_mapping=None, status=None, stream=None):
    """Append the accepted path's K/V rows to the cache (contiguous [B, Hkv,
    Lmax, dh], or page pools [num_pages, Hkv, page_size, dh] with a
    block_table); kv_len is updated in place.  Returns slot_mapping [B, n]."""
    lib = load_library()
    _cuda(k_tree, "k_tree")
    B, Hkv, n, dh = k_tree.shape
    D = path_nodes.shape[1] - 1
    if slot_mapping is None:
        slot_mapping = torch.empty((B, n), dtype=torch.int32, device=k_tree.device)
    if block_table is None:
        Lmax, max_pages, page_size, num_pages = k_cache.shape[2], 0, 0, 0
    else:
        Lmax = 0
        num_pages, _, page_size, _ = k_cache.shape
        max_pages = block_table.shape[1]
    _check(lib.eagle_kv_commit(_ptr(k_tree), _ptr(v_tree), _dtype_code(k_tree), B, n, Hkv, dh, _ptr(accept_len),
                               _ptr(path_nodes), D, _ptr(k_cache), _ptr(v_cache), Lmax, _ptr(block_table),
                               max_pages, page_size, num_pages, _ptr(kv_len), _ptr(slot_mapping), _ptr(status),
                               _stream(stream)), "eagle_kv_commit")
    return slot_mapping


# ---- the serving loop around the step: pages, positions, the 8-bit cache ------

def _need(t, name, dtype, shape, dev):
    """Address of t, if it is a contiguous tensor of that type and shape (None:
    any) on CUDA device number dev."""
    if t.get_device() != dev or t.dtype != dtype or (shape is not None and t.shape != shape) or not t.is_contiguous():
        what = "" if shape is None else f" of shape {tuple(shape)}"
        raise EagleError(f"{name} must be a contiguous {dtype} CUDA tensor{what} on device {dev}, not {t.dtype} "
                         f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _maybe(t, name, dtype, shape, dev):
    return None if t is None else _need(t, name, dtype, shape, dev)


def _device_of(t, name):
    dev = t.get_device()
    if dev < 0:
        raise EagleError(f"{name} must be a CUDA tensor")
    return dev


@functools.lru_cache(maxsize=1024)
def _workspace_size(name, dev, *sizes):
    """Bytes that the named query asks for on CUDA device number dev: a number
    of the sizes alone, kept because asking takes a microsecond of a call that
    takes fourteen."""
    with torch.cuda.device(dev):
        return getattr(load_library(), name)(*sizes)


def _call(what, fn, dev, stream, *args):
    """fn(*args, stream) with device number `dev` current, on its current stream
    unless one is given."""
    # the stream's handle without a Stream object around it and the device without
    # a look at the runtime's state (a CUDA tensor is at hand): two microseconds of
    # a call that takes nine
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        _check(rc, what)


def page_map(kv_len, new_len, block_table, page_count, free_pages, free_count, page_size, slot_map=None,
             new_start=None, status=None, stream=None, granted=None):
    """Maps the pages that new_len [B] more tokens need and lists the tokens'
    slots (eagle_page_map).  kv_len, new_len, page_count int32 [B], block_table
    int32 [B, max_pages], free_pages int32 [num_pages], free_count int32 [1];
    block_table, page_count and free_count are updated in place.  slot_map
    int32 [T] (optional) receives the slots of the new tokens, request by
    request, then -1; new_start int32 [B+1] (optional) their first indices.
    Returns slot_map.  Too few free pages leave everything as it was and set
    `status` to -6; with `granted` int32 [1] (eagle_page_reserve) slot_map is
    then -1 throughout, and granted 0 instead of 1."""
    lib = load_library()
    dev, i32 = _device_of(kv_len, "kv_len"), torch.int32
    B, max_pages = block_table.shape
    num_pages = free_pages.shape[0]
    name, more = "eagle_page_map", ()
    if granted is not None:
        name, more = "eagle_page_reserve", (_need(granted, "granted", i32, (1,), dev),)
    _call(name, getattr(lib, name), dev, stream, _need(kv_len, "kv_len", i32, (B,), dev),
          _need(new_len, "new_len", i32, (B,), dev), B, page_size, max_pages, num_pages,
          _need(block_table, "block_table", i32, None, dev), _need(page_count, "page_count", i32, (B,), dev),
          _need(free_pages, "free_pages", i32, (num_pages,), dev), _need(free_count, "free_count", i32, (1,), dev),
          _maybe(slot_map, "slot_map", i32, None, dev), 0 if slot_map is None else slot_map.numel(),
          _maybe(new_start, "new_start", i32, (B + 1,), dev), *more, _maybe(status, "status", i32, None, dev))
    return slot_map


def page_release(keep_len, block_table, page_count, free_pages, free_count, page_size, status=None, stream=None):
    """Gives back the pages past keep_len [B] tokens of each request
    (eagle_page_release): 0 ends a request, its kv_len trims it to what it
    uses, a negative length leaves it alone.  The other arrays are those of
    page_map, updated in place."""
    lib = load_library()
    dev, i32 = _device_of(keep_len, "keep_len"), torch.int32
    B, max_pages = block_table.shape
    num_pages = free_pages.shape[0]
    _call("eagle_page_release", lib.eagle_page_release, dev, stream, _need(keep_len, "keep_len", i32, (B,), dev), B,
          page_size, max_pages, num_pages, _need(block_table, "block_table", i32, None, dev),
          _need(page_count, "page_count", i32, (B,), dev), _need(free_pages, "free_pages", i32, (num_pages,), dev),
          _need(free_count, "free_count", i32, (1,), dev), _maybe(status, "status", i32, None, dev))


def rope_freqs(rot_dim, theta=10000.0, kind="plain", stretch=1.0, orig_len=4096, low=1.0, high=None, device=None):
    """Frequencies of rope() (eagle_rope_freqs): (inv_freq float64 [rot_dim/2]
    on `device`, factor).  kind: "plain", "linear", "bands" (stretched below
    `low` turns over orig_len tokens, kept above `high`) or "yarn".  `high` is
    4 for "bands" and 32 for "yarn" where it is not given."""
    if kind not in ROPE_KINDS:
        raise EagleError(f"unknown kind {kind!r}: one of {sorted(ROPE_KINDS)}")
    if high is None:
        high = 4.0 if kind == "bands" else 32.0
    out = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64)
    factor = ctypes.c_float()
    _check(load_library().eagle_rope_freqs(int(rot_dim), float(theta), ROPE_KINDS[kind], float(stretch),
                                           int(orig_len), float(low), float(high), out.data_ptr(),
                                           ctypes.addressof(factor)), "eagle_rope_freqs")
    return out.to(device or "cuda"), factor.value


def _heads(t, name, B, n, dh, dtype, device):
    """Node stride of [B, n, heads, dh] whose heads are dense and whose nodes
    are evenly spaced."""
    if t.get_device() != device or t.dtype != dtype:
        raise EagleError(f"{name} must be a {dtype} CUDA tensor on device {device}")
    shape = t.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != n or shape[3] != dh:
        raise EagleError(f"{name} must be [B, n, heads, dh]")
    heads = shape[2]
    sb, sn, sh, sd = t.stride()
    if n == 1 and B > 1:
        sn = sb                # the one node's stride says nothing
    elif n == 1:
        sn = max(sn, heads * dh)
    if sd != 1 or (heads > 1 and sh != dh) or (B > 1 and sb != n * sn):
        raise EagleError(f"{name} must have dense heads and evenly spaced nodes")
    return sn


def _rope_args(q, k, v, inv_freq, pos_base, pos_off, shift, factor, interleaved, q_out, k_tree, v_tree):
    """What rope() and qk_norm_rope() hand on, checked: the arguments up to the
    strides, and those from the frequencies on with the three outputs behind them."""
    dev, dt = _device_of(q, "q"), q.dtype
    if q.dim() != 4 or k.dim() != 4:
        raise EagleError("q and k must be [B, n, heads, dh]")
    B, n, Hq, dh = q.shape
    Hkv = k.shape[2]
    ld_q, ld_k = _heads(q, "q", B, n, dh, dt, dev), _heads(k, "k", B, n, dh, dt, dev)
    ld_v = 0
    if v is not None:
        ld_v = _heads(v, "v", B, n, dh, dt, dev)
        if v.shape[2] != Hkv:
            raise EagleError("k and v must have the same heads")
    if q_out is None:
        q_out = q.new_empty((B, n, Hq, dh))
    if k_tree is None:
        k_tree = q.new_empty((B, Hkv, n, dh))
    if v_tree is None and v is not None:
        v_tree = q.new_empty((B, Hkv, n, dh))
    i32 = torch.int32
    head = (q.data_ptr(), k.data_ptr(), None if v is None else v.data_ptr(), _dtype_code(q), B, n, Hq, Hkv, dh, ld_q, ld_k, ld_v)
    tail = [_need(inv_freq, "inv_freq", torch.float64, None, dev), 2 * inv_freq.numel(), int(interleaved), factor,
            _maybe(pos_base, "pos_base", i32, (B,), dev), _maybe(pos_off, "pos_off", i32, (B, n), dev), shift,
            _need(q_out, "q_out", dt, (B, n, Hq, dh), dev), _need(k_tree, "k_tree", dt, (B, Hkv, n, dh), dev),
            _maybe(v_tree, "v_tree", dt, (B, Hkv, n, dh), dev), (q_out, k_tree, v_tree)]
    return head, tail


def rope(q, k, v, inv_freq, pos_base=None, pos_off=None, shift=0, factor=1.0, interleaved=False, q_out=None,
         k_tree=None, v_tree=None, stream=None):
    """Rotary positions (eagle_rope).  q [B, n, Hq, dh], k and v [B, n, Hkv, dh]
    (v may be None), nodes evenly spaced, so slices of one fused projection do
    -> q_out [B, n, Hq, dh], k_tree and v_tree [B, Hkv, n, dh], as tree_attn
    takes them.  Node i of sequence b is at position pos_base[b] + pos_off[b,
    i] + shift (0 and i where they are None).  inv_freq float64 [rot_dim/2]
    and factor as rope_freqs gives them."""
    if stream is not None:     # what is allocated here belongs to that stream
        with torch.cuda.stream(stream):
            return rope(q, k, v, inv_freq, pos_base, pos_off, shift, factor, interleaved, q_out, k_tree, v_tree)
    lib = load_library()
    head, tail = _rope_args(q, k, v, inv_freq, pos_base, pos_off, shift, factor, interleaved, q_out, k_tree, v_tree)
    out = tail.pop()
    _call("eagle_rope", lib.eagle_rope, q.get_device(), None, *head, *tail)
    return out


def qk_norm_rope(q, k, v, inv_freq, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0, pos_base=None, pos_off=None,
                 shift=0, factor=1.0, interleaved=False, q_out=None, k_tree=None, v_tree=None, stream=None):
    """rope() after a norm of each head of q and k (eagle_qk_norm_rope): a head
    x becomes x / sqrt(mean(x^2) + eps) * (weight + weight_offset), then turns.
    q_weight, k_weight [dh] of q's type, or None for a norm without a weight; the
    other arguments and what is returned are rope()'s."""
    if stream is not None:     # what is allocated here belongs to that stream
        with torch.cuda.stream(stream):
            return qk_norm_rope(q, k, v, inv_freq, q_weight, k_weight, eps, weight_offset, pos_base, pos_off, shift, factor,
                                interleaved, q_out, k_tree, v_tree)
    lib = load_library()
    head, tail = _rope_args(q, k, v, inv_freq, pos_base, pos_off, shift, factor, interleaved, q_out, k_tree, v_tree)
    out = tail.pop()
    dev, dt, shape = q.get_device(), q.dtype, q.shape[3:]
    _call("eagle_qk_norm_rope", lib.eagle_qk_norm_rope, dev, None, *head, _maybe(q_weight, "q_weight", dt, shape, dev),
          _maybe(k_weight, "k_weight", dt, shape, dev), weight_offset, eps, *tail)
    return out


_POOL_TYPES = (torch.float8_e4m3fn, torch.uint8)


def _pools(k_pages, v_pages, k_scale, v_scale, device):
    """The 8-bit cache's four pointers, checked against each other."""
    if k_pages.dtype not in _POOL_TYPES or k_pages.dim() != 4:
        raise EagleError("k_pages must be float8_e4m3fn (or uint8) [num_pages, Hkv, page_size, dh]")
    shape = k_pages.shape
    return (_need(k_pages, "k_pages", k_pages.dtype, None, device), _need(v_pages, "v_pages", k_pages.dtype, shape, device),
            _need(k_scale, "k_scale", torch.float32, shape[:2], device),
            _need(v_scale, "v_scale", torch.float32, shape[:2], device))


def kv8_append(k, v, slot_map, k_pages, v_pages, k_scale, v_scale, status=None, stream=None):
    """Writes tokens' keys and values (k, v [T, Hkv, dh], any token and head
    strides but those of a broadcast, the same for both) to the slots slot_map
    int32 [T] of the 8-bit cache (eagle_kv8_append): k_pages, v_pages float8_e4m3fn [num_pages, Hkv,
    page_size, dh], k_scale, v_scale float32 [num_pages, Hkv]."""
    lib = load_library()
    dev, shape, stride = _device_of(k, "k"), k.shape, k.stride()
    if len(shape) != 3:
        raise EagleError("k must be [T, Hkv, dh]")
    if v.shape != shape or v.stride() != stride or v.dtype != k.dtype or v.get_device() != dev:
        raise EagleError("v must have k's shape, strides, type and device")
    T, Hkv, dh = shape
    per_token, per_head, per_element = stride
    if T and per_element != 1:
        raise EagleError("k must have unit stride in dh")
    num_pages, H, page_size, d = k_pages.shape
    if H != Hkv or d != dh:
        raise EagleError("k must have the pages' heads and head dimension")
    if T > 1 and Hkv > 1 and (per_token == 0 or per_head == 0):
        raise EagleError("k must not be a broadcast view")
    _call("eagle_kv8_append", lib.eagle_kv8_append, dev, stream, k.data_ptr(), v.data_ptr(), _dtype_code(k), T, Hkv,
          dh, per_token, per_head, _need(slot_map, "slot_map", torch.int32, (T,), dev),
          *_pools(k_pages, v_pages, k_scale, v_scale, dev), page_size, num_pages,
          _maybe(status, "status", torch.int32, None, dev))


def kv8_commit(k_tree, v_tree, accept_len, path_nodes, k_pages, v_pages, k_scale, v_scale, kv_len, block_table,
               slot_mapping=None, status=None, stream=None, root=False):
    """kv_commit into the 8-bit cache (eagle_kv8_commit): the accepted path's
    rows of k_tree, v_tree [B, Hkv, n, dh] join the pages, kv_len is updated
    in place.  With `root` (eagle_kv8_commit_root) the root's rows go before
    them, and kv_len is the attention's; without it the root is stored already.
    Returns slot_mapping [B, n]."""
    if stream is not None:     # what is allocated here belongs to that stream
        with torch.cuda.stream(stream):
            return kv8_commit(k_tree, v_tree, accept_len, path_nodes, k_pages, v_pages, k_scale, v_scale, kv_len,
                              block_table, slot_mapping, status, root=root)
    lib = load_library()
    dev, i32 = _device_of(k_tree, "k_tree"), torch.int32
    B, Hkv, n, dh = k_tree.shape
    num_pages, H, page_size, d = k_pages.shape
    if H != Hkv or d != dh:
        raise EagleError("k_tree must have the pages' heads and head dimension")
    D = path_nodes.shape[1] - 1
    max_pages = block_table.shape[1]
    if slot_mapping is None:
        slot_mapping = torch.empty((B, n), dtype=i32, device=k_tree.device)
    name = "eagle_kv8_commit_root" if root else "eagle_kv8_commit"
    _call(name, getattr(lib, name), dev, None, _need(k_tree, "k_tree", k_tree.dtype, None, dev),
          _need(v_tree, "v_tree", k_tree.dtype, (B, Hkv, n, dh), dev), _dtype_code(k_tree), B, n, Hkv, dh,
          _need(accept_len, "accept_len", i32, (B,), dev), _need(path_nodes, "path_nodes", i32, (B, D + 1), dev), D,
          *_pools(k_pages, v_pages, k_scale, v_scale, dev),
          _need(block_table, "block_table", i32, (B, max_pages), dev), max_pages, page_size, num_pages,
          _need(kv_len, "kv_len", i32, (B,), dev), _need(slot_mapping, "slot_mapping", i32, (B, n), dev),
          _maybe(status, "status", i32, None, dev))
    return slot_mapping


def tree_attn_kv8(q, k_pages, v_pages, k_scale, v_scale, block_table, kv_len, k_tree, v_tree, mask, scale=None,
                  out=None, lse=None, workspace=None, status=None, stream=None):
    """Tree attention over the 8-bit paged cache (eagle_tree_attn_kv8): q
    [B, n, Hq, dh] and k_tree, v_tree [B, Hkv, n, dh] bf16, pages and scales as
    kv8_append writes them, block_table int32 [B, max_pages]; else as
    tree_attn.  n = 1 with mask 1 decodes single tokens."""
    if stream is not None:     # what is allocated here belongs to that stream
        with torch.cuda.stream(stream):
            return tree_attn_kv8(q, k_pages, v_pages, k_scale, v_scale, block_table, kv_len, k_tree, v_tree, mask,
                                 scale, out, lse, workspace, status)
    lib = load_library()
    dev, dt = _device_of(q, "q"), q.dtype
    B, n, Hq, dh = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    max_pages = block_table.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    if out is None:
        out = torch.empty((B, n, Hq, dh), dtype=dt, device=q.device)
    if lse is None:
        lse = torch.empty((B, n, Hq), dtype=torch.float32, device=q.device)
    code = _dtype_code(q)
    if k_pages.shape[3] != dh:
        raise EagleError("q must have the pages' head dimension")
    need = lib.eagle_tree_attn_kv8_workspace_size(code, B, n, Hq, Hkv, dh, max_pages, page_size)
    buf, nbytes = (workspace or Workspace(q.device)).get(need)
    if buf is not None and buf.get_device() != dev:
        raise EagleError(f"the workspace must be on device {dev}, not on {buf.device}")
    _call("eagle_tree_attn_kv8", lib.eagle_tree_attn_kv8, dev, None, _need(q, "q", dt, None, dev),
          *_pools(k_pages, v_pages, k_scale, v_scale, dev),
          _need(block_table, "block_table", torch.int32, (B, max_pages), dev), max_pages, page_size, num_pages,
          _need(kv_len, "kv_len", torch.int32, (B,), dev), _need(k_tree, "k_tree", dt, (B, Hkv, n, dh), dev),
          _need(v_tree, "v_tree", dt, (B, Hkv, n, dh), dev),
          _need(mask, "mask", torch.int64, (B, n, (n + 63) // 64), dev), code, B, n, Hq, Hkv, dh, scale,
          _need(out, "out", dt, (B, n, Hq, dh), dev), _need(lse, "lse", torch.float32, (B, n, Hq), dev),
          _maybe(status, "status", torch.int32, None, dev), None if buf is None else buf.data_ptr(), nbytes)
    return out, lse


def _bounds(k_bounds, num_pages, Hkv, dh, dev):
    if k_bounds.dtype not in _POOL_TYPES:
        raise EagleError("k_bounds must be float8_e4m3fn (or uint8) [num_pages, Hkv, 2, dh]")
    return _need(k_bounds, "k_bounds", k_bounds.dtype, (num_pages, Hkv, 2, dh), dev)


def kv8_bounds(k_pages, block_table, from_len, kv_len, k_bounds, status=None, stream=None):
    """Renews the bounds k_bounds float8_e4m3fn [num_pages, Hkv, 2, dh] (the least
    and the greatest number of each column, rounded outwards to halves, in units
    of the page's scale) of the pages that hold positions from_len[b] ..
    kv_len[b]-1 (eagle_kv8_bounds): after an append or a commit, with the
    lengths before it."""
    lib = load_library()
    dev, i32 = _device_of(k_pages, "k_pages"), torch.int32
    if k_pages.dtype not in _POOL_TYPES or k_pages.dim() != 4:
        raise EagleError("k_pages must be float8_e4m3fn (or uint8) [num_pages, Hkv, page_size, dh]")
    num_pages, Hkv, page_size, dh = k_pages.shape
    B, max_pages = block_table.shape
    _call("eagle_kv8_bounds", lib.eagle_kv8_bounds, dev, stream, _need(k_pages, "k_pages", k_pages.dtype, None, dev),
          _need(block_table, "block_table", i32, (B, max_pages), dev), max_pages, page_size, num_pages,
          _need(from_len, "from_len", i32, (B,), dev), _need(kv_len, "kv_len", i32, (B,), dev), B, Hkv, dh,
          _bounds(k_bounds, num_pages, Hkv, dh, dev), _maybe(status, "status", i32, None, dev))


def kv8_select(q, k_bounds, k_scale, block_table, kv_len, page_size, top, first=1, last=1, out=None, score=None, workspace=None,
               status=None, stream=None):
    """The pages of the prefix that each node and KV head is to attend to
    (eagle_kv8_select): q [B, n, Hq, dh] bf16, k_bounds as kv8_bounds writes them,
    k_scale float32 [num_pages, Hkv], block_table int32 [B, max_pages] -> sel int32
    [B, n, Hkv, top], logical pages in ascending order, then -1: the first `first` and
    the last `last` pages of the prefix and those whose bounds allow the greatest
    product with the query, each row of it rounded to whole numbers of at most 128
    times a power of two.  `score` float32 of the same shape receives theirs."""
    if stream is not None:     # what is allocated here belongs to that stream
        with torch.cuda.stream(stream):
            return kv8_select(q, k_bounds, k_scale, block_table, kv_len, page_size, top, first, last, out, score, workspace, status)
    lib = load_library()
    dev, i32 = _device_of(q, "q"), torch.int32
    B, n, Hq, dh = q.shape
    num_pages, Hkv = k_scale.shape
    max_pages = block_table.shape[1]
    if out is None:
        out = torch.empty((B, n, Hkv, top), dtype=i32, device=q.device)
    code = _dtype_code(q)
    need = _workspace_size("eagle_kv8_select_workspace_size", dev, code, B, n, Hq, Hkv, dh, max_pages, page_size)
    buf, nbytes = (workspace or Workspace(q.device)).get(need)
    if buf is not None and buf.get_device() != dev:
        raise EagleError(f"the workspace must be on device {dev}, not on {buf.device}")
    _call("eagle_kv8_select", lib.eagle_kv8_select, dev, None, _need(q, "q", q.dtype, None, dev), code,
          _bounds(k_bounds, num_pages, Hkv, dh, dev), _need(k_scale, "k_scale", torch.float32, None, dev),
          _need(block_table, "block_table", i32, (B, max_pages), dev), max_pages, page_size, num_pages,
          _need(kv_len, "kv_len", i32, (B,), dev), B, n, Hq, Hkv, dh, top, first, last,
          _need(out, "out", i32, (B, n, Hkv, top), dev), _maybe(score, "score", torch.float32, (B, n, Hkv, top), dev),
          _maybe(status, "status", i32, None, dev), None if buf is None else buf.data_ptr(), nbytes)
    return out


def tree_attn_kv8_pages(q, k_pages, v_pages, k_scale, v_scale, block_table, kv_len, k_tree, v_tree, mask, sel, scale=None,
                        out=None, lse=None, workspace=None, status=None, stream=None):
    """tree_attn_kv8 with the prefix of each node and KV head cut down to the
    pages that sel int32 [B, n, Hkv, top] lists, as kv8_select writes it
    (eagle_tree_attn_kv8_pages)."""
    if stream is not None:     # what is allocated here belongs to that stream
        with torch.cuda.stream(stream):
            return tree_attn_kv8_pages(q, k_pages, v_pages, k_scale, v_scale, block_table, kv_len, k_tree, v_tree, mask, sel,
                                       scale, out, lse, workspace, status)
    lib = load_library()
    dev, dt = _device_of(q, "q"), q.dtype
    B, n, Hq, dh = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    max_pages, top = block_table.shape[1], sel.shape[-1]
    scale = dh ** -0.5 if scale is None else scale
    if out is None:
        out = torch.empty((B, n, Hq, dh), dtype=dt, device=q.device)
    if lse is None:
        lse = torch.empty((B, n, Hq), dtype=torch.float32, device=q.device)
    code = _dtype_code(q)
    if k_pages.shape[3] != dh:
        raise EagleError("q must have the pages' head dimension")
    need = _workspace_size("eagle_tree_attn_kv8_pages_workspace_size", dev, code, B, n, Hq, Hkv, dh, top, max_pages, page_size)
    buf, nbytes = (workspace or Workspace(q.device)).get(need)
    if buf is not None and buf.get_device() != dev:
        raise EagleError(f"the workspace must be on device {dev}, not on {buf.device}")
    _call("eagle_tree_attn_kv8_pages", lib.eagle_tree_attn_kv8_pages, dev, None, _need(q, "q", dt, None, dev),
          *_pools(k_pages, v_pages, k_scale, v_scale, dev),
          _need(block_table, "block_table", torch.int32, (B, max_pages), dev), max_pages, page_size, num_pages,
          _need(kv_len, "kv_len", torch.int32, (B,), dev), _need(k_tree, "k_tree", dt, (B, Hkv, n, dh), dev),
          _need(v_tree, "v_tree", dt, (B, Hkv, n, dh), dev),
          _need(mask, "mask", torch.int64, (B, n, (n + 63) // 64), dev),
          _need(sel, "sel", torch.int32, (B, n, Hkv, top), dev), top, code, B, n, Hq, Hkv, dh, scale,
          _need(out, "out", dt, (B, n, Hq, dh), dev), _need(lse, "lse", torch.float32, (B, n, Hq), dev),
          _maybe(status, "status", torch.int32, None, dev), None if buf is None else buf.data_ptr(), nbytes)
    return out, lse


def selftest_wait(limit_ns=1_000_000, which=0, stream=None):
    """Runs eagle_selftest_wait: one warp waits on an mbarrier that nothing
    completes, with the kernels' own bounded-wait helper number `which` (0,
    1, 3 or 4, see include/eagle.h).  Returns (status
    code written by the device, nanoseconds waited); the status is
    EAGLE_ERR_TIMEOUT (-5) when the wait gave up as designed."""
    lib = load_library()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    elapsed = torch.zeros(1, dtype=torch.int64, device="cuda")
    _check(lib.eagle_selftest_wait(int(limit_ns), int(which), _ptr(status), _ptr(elapsed), _stream(stream)),
           "eagle_selftest_wait")
    (stream or torch.cuda.current_stream()).synchronize()
    return int(status.item()), int(elapsed.item())


def step_workspace_size(args):
    """Bytes of the one workspace eagle_step needs for these arguments."""
    return load_library().eagle_step_workspace_size(ctypes.byref(args))


def run_step(args, workspace, stream=None):
    """eagle_step: the four stages in order on the current stream.  `args`
    is a StepArgs (TreeStep.step_args builds one); `workspace` a Workspace."""
    lib = load_library()
    buf, nbytes = workspace.get(lib.eagle_step_workspace_size(ctypes.byref(args)))
    _check(lib.eagle_step(ctypes.byref(args), _ptr(buf), nbytes, _stream(stream)), "eagle_step")


class StepGraph:
    """eagle_step_graph_*: the step recorded once (after one plain run) and
    replayed by launch().  The buffers named in `args` and the workspace
    must stay allocated until close(); their contents may change between
    launches."""

    def __init__(self, args, workspace):
        lib = load_library()
        self._args = args
        buf, nbytes = workspace.get(lib.eagle_step_workspace_size(ctypes.byref(args)))
        self._ws = buf
        # the library's first run is on a stream of its own: the inputs'
        # producers on this stream must have finished
        torch.cuda.current_stream().synchronize()
        handle = ctypes.c_void_p()
        _check(lib.eagle_step_graph_create(ctypes.byref(args), _ptr(buf), nbytes, ctypes.byref(handle)),
               "eagle_step_graph_create")
        self._h = handle

    def launch(self, stream=None):
        if self._h is None:
            raise EagleError("the step graph is closed")
        _check(load_library().eagle_step_graph_launch(self._h, _stream(stream)), "eagle_step_graph_launch")

    def close(self):
        """Destroys the graph; its launches must have completed (synchronise
        the streams they were issued on first)."""
        if self._h is not None:
            _check(load_library().eagle_step_graph_destroy(self._h), "eagle_step_graph_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
