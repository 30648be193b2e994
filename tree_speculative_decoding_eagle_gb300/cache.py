"""A paged KV cache in 8 bits for a batch of requests and the layers of a model.

KV8Cache owns the pages (e4m3 numbers and their scales, one pool of keys and one of
values per layer), the block tables, the free list and the requests' lengths,
all on the device, and calls the library's entry points on the current stream:
    reserve  -> eagle_page_reserve  pages and slots for new tokens
    append   -> eagle_kv8_append    a prompt's (or single tokens') keys and values
    attend   -> eagle_tree_attn_kv8 draft nodes or single tokens over the cache
    commit   -> eagle_kv8_commit_root (root=True), eagle_kv8_commit
                                    the accepted path, in every layer
    release  -> eagle_page_release  pages back: of requests that ended, or past kv_len
kv_len counts the positions before the tree's root, which is node 0 of the tree,
at position kv_len.  So one step over a tree of depth D is
    reserve(D + 1) -> rope(pos_base=kv_len, pos_off=depth) -> attend -> verify
    -> commit(root=True) -> trim
(TreeStep.attend_kv8 and commit_kv8), and the bonus token is the next root.
Nothing is allocated and nothing synchronises after the constructor (but for the
attention's workspace, which grows to the largest call), so the calls can be
captured in a CUDA graph; a workspace that a larger call replaces stays, for the
graphs that hold its address.  Calls on one cache, and graphs captured from it,
follow one another; layers attended at the same time on several streams take a
Workspace each.  The layers share block tables and lengths.
"""
import torch

from . import EagleError, Workspace, kv8_append, kv8_commit, page_map, page_release, tree_attn_kv8


class _KeptWorkspace(Workspace):
    """A workspace whose outgrown buffers live as long as it does."""

    def __init__(self, device=None):
        super().__init__(device)
        self._outgrown = []

    def get(self, nbytes):
        before = self.buf
        got = super().get(nbytes)
        if before is not None and self.buf is not before:
            self._outgrown.append(before)
        return got


class KV8Cache:
    def __init__(self, B, Hkv, dh, page_size, num_pages, max_pages, layers=1, device="cuda"):
        if layers < 1:
            raise EagleError("a cache needs a layer")
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = page_size
        shape = (num_pages, Hkv, page_size, dh)
        self.k_pages = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(layers)]
        self.v_pages = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(layers)]
        self.k_scale = [torch.ones((num_pages, Hkv), device=device) for _ in range(layers)]
        self.v_scale = [torch.ones((num_pages, Hkv), device=device) for _ in range(layers)]
        self.block_table = torch.full((B, max_pages), -1, **i32)
        self.page_count = torch.zeros(B, **i32)
        self.free_pages = torch.arange(num_pages - 1, -1, -1, **i32)      # page 0 on top
        self.free_count = torch.full((1,), num_pages, **i32)
        self.kv_len = torch.zeros(B, **i32)
        self.status = torch.zeros(1, **i32)
        self._len = torch.zeros(B, **i32)      # the lengths that all layers but the last commit to
        self.granted = torch.ones(1, **i32)    # whether the last reservation was served
        self._ws = _KeptWorkspace(self.kv_len.device)      # not `device`: "cuda" is another one later

    def _pools(self, layer):
        return self.k_pages[layer], self.v_pages[layer], self.k_scale[layer], self.v_scale[layer]

    def reserve(self, new_len, slot_map=None, new_start=None):
        """Pages for new_len [B] more tokens; their slots into slot_map.  With
        too few free pages nobody gets any: `status` says so, slot_map is -1
        throughout, so that append() writes nothing, and grow() counts nothing."""
        return page_map(self.kv_len, new_len, self.block_table, self.page_count, self.free_pages, self.free_count,
                        self.page_size, slot_map=slot_map, new_start=new_start, status=self.status, granted=self.granted)

    def append(self, layer, k, v, slot_map):
        """One layer's keys and values [T, Hkv, dh] to the reserved slots;
        grow() counts them once every layer has them."""
        kv8_append(k, v, slot_map, *self._pools(layer), status=self.status)

    def grow(self, new_len):
        """new_len [B] (or one number) tokens have been appended; counts nothing
        where the last reservation was refused, since append() wrote none."""
        if torch.is_tensor(new_len):
            self.kv_len.addcmul_(self.granted, new_len.to(torch.int32))
        else:
            torch.add(self.kv_len, self.granted, alpha=new_len, out=self.kv_len)

    def attend(self, layer, q, k_tree, v_tree, mask, scale=None, out=None, lse=None, workspace=None):
        return tree_attn_kv8(q, *self._pools(layer), self.block_table, self.kv_len, k_tree, v_tree, mask, scale=scale,
                             out=out, lse=lse, workspace=workspace or self._ws, status=self.status)

    def commit(self, k_trees, v_trees, accept_len, path_nodes, slot_mapping=None, root=False):
        """The accepted path of every layer (lists of k_tree, v_tree).  With
        `root` the root's rows and the path's are stored, and kv_len grows by
        accept_len + 1; without it by accept_len, and the caller has appended
        the root's rows and grown kv_len by one between the attention and this
        call."""
        last = len(self.k_pages) - 1
        if len(k_trees) != last + 1 or len(v_trees) != last + 1:
            raise EagleError("commit takes the tree K/V of every layer")
        for layer, (k, v) in enumerate(zip(k_trees, v_trees)):
            lens = self.kv_len
            if layer < last:
                lens = self._len
                lens.copy_(self.kv_len)
            slot_mapping = kv8_commit(k, v, accept_len, path_nodes, *self._pools(layer), lens, self.block_table,
                                      slot_mapping=slot_mapping, status=self.status, root=root)
        return slot_mapping

    def trim(self):
        """Back to the free list: the pages past each request's length."""
        self.release(self.kv_len)

    def release(self, keep_len):
        """Pages past keep_len [B] back to the free list (0 ends a request,
        negative leaves it alone).  kv_len is the caller's to reset."""
        page_release(keep_len, self.block_table, self.page_count, self.free_pages, self.free_count, self.page_size,
                     status=self.status)
