"""The 8-bit paged cache, attention over it, and sampling, on torch tensors.

Argument checks and marshalling only, like ``binding``: every step of the computation runs
in the CUDA kernels of ``libls_verify_attn.so``, declared in ``include/ls_verify_attn.h``,
and there is no fallback. Every call runs on the current stream of the tensors' device,
whichever device is current, and returns without waiting for it.

One verification step of a served model, with a cache that stays on the device::

    cache = KVCacheQ8.empty(num_pages, 64, H_kv, d, page_table)
    cu = cache.append(k_prompt, v_prompt, cu, cu_new, max_new)            # the prompts
    attend = VerifyAttnQ8(B, H_q, H_kv, d, T, max_prefix_len=longest)
    out, lse = attend(q, cache, k_tree, v_tree, parent, cu)               # each layer
    tokens, n, path, after = tree_accept_sample(logits, u, draft, parent, T, temperature=t)
    cu = cache.commit(k_tree, v_tree, cu, n, path)                        # what was accepted
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding
from .binding import LS_OK, LSError, TreeOpts, load_library, make_dims

__all__ = ["KVCacheQ8", "VerifyAttnQ8", "CrossAttnQ8", "sample", "tree_accept_sample"]

SCALE_BLOCKS = (16, 32, 64, 128)


def _tensor(t, name: str, dtypes, device=None):
    """A dense CUDA tensor of one of `dtypes` on `device`, or an error that names it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in (dtypes if isinstance(dtypes, tuple) else (dtypes,)):
        raise TypeError(f"{name} must be {dtypes}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _shape(t, name: str, *shape):
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _ints(t, name: str, device, *shape):
    _tensor(t, name, torch.int32, device)
    _shape(t, name, *shape)
    return t.data_ptr()


def _call(device, what: str, fn, *args):
    """fn(*args, stream) on `device` and its current stream; raises what it returns."""
    with torch.cuda.device(device):
        rc = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if rc != LS_OK:
        raise LSError(rc, what)


class KVCacheQ8:
    """A paged K/V cache in 8 bits (e4m3) with one scale per block of tokens and kv head.

    k_pages, v_pages: float8_e4m3fn (or uint8) [num_pages, page_size, H_kv, d]; k_scale,
    v_scale: fp32 [num_pages, page_size // scale_block, H_kv]; page_table: int32 [B,
    max_pages_per_seq]. The object keeps the tensors, which it reads and writes in place;
    their values at the time of a call's kernels count.
    """

    def __init__(self, k_pages, v_pages, k_scale, v_scale, page_table):
        codes = (torch.float8_e4m3fn, torch.uint8)
        _tensor(k_pages, "k_pages", codes)
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [num_pages, page_size, H_kv, d]")
        self.device = k_pages.device
        self.num_pages, self.page_size, self.num_kv_heads, self.head_dim = map(int, k_pages.shape)
        _tensor(v_pages, "v_pages", codes, self.device)
        _shape(v_pages, "v_pages", *k_pages.shape)
        _tensor(k_scale, "k_scale", torch.float32, self.device)
        if k_scale.dim() != 3 or k_scale.shape[1] < 1 or self.page_size % k_scale.shape[1]:
            raise ValueError("k_scale must be [num_pages, page_size // scale_block, H_kv]")
        _shape(k_scale, "k_scale", self.num_pages, k_scale.shape[1], self.num_kv_heads)
        _tensor(v_scale, "v_scale", torch.float32, self.device)
        _shape(v_scale, "v_scale", *k_scale.shape)
        _tensor(page_table, "page_table", torch.int32, self.device)
        if page_table.dim() != 2:
            raise ValueError("page_table must be [B, max_pages_per_seq]")
        self.scale_block = self.page_size // int(k_scale.shape[1])
        self.batch, self.max_pages_per_seq = map(int, page_table.shape)
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.page_table = page_table
        self._struct = binding.KvQ8(self.page_size, self.scale_block, self.max_pages_per_seq, self.num_pages,
                                    page_table.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                    k_scale.data_ptr(), v_scale.data_ptr())
        self._ref = ctypes.byref(self._struct)
        # the writers' dims: batch, kv heads and head dimension (the tree size is the call's)
        self._dims = {}

    @classmethod
    def empty(cls, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, page_table, *,
              scale_block: Optional[int] = None):
        """A cache without tokens on page_table's device; scale_block: the page size, at most 64."""
        if scale_block is None:
            scale_block = min(page_size, 64)
        if scale_block not in SCALE_BLOCKS or page_size % scale_block:
            raise ValueError("scale_block must be 16, 32, 64 or 128 and divide page_size")
        dev = page_table.device
        codes = [torch.zeros(num_pages, page_size, num_kv_heads, head_dim, dtype=torch.uint8, device=dev)
                 .view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.ones(num_pages, page_size // scale_block, num_kv_heads, device=dev) for _ in range(2)]
        return cls(*codes, *scales, page_table)

    def _write_dims(self, tree_size: int):
        if tree_size not in self._dims:
            self._dims[tree_size] = make_dims(self.batch, self.num_kv_heads, self.num_kv_heads, self.head_dim,
                                              tree_size)[0]
        return ctypes.byref(self._dims[tree_size])

    def _rows(self, k, v, names):
        _tensor(k, names[0], torch.bfloat16, self.device)
        _tensor(v, names[1], torch.bfloat16, self.device)
        if k.dim() != 3 or tuple(k.shape[1:]) != (self.num_kv_heads, self.head_dim):
            raise ValueError(f"{names[0]} must be [rows, {self.num_kv_heads}, {self.head_dim}], got {tuple(k.shape)}")
        _shape(v, names[1], *k.shape)
        return k.data_ptr(), v.data_ptr()

    def append(self, k_new, v_new, cu_seqlens, cu_new, max_new: int, *, cu_seqlens_out=None):
        """Rows cu_new[b]:cu_new[b+1] of k_new / v_new (bf16 [rows, H_kv, d]) become the next
        tokens of sequence b, at most max_new of them. Returns the new cu_seqlens
        (cu_seqlens_out, or a new tensor; never cu_seqlens itself)."""
        k, v = self._rows(k_new, v_new, ("k_new", "v_new"))
        cu = _ints(cu_seqlens, "cu_seqlens", self.device, self.batch + 1)
        new = _ints(cu_new, "cu_new", self.device, self.batch + 1)
        if cu_seqlens_out is None:
            cu_seqlens_out = torch.empty_like(cu_seqlens)
        out = _ints(cu_seqlens_out, "cu_seqlens_out", self.device, self.batch + 1)
        _call(self.device, "ls_kv_append_q8", load_library().ls_kv_append_q8, k, v, new, int(k_new.shape[0]),
              int(max_new), cu, out, self._ref, self._write_dims(1))
        return cu_seqlens_out

    def commit(self, k_tree, v_tree, cu_seqlens, accept_len, accept_path, *, cu_tree=None, cu_seqlens_out=None):
        """The accepted path of every tree becomes the next tokens of its sequence: rows
        accept_path[b, :accept_len[b] + 1] of the tree's k_tree / v_tree. accept_path is [B, T]
        as the acceptance calls return it; trees are packed by cu_tree, or T nodes each.
        Returns the new cu_seqlens."""
        k, v = self._rows(k_tree, v_tree, ("k_tree", "v_tree"))
        cu = _ints(cu_seqlens, "cu_seqlens", self.device, self.batch + 1)
        length = _ints(accept_len, "accept_len", self.device, self.batch)
        _tensor(accept_path, "accept_path", torch.int32, self.device)
        if accept_path.dim() != 2 or accept_path.shape[0] != self.batch:
            raise ValueError(f"accept_path must be [{self.batch}, T]")
        size, nodes = int(accept_path.shape[1]), int(k_tree.shape[0])
        trees = None
        if cu_tree is not None:
            trees = _ints(cu_tree, "cu_tree", self.device, self.batch + 1)
        elif nodes != self.batch * size:
            raise ValueError(f"k_tree must have {self.batch} * {size} rows, got {nodes}")
        if cu_seqlens_out is None:
            cu_seqlens_out = torch.empty_like(cu_seqlens)
        out = _ints(cu_seqlens_out, "cu_seqlens_out", self.device, self.batch + 1)
        _call(self.device, "ls_kv_commit_q8", load_library().ls_kv_commit_q8, k, v, trees, nodes, length,
              accept_path.data_ptr(), cu, out, self._ref, self._write_dims(size))
        return cu_seqlens_out


class _AttnQ8:
    """What the two attention calls share: fixed dims and one workspace, any inputs of those
    shapes. Calls of one object, captured ones included, must not overlap on the GPU."""

    with_tree = True

    def __init__(self, batch, num_q_heads, num_kv_heads, head_dim, tree_size, *, cu_seqlens_host=None,
                 max_prefix_len=0, softmax_scale=0.0, tree: Optional[TreeOpts] = None, device=None):
        self.dims, self._keep = make_dims(batch, num_q_heads, num_kv_heads, head_dim, tree_size, max_prefix_len,
                                          cu_seqlens_host, softmax_scale)
        if cu_seqlens_host is not None and len(self._keep) != batch + 1:
            raise ValueError("cu_seqlens_host must have batch + 1 entries")
        self.tree = tree
        self._tree_ref = None if tree is None else ctypes.byref(tree)
        self._dims_ref = ctypes.byref(self.dims)
        dev = torch.device(device if device is not None else "cuda")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        with torch.cuda.device(dev):
            self.ws_bytes = self._size()
        if self.ws_bytes == 0:
            raise LSError(1, f"{self._name}_workspace_size returned 0 (invalid or unsupported dims)")
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)

    def _check(self, q, cache, cu_seqlens, out, lse):
        d = self.dims
        if not isinstance(cache, KVCacheQ8):
            raise TypeError("cache must be a KVCacheQ8")
        if (cache.batch, cache.num_kv_heads, cache.head_dim) != (d.batch, d.num_kv_heads, d.head_dim):
            raise ValueError("the cache's batch, kv heads or head dimension are not the call's")
        if cache.device != self.device:
            raise ValueError(f"the cache is on {cache.device}, the call on {self.device}")
        self._rows = d.batch * d.tree_size
        if self.tree is not None and self.tree.cu_tree:
            self._rows = self.tree.total_nodes
        _tensor(q, "q", torch.bfloat16, self.device)
        _shape(q, "q", self._rows, d.num_q_heads, d.head_dim)
        if out is None:
            out = torch.empty_like(q)
        else:
            _tensor(out, "out", torch.bfloat16, self.device)
            _shape(out, "out", *q.shape)
        if lse is None:
            lse = torch.empty(self._rows, d.num_q_heads, dtype=torch.float32, device=self.device)
        else:
            _tensor(lse, "lse", torch.float32, self.device)
            _shape(lse, "lse", self._rows, d.num_q_heads)
        return _ints(cu_seqlens, "cu_seqlens", self.device, d.batch + 1), out, lse

    def check(self) -> int:
        """Waits for the current stream; the device status of the last call (binding.STATUS_NAMES)."""
        with torch.cuda.device(self.device):
            return binding.check(self.dims, self.workspace.data_ptr(),
                                 torch.cuda.current_stream(self.device).cuda_stream)


class VerifyAttnQ8(_AttnQ8):
    """Tree-verification attention over a KVCacheQ8 (``ls_verify_attn_q8``); tree_size = 1 is a
    decoding step whose own key and value are not in the cache yet. tree: a TreeOpts with
    per-sequence trees (cu_tree: its device address, kept alive by the caller), a window or
    RoPE. cu_seqlens_host balances the work over the actual lengths; with max_prefix_len
    alone, an upper bound, one object serves a cache that grows."""

    _name = "ls_verify_attn_q8"

    def _size(self):
        return int(load_library().ls_verify_attn_q8_workspace_size(self._dims_ref, self._tree_ref))

    def __call__(self, q, cache, k_tree, v_tree, parent, cu_seqlens, out=None, lse=None):
        cu, out, lse = self._check(q, cache, cu_seqlens, out, lse)
        d = self.dims
        for t, name in ((k_tree, "k_tree"), (v_tree, "v_tree")):
            _tensor(t, name, torch.bfloat16, self.device)
            _shape(t, name, self._rows, d.num_kv_heads, d.head_dim)
        par = _ints(parent, "tree_parent", self.device, self._rows)
        _call(self.device, self._name, load_library().ls_verify_attn_q8, q.data_ptr(), cache._ref, k_tree.data_ptr(),
              v_tree.data_ptr(), par, cu, self._tree_ref, out.data_ptr(), lse.data_ptr(), self._dims_ref,
              self.workspace.data_ptr(), self.ws_bytes)
        return out, lse


class CrossAttnQ8(_AttnQ8):
    """Prefix-only attention over a KVCacheQ8 (``ls_cross_attn_q8``): tree_size queries per
    sequence over all its cached tokens, as a decoding step whose token was appended first."""

    _name = "ls_cross_attn_q8"

    def __init__(self, *args, **kwargs):
        if kwargs.get("tree") is not None:
            raise ValueError("prefix-only attention takes no tree options")
        super().__init__(*args, **kwargs)

    def _size(self):
        return int(load_library().ls_cross_attn_q8_workspace_size(self._dims_ref))

    def __call__(self, q, cache, cu_seqlens, out=None, lse=None):
        cu, out, lse = self._check(q, cache, cu_seqlens, out, lse)
        _call(self.device, self._name, load_library().ls_cross_attn_q8, q.data_ptr(), cache._ref, cu, out.data_ptr(),
              lse.data_ptr(), self._dims_ref, self.workspace.data_ptr(), self.ws_bytes)
        return out, lse


def _sampling(logits, uniform, temperature, top_k, top_p, min_p, dense: bool):
    """(rows, vocab, row stride, dtype, options and what they keep alive) of checked logits."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch tensor")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    if not logits.is_cuda:
        raise ValueError("logits must be on a CUDA device")
    if logits.dim() != 2 or logits.shape[1] < 1:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = map(int, logits.shape)
    stride = int(logits.stride(0)) if rows > 1 else vocab
    if vocab > 1 and logits.stride(1) != 1 or stride < vocab or dense and not logits.is_contiguous():
        raise ValueError("logits must be contiguous" if dense else "logits must have contiguous, disjoint rows")
    dev = logits.device
    _tensor(uniform, "uniform", torch.float32, dev)
    _shape(uniform, "uniform", rows)
    keep, ptrs = [], []
    for value, name, dtype in ((temperature, "temperature", torch.float32), (top_k, "top_k", torch.int32),
                               (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32)):
        if value is None:
            ptrs.append(None)
            continue
        if isinstance(value, (int, float)):  # one value for every row
            value = torch.full((rows,), value, dtype=dtype, device=dev)
        _tensor(value, name, dtype, dev)
        _shape(value, name, rows)
        keep.append(value)
        ptrs.append(value.data_ptr())
    kind = binding.LS_DTYPE_F32 if logits.dtype == torch.float32 else binding.LS_DTYPE_BF16
    return rows, vocab, stride, kind, binding.SampleOpts(*ptrs), keep


def sample(logits, uniform, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None):
    """One token for each row of logits (bf16 or fp32 [rows, vocab], rows may be strided) from
    uniform fp32 [rows] in [0, 1). temperature, top_k, top_p, min_p: a number for all rows, a
    tensor with one per row (fp32; top_k int32), or None (1, off, off, off); temperature 0 is
    greedy. The order of the filters and the draw are those of ``ls_sample``. Returns int32
    [rows]."""
    rows, vocab, stride, kind, opts, keep = _sampling(logits, uniform, temperature, top_k, top_p, min_p, False)
    dev = logits.device
    if out is None:
        out = torch.empty(rows, dtype=torch.int32, device=dev)
    _ints(out, "out", dev, rows)
    _call(dev, "ls_sample", load_library().ls_sample, logits.data_ptr(), stride, uniform.data_ptr(),
          ctypes.byref(opts), out.data_ptr(), rows, vocab, kind)
    return out


def tree_accept_sample(logits, uniform, tree_tokens, tree_parent, tree_size: int, *, cu_tree=None, temperature=None,
                       top_k=None, top_p=None, min_p=None):
    """Draws the target's token at every tree node and walks each tree from its root to the
    child whose draft token was drawn (``ls_tree_accept_sample``). logits [N, vocab], one row
    per node; trees of tree_size nodes each, or packed by cu_tree int32 [B+1] with at most
    tree_size nodes. Returns (node_token [N], accept_len [B], accept_path [B, tree_size],
    next_token [B]), int32."""
    rows, vocab, _, kind, opts, keep = _sampling(logits, uniform, temperature, top_k, top_p, min_p, True)
    dev = logits.device
    if tree_size < 1:
        raise ValueError("tree_size must be positive")
    trees = None
    if cu_tree is not None:
        _tensor(cu_tree, "cu_tree", torch.int32, dev)
        if cu_tree.dim() != 1 or cu_tree.shape[0] < 2:
            raise ValueError("cu_tree must be [B + 1]")
        batch, trees = int(cu_tree.shape[0]) - 1, cu_tree.data_ptr()
    else:
        batch = rows // tree_size
        if batch < 1 or batch * tree_size != rows:
            raise ValueError(f"{rows} rows of logits are not whole trees of {tree_size} nodes")
    tok = _ints(tree_tokens, "tree_tokens", dev, rows)
    par = _ints(tree_parent, "tree_parent", dev, rows)
    node_token = torch.empty(rows, dtype=torch.int32, device=dev)
    accept_path = torch.empty(batch, tree_size, dtype=torch.int32, device=dev)
    accept_len, next_token = torch.empty(2, batch, dtype=torch.int32, device=dev)
    dims = binding.AcceptDims(batch, tree_size, vocab, kind)
    _call(dev, "ls_tree_accept_sample", load_library().ls_tree_accept_sample, logits.data_ptr(), uniform.data_ptr(),
          ctypes.byref(opts), tok, par, trees, rows, node_token.data_ptr(), accept_len.data_ptr(),
          accept_path.data_ptr(), next_token.data_ptr(), ctypes.byref(dims))
    return node_token, accept_len, accept_path, next_token
