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
    tokens, n, path, after = tree_accept_sample(logits, u, draft, parent, T, temperature=t)  # t: a tensor
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
CODE_DTYPES = (torch.float8_e4m3fn, torch.uint8)


def _refuse(t, name: str, dtypes, device, shape):
    """Raises the error that says what of `t` does not fit."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(t, name: str, dtype, device, shape=None):
    """The address of a dense CUDA tensor of this dtype, device and shape, or an error that
    names it. (One test on the way that every call takes: small calls are bound by it.)"""
    try:
        if (t.dtype is dtype and t.get_device() == device.index and t.is_contiguous()
                and (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, (dtype,), device, shape)


_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _call(device, what: str, fn, *args):
    """fn(*args, stream) on `device` and its current stream; raises what it returns."""
    index = device.index
    if _current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
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
        for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            if not isinstance(t, torch.Tensor) or t.dtype not in CODE_DTYPES or not t.is_cuda or not t.is_contiguous():
                _refuse(t, name, CODE_DTYPES, None, None)
            if t.dim() != 4:
                raise ValueError(f"{name} must be [num_pages, page_size, H_kv, d]")
        self.device = k_pages.device
        self.num_pages, self.page_size, self.num_kv_heads, self.head_dim = map(int, k_pages.shape)
        if v_pages.device != self.device or v_pages.shape != k_pages.shape:
            _refuse(v_pages, "v_pages", CODE_DTYPES, self.device, k_pages.shape)
        _ptr(k_scale, "k_scale", torch.float32, self.device)
        if k_scale.dim() != 3 or k_scale.shape[1] < 1 or self.page_size % k_scale.shape[1]:
            raise ValueError("k_scale must be [num_pages, page_size // scale_block, H_kv]")
        _ptr(k_scale, "k_scale", torch.float32, self.device, (self.num_pages, k_scale.shape[1], self.num_kv_heads))
        _ptr(v_scale, "v_scale", torch.float32, self.device, k_scale.shape)
        _ptr(page_table, "page_table", torch.int32, self.device)
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
        self._kind = (self.batch, self.num_kv_heads, self.head_dim, self.device.index)
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
        if not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError(f"{names[0]} must be a tensor [rows, {self.num_kv_heads}, {self.head_dim}]")
        shape = (k.shape[0], self.num_kv_heads, self.head_dim)
        return (_ptr(k, names[0], torch.bfloat16, self.device, shape),
                _ptr(v, names[1], torch.bfloat16, self.device, shape))

    def append(self, k_new, v_new, cu_seqlens, cu_new, max_new: int, *, cu_seqlens_out=None):
        """Rows cu_new[b]:cu_new[b+1] of k_new / v_new (bf16 [rows, H_kv, d]) become the next
        tokens of sequence b, at most max_new of them. Returns the new cu_seqlens
        (cu_seqlens_out, or a new tensor; never cu_seqlens itself)."""
        k, v = self._rows(k_new, v_new, ("k_new", "v_new"))
        ends = (self.batch + 1,)
        cu = _ptr(cu_seqlens, "cu_seqlens", torch.int32, self.device, ends)
        new = _ptr(cu_new, "cu_new", torch.int32, self.device, ends)
        if cu_seqlens_out is None:
            cu_seqlens_out = torch.empty_like(cu_seqlens)
        out = _ptr(cu_seqlens_out, "cu_seqlens_out", torch.int32, self.device, ends)
        _call(self.device, "ls_kv_append_q8", load_library().ls_kv_append_q8, k, v, new, k_new.shape[0],
              int(max_new), cu, out, self._ref, self._write_dims(1))
        return cu_seqlens_out

    def commit(self, k_tree, v_tree, cu_seqlens, accept_len, accept_path, *, cu_tree=None, cu_seqlens_out=None):
        """The accepted path of every tree becomes the next tokens of its sequence: rows
        accept_path[b, :accept_len[b] + 1] of the tree's k_tree / v_tree. accept_path is [B, T]
        as the acceptance calls return it; trees are packed by cu_tree, or T nodes each.
        Returns the new cu_seqlens."""
        k, v = self._rows(k_tree, v_tree, ("k_tree", "v_tree"))
        ends = (self.batch + 1,)
        cu = _ptr(cu_seqlens, "cu_seqlens", torch.int32, self.device, ends)
        length = _ptr(accept_len, "accept_len", torch.int32, self.device, (self.batch,))
        path = _ptr(accept_path, "accept_path", torch.int32, self.device)
        if accept_path.dim() != 2 or accept_path.shape[0] != self.batch:
            raise ValueError(f"accept_path must be [{self.batch}, T]")
        size, nodes = accept_path.shape[1], k_tree.shape[0]
        trees = None
        if cu_tree is not None:
            trees = _ptr(cu_tree, "cu_tree", torch.int32, self.device, ends)
        elif nodes != self.batch * size:
            raise ValueError(f"k_tree must have {self.batch} * {size} rows, got {nodes}")
        if cu_seqlens_out is None:
            cu_seqlens_out = torch.empty_like(cu_seqlens)
        out = _ptr(cu_seqlens_out, "cu_seqlens_out", torch.int32, self.device, ends)
        _call(self.device, "ls_kv_commit_q8", load_library().ls_kv_commit_q8, k, v, trees, nodes, length, path, cu, out,
              self._ref, self._write_dims(size))
        return cu_seqlens_out


class _AttnQ8:
    """What the two attention calls share: fixed dims and one workspace, any inputs of those
    shapes. Calls of one object, captured ones included, must not overlap on the GPU, and a
    graph that holds one needs the object for as long as it is replayed."""

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
        self._ws_ptr = self.workspace.data_ptr()
        self._home = _raw_stream(dev.index)  # the stream that the workspace was allocated on
        self._fn = getattr(load_library(), self._name)
        self._rows = batch * tree_size
        self._kind = (batch, num_kv_heads, head_dim, dev.index)
        self._shapes = self._shapes_of(self._rows)

    def _begin(self, q, cache, cu_seqlens, out, lse):
        """(out, lse, the addresses of q, cu_seqlens, out, lse, and the shape of the tree's rows)"""
        if not isinstance(cache, KVCacheQ8):
            raise TypeError("cache must be a KVCacheQ8")
        if cache._kind != self._kind:
            if cache.device != self.device:
                raise ValueError(f"the cache is on {cache.device}, the call on {self.device}")
            raise ValueError("the cache's batch, kv heads or head dimension are not the call's")
        dev, d = self.device, self.dims
        if _raw_stream(dev.index) != self._home and not torch.cuda.is_current_stream_capturing():
            # freed with this object, the memory waits for the call's stream before it is used again
            self.workspace.record_stream(torch.cuda.current_stream(dev))
        rows = self.tree.total_nodes if self.tree is not None and self.tree.cu_tree else self._rows
        if rows != self._shapes[3][0]:
            self._shapes = self._shapes_of(rows)
        q_shape, lse_shape, cu_shape, kv_shape = self._shapes
        qp = _ptr(q, "q", torch.bfloat16, dev, q_shape)
        if out is None:
            out = torch.empty_like(q)
            op = out.data_ptr()
        else:
            op = _ptr(out, "out", torch.bfloat16, dev, q_shape)
        if lse is None:
            lse = torch.empty_like(self._lse_like)
            lp = lse.data_ptr()
        else:
            lp = _ptr(lse, "lse", torch.float32, dev, lse_shape)
        return out, lse, qp, _ptr(cu_seqlens, "cu_seqlens", torch.int32, dev, cu_shape), op, lp, kv_shape

    def _shapes_of(self, rows):
        d = self.dims
        # one element seen as many: what empty_like (half the cost of empty) takes its shape from
        self._lse_like = torch.empty((), dtype=torch.float32, device=self.device).expand(rows, d.num_q_heads)
        return ((rows, d.num_q_heads, d.head_dim), (rows, d.num_q_heads), (d.batch + 1,),
                (rows, d.num_kv_heads, d.head_dim))

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
        out, lse, qp, cu, op, lp, shape = self._begin(q, cache, cu_seqlens, out, lse)
        dev = self.device
        _call(dev, self._name, self._fn, qp, cache._ref, _ptr(k_tree, "k_tree", torch.bfloat16, dev, shape),
              _ptr(v_tree, "v_tree", torch.bfloat16, dev, shape), _ptr(parent, "tree_parent", torch.int32, dev, shape[:1]),
              cu, self._tree_ref, op, lp, self._dims_ref, self._ws_ptr, self.ws_bytes)
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
        out, lse, qp, cu, op, lp, _ = self._begin(q, cache, cu_seqlens, out, lse)
        _call(self.device, self._name, self._fn, qp, cache._ref, cu, op, lp, self._dims_ref, self._ws_ptr, self.ws_bytes)
        return out, lse


_KINDS = {torch.float32: binding.LS_DTYPE_F32, torch.bfloat16: binding.LS_DTYPE_BF16}


def _sampling(logits, uniform, temperature, top_k, top_p, min_p, dense: bool):
    """(rows, vocab, row stride, uniform's address, dtype, options and what they keep alive)"""
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _KINDS or not logits.is_cuda:
        _refuse(logits, "logits", tuple(_KINDS), None, None)
    shape = logits.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError("logits must be [rows, vocab]")
    rows, vocab = shape
    stride = vocab
    if not logits.is_contiguous():
        stride, inner = logits.stride()
        if rows < 2:
            stride = vocab
        if dense or vocab > 1 and inner != 1 or stride < vocab:
            raise ValueError("logits must be contiguous" if dense else "logits must have contiguous, disjoint rows")
    dev, per_row = logits.device, (rows,)
    u = _ptr(uniform, "uniform", torch.float32, dev, per_row)
    keep, ptrs = [], []
    for value, name, dtype in ((temperature, "temperature", torch.float32), (top_k, "top_k", torch.int32),
                               (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32)):
        if value is None:
            ptrs.append(None)
            continue
        if isinstance(value, (int, float)):  # one value for every row
            value = torch.full(per_row, value, dtype=dtype, device=dev)
            keep.append(value)
        ptrs.append(_ptr(value, name, dtype, dev, per_row))
    return rows, vocab, stride, u, _KINDS[logits.dtype], binding.SampleOpts(*ptrs), keep


def sample(logits, uniform, *, temperature=None, top_k=None, top_p=None, min_p=None, out=None):
    """One token for each row of logits (bf16 or fp32 [rows, vocab], rows may be strided) from
    uniform fp32 [rows] in [0, 1). temperature, top_k, top_p, min_p: a tensor with one value per
    row (fp32; top_k int32), a number for all rows (a tensor is filled with it each call, which
    costs a launch: keep a tensor where calls are small), or None (1, off, off, off); temperature
    0 is greedy. The order of the filters and the draw are those of ``ls_sample``. Returns int32
    [rows]."""
    rows, vocab, stride, u, kind, opts, keep = _sampling(logits, uniform, temperature, top_k, top_p, min_p, False)
    dev = logits.device
    if out is None:
        out = torch.empty_like(uniform, dtype=torch.int32)
    _call(dev, "ls_sample", load_library().ls_sample, logits.data_ptr(), stride, u, ctypes.byref(opts),
          _ptr(out, "out", torch.int32, dev, (rows,)), rows, vocab, kind)
    return out


def tree_accept_sample(logits, uniform, tree_tokens, tree_parent, tree_size: int, *, cu_tree=None, temperature=None,
                       top_k=None, top_p=None, min_p=None):
    """Draws the target's token at every tree node and walks each tree from its root to the
    child whose draft token was drawn (``ls_tree_accept_sample``). logits [N, vocab], one row
    per node; trees of tree_size nodes each, or packed by cu_tree int32 [B+1] with at most
    tree_size nodes. Returns (node_token [N], accept_len [B], accept_path [B, tree_size],
    next_token [B]), int32."""
    rows, vocab, _, u, kind, opts, keep = _sampling(logits, uniform, temperature, top_k, top_p, min_p, True)
    dev = logits.device
    if tree_size < 1:
        raise ValueError("tree_size must be positive")
    trees = None
    if cu_tree is not None:
        trees = _ptr(cu_tree, "cu_tree", torch.int32, dev)
        if cu_tree.dim() != 1 or cu_tree.shape[0] < 2:
            raise ValueError("cu_tree must be [B + 1]")
        batch = cu_tree.shape[0] - 1
    else:
        batch = rows // tree_size
        if batch < 1 or batch * tree_size != rows:
            raise ValueError(f"{rows} rows of logits are not whole trees of {tree_size} nodes")
    tok = _ptr(tree_tokens, "tree_tokens", torch.int32, dev, (rows,))
    par = _ptr(tree_parent, "tree_parent", torch.int32, dev, (rows,))
    node_token = torch.empty_like(tree_tokens)
    accept_path = torch.empty((batch, tree_size), dtype=torch.int32, device=dev)
    accept_len = torch.empty((batch,), dtype=torch.int32, device=dev)
    next_token = torch.empty_like(accept_len)
    dims = binding.AcceptDims(batch, tree_size, vocab, kind)
    _call(dev, "ls_tree_accept_sample", load_library().ls_tree_accept_sample, logits.data_ptr(), u,
          ctypes.byref(opts), tok, par, trees, rows, node_token.data_ptr(), accept_len.data_ptr(),
          accept_path.data_ptr(), next_token.data_ptr(), ctypes.byref(dims))
    return node_token, accept_len, accept_path, next_token
