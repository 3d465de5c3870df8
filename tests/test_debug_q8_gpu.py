"""The 8-bit cache's attention through the index-checking build: every page that a kernel looks
up lies in the table and the cache, every tree row and partial in its tensor, or the call's
status says LS_ERR_INDEX. That build's waits probe without suspending, so that a wait limit of
one nanosecond runs out in the tensor-core kernel: it must report LS_ERR_TIMEOUT and leave
nothing behind. Nothing here faults or hangs the GPU: the page lookups are bounded in both
builds, and a wait that runs out ends its CTA after its copies and products in flight."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from tests.q8_harness import Case, compare
from tree_verification_attention_longspec_b200 import binding, build

pytestmark = pytest.mark.gpu

LS_ERR_TIMEOUT, LS_ERR_INDEX = 6, 8


@pytest.fixture(scope="module")
def dlib():
    build.build(debug=True)
    return binding.load_debug_library()


class _Call:
    def __init__(self, lib, case, *, host=True, cross=False, bound=None, **opts):
        self.lib, self.case, self.cross = lib, case, cross
        self.cache, self.q, self.kt, self.vt, self.par, self.cu = case.device()
        self.opts = opts
        self.dims, self._keep = binding.make_dims(case.B, case.Hq, case.Hkv, case.d, case.T,
                                                  max_prefix_len=bound or max(case.lens), cu_seqlens_host=case.cu if host else None)
        self.stream = torch.cuda.current_stream().cuda_stream
        ref = ctypes.byref(self.dims)
        if cross:
            self.bytes = lib.ls_cross_attn_q8_workspace_size(ref)
        else:
            self.bytes = lib.ls_verify_attn_q8_workspace_size(ref, ctypes.byref(case.opts(**opts)))
        assert self.bytes > 0

    def workspace(self):
        return torch.full((self.bytes,), 255, dtype=torch.uint8, device="cuda")

    def __call__(self, ws, wait_ns=0):
        r, q = ctypes.byref, self.q
        out, lse = torch.full_like(q, float("nan")), torch.full((q.shape[0], self.case.Hq), float("nan"), device="cuda")
        if self.cross:
            rc = self.lib.ls_cross_attn_q8(q.data_ptr(), self.cache._ref, self.cu.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                           r(self.dims), ws.data_ptr(), self.bytes, self.stream)
        else:
            tree = self.case.opts(wait_ns=wait_ns, **self.opts)
            rc = self.lib.ls_verify_attn_q8(q.data_ptr(), self.cache._ref, self.kt.data_ptr(), self.vt.data_ptr(),
                                            self.par.data_ptr(), self.cu.data_ptr(), r(tree), out.data_ptr(), lse.data_ptr(),
                                            r(self.dims), ws.data_ptr(), self.bytes, self.stream)
        assert rc == 0
        return out, lse, self.lib.ls_verify_attn_check(r(self.dims), ws.data_ptr(), self.stream)


SHAPES = [
    # lens, heads, kv, d, nodes, page, block
    ((1,), 1, 1, 128, 1, 16, 16),
    ((0, 15, 16, 17), 8, 2, 64, 2, 16, 16),
    ((1000, 3, 0, 257), 16, 2, 128, 1, 32, 16),
    ((511, 512, 513), 8, 8, 64, 16, 128, 64),
    ((300, 1025), 4, 1, 128, 16, 64, 32),
    ((127, 900), 16, 4, 64, 33, 32, 32),
    ((640, 100), 8, 2, 128, 32, 384, 64),
    ((260, 5), 4, 1, 64, 128, 16, 16),
    ((40, 3000), 64, 1, 64, 5, 64, 16),
]


@pytest.mark.parametrize("lens,heads,kv,d,nodes,page,block", SHAPES)
@pytest.mark.parametrize("host", [True, False])
@pytest.mark.parametrize("cross", [True, False])
def test_no_index_violation(dlib, lens, heads, kv, d, nodes, page, block, host, cross):
    case = Case(lens, heads, kv, d, nodes, page, block, seed=nodes)
    call = _Call(dlib, case, host=host, cross=cross)
    out, lse, status = call(call.workspace())
    assert status == 0
    compare(out, lse, case.reference(with_tree=not cross))


@pytest.mark.parametrize("heads,kv,d,sizes,window,theta", [(8, 2, 64, (5, 32, 0, 17), 0, 0.0), (8, 2, 128, (1, 1, 1, 1), 60, 0.0),
                                                          (14, 2, 128, (128, 1, 60, 3), 300, 0.0), (8, 2, 64, (7, 0, 20, 2), 0, 1e4)])
def test_ragged_trees_windows_and_rope(dlib, heads, kv, d, sizes, window, theta):
    case = Case((300, 0, 777, 130), heads, kv, d, max(sizes), 32, 32, sizes=sizes, seed=3)
    call = _Call(dlib, case, window=window, theta=theta)
    out, lse, status = call(call.workspace())
    assert status == 0
    if not theta:
        compare(out, lse, case.reference(window=window))


@pytest.mark.parametrize("nodes", [1, 16, 64])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_planted_pages_outside_the_cache_are_reported(dlib, nodes, entry):
    case = Case((500,), 8, 2, 128, nodes, 32, 16)
    right = case.table[0, 3]
    case.table[0, 3] = entry
    call = _Call(dlib, case)
    assert call(call.workspace())[2] == LS_ERR_INDEX
    case.table[0, 3] = right
    call = _Call(dlib, case)
    assert call(call.workspace())[2] == 0


@pytest.mark.parametrize("lens,heads,kv,d,nodes,page,theta", [
    ((9000, 20000), 28, 4, 128, 64, 64, 0.0),   # two query tiles a unit
    ((30000,), 4, 1, 64, 16, 16, 0.0),          # 64 rows: both tiles on them, blocks by turns
    ((5000, 300), 16, 2, 128, 40, 256, 1e4),    # behind the tree kernel's rotation
])
def test_expired_waits_are_reported_and_leave_nothing_behind(dlib, lens, heads, kv, d, nodes, page, theta):
    case = Case(lens, heads, kv, d, nodes, page, 16, seed=d)
    call = _Call(dlib, case, theta=theta)
    ws = call.workspace()
    for _ in range(3):
        assert call(ws, wait_ns=1)[2] == LS_ERR_TIMEOUT
    first, again = call(ws), call(call.workspace())
    assert first[2] == again[2] == 0
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert np.isfinite(first[1].cpu().numpy()).all()
