"""A sliding window with a bound on the lengths instead of the lengths: any sequence up to the
bound is served, though a shorter one may attend one block of keys more than the bound's."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.q8_harness import Case, compare
from tree_verification_attention_longspec_b200 import binding

pytestmark = pytest.mark.gpu


# nodes: rows a kv head up to 8, 32 and above; bound 768 attends 256 keys, 727 of them 343
@pytest.mark.parametrize("nodes", [1, 8, 32])
@pytest.mark.parametrize("window,bound,lens", [(248, 768, (6, 727)), (57, 320, (290, 1)), (600, 1536, (1391, 797, 0)),
                                               (130, 256, (255, 256, 129))])
def test_8_bit_cache(nodes, window, bound, lens):
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case(lens, 8, 2, 64, nodes, 16, 16, seed=window)
    table = np.full((len(lens), bound // 16), -1, dtype=np.int32)
    table[:, :case.table.shape[1]] = case.table[:, :table.shape[1]]
    case.table = table
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(case.B, 8, 2, 64, nodes, max_prefix_len=bound, tree=case.opts(window=window))
    call.workspace.fill_(0xFF)
    out, lse = call(q, cache, kt, vt, par, cu)
    assert call.check() == 0
    compare(out, lse, case.reference(window=window))


def test_a_cache_that_grows_under_one_object():
    """Every length up to the bound, as decoding steps reach them."""
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    bound, window = 320, 57
    call = None
    for n in range(bound - 140, bound + 1, 3):
        case = Case((n,), 4, 1, 64, 1, 16, 16, seed=n)
        table = np.full((1, bound // 16), -1, dtype=np.int32)
        table[:, :min(case.table.shape[1], bound // 16)] = case.table[:, :bound // 16]
        case.table = table
        cache, q, kt, vt, par, cu = case.device()
        if call is None:
            call = VerifyAttnQ8(1, 4, 1, 64, 1, max_prefix_len=bound, tree=case.opts(window=window))
        out, lse = call(q, cache, kt, vt, par, cu)
        assert call.check() == 0, n
        compare(out, lse, case.reference(window=window))


@pytest.mark.parametrize("nodes", [1, 40])
def test_packed_cache(nodes):
    """The same of ls_verify_attn_ex, whose plan it is: as with the lengths given."""
    window, bound, lens, H, d = 248, 768, (6, 727), 4, 64
    g = torch.Generator().manual_seed(nodes)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    B, total = len(lens), sum(lens)
    q, kt, vt, kc, vc = rand(B * nodes, H, d), rand(B * nodes, 1, d), rand(B * nodes, 1, d), rand(B * bound, 1, d), rand(B * bound, 1, d)
    par = torch.arange(-1, nodes - 1, dtype=torch.int32).repeat(B).cuda()
    cu_host = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cu = torch.from_numpy(cu_host).cuda()
    assert total <= B * bound
    tree = binding.TreeOpts(window=window)
    got = []
    for kw in (dict(cu_seqlens_host=cu_host), dict(max_prefix_len=bound)):
        dims, keep = binding.make_dims(B, H, 1, d, nodes, **kw)
        wsb = binding.ex_workspace_size(dims, tree)
        ws = torch.full((wsb,), 255, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(B * nodes, H, device="cuda")
        stream = torch.cuda.current_stream().cuda_stream
        assert binding.call_ex_raw(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), None, kt.data_ptr(), vt.data_ptr(),
                                   par.data_ptr(), cu.data_ptr(), tree, out.data_ptr(), lse.data_ptr(), dims,
                                   ws.data_ptr(), wsb, stream) == 0
        assert binding.check(dims, ws.data_ptr(), stream) == 0
        got.append((out.float(), lse))
    # the chunks differ, and with them the order of fp32 sums and of bf16 weights
    assert (got[0][0] - got[1][0]).abs().max() <= 1e-2 and (got[0][1] - got[1][1]).abs().max() <= 1e-3
