"""Attention over the 8-bit paged cache against the fp64 oracle: heads, lengths, pages,
scale blocks, trees, windows, RoPE, prefix-only calls, streams and captured graphs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.q8_harness import Case, compare

pytestmark = pytest.mark.gpu


def _verify(case, host=True, **opts):
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    cache, q, kt, vt, par, cu = case.device()
    tree = case.opts(**opts) if opts or case.ragged else None
    call = VerifyAttnQ8(case.B, case.Hq, case.Hkv, case.d, case.T, cu_seqlens_host=case.cu if host else None,
                        max_prefix_len=max(case.lens), tree=tree)
    call.workspace.fill_(0xFF)  # NaN wherever a partial is read before it is written
    out, lse = call(q, cache, kt, vt, par, cu)
    assert call.check() == 0
    return out, lse


# rows a kv head: 1 .. 8, 9 .. 16, up to 128, up to 256, and beyond
SHAPES = [
    # lens, heads, kv, d, nodes, page, block
    ((1,), 1, 1, 128, 1, 16, 16),
    ((129,), 7, 1, 128, 1, 64, 64),
    ((0, 15, 16, 17), 8, 2, 64, 2, 16, 16),
    ((1000, 3, 0, 257), 16, 2, 128, 1, 32, 16),
    ((511, 512, 513), 8, 8, 64, 16, 128, 64),
    ((700, 33), 10, 2, 128, 3, 256, 128),
    ((300, 1025), 4, 1, 128, 16, 64, 32),
    ((127, 900), 16, 4, 64, 33, 32, 32),
    ((640, 100), 8, 2, 128, 32, 384, 64),
    ((2000,), 14, 2, 128, 37, 64, 64),
    ((260, 5), 4, 1, 64, 128, 16, 16),
    ((515,), 64, 1, 128, 5, 128, 128),
    ((40,), 256, 1, 64, 2, 64, 16),
]


@pytest.mark.parametrize("lens,heads,kv,d,nodes,page,block", SHAPES)
@pytest.mark.parametrize("host", [True, False])
def test_tree_attention(lens, heads, kv, d, nodes, page, block, host):
    case = Case(lens, heads, kv, d, nodes, page, block, seed=len(lens) + nodes, scale_spread=0.5)
    compare(*_verify(case, host), case.reference())


@pytest.mark.parametrize("lens,heads,kv,d,nodes,page,block", SHAPES)
@pytest.mark.parametrize("host", [True, False])
def test_prefix_attention(lens, heads, kv, d, nodes, page, block, host):
    from tree_verification_attention_longspec_b200 import CrossAttnQ8
    case = Case(lens, heads, kv, d, nodes, page, block, seed=nodes, scale_spread=0.5)
    cache, q, _, _, _, cu = case.device()
    call = CrossAttnQ8(case.B, case.Hq, case.Hkv, case.d, case.T, cu_seqlens_host=case.cu if host else None,
                       max_prefix_len=max(lens))
    call.workspace.fill_(0xFF)
    out, lse = call(q, cache, cu)
    assert call.check() == 0
    compare(out, lse, case.reference(with_tree=False))


@pytest.mark.parametrize("heads,kv,d,sizes", [(7, 1, 128, (1, 0, 3)), (8, 2, 64, (5, 32, 0, 17)), (14, 2, 128, (128, 1, 60))])
def test_per_sequence_trees(heads, kv, d, sizes):
    lens = (300, 0, 77, 130)[:len(sizes)]
    case = Case(lens, heads, kv, d, max(sizes), 32, 32, sizes=sizes, seed=3)
    compare(*_verify(case), case.reference())


@pytest.mark.parametrize("heads,kv,d,nodes,window", [(8, 1, 128, 1, 1), (8, 2, 64, 4, 100), (8, 2, 128, 33, 64), (14, 2, 128, 64, 300)])
def test_window(heads, kv, d, nodes, window):
    case = Case((1000, 90, 0, window), heads, kv, d, nodes, 64, 16, seed=5)
    compare(*_verify(case, window=window), case.reference(window=window))


@pytest.mark.parametrize("heads,kv,d,sizes,theta", [(8, 1, 128, (1, 1, 1), 1e6), (8, 2, 64, (20, 0, 7), 1e4), (28, 4, 128, (64, 33, 2), 5e5)])
def test_rope(heads, kv, d, sizes, theta):
    case = Case((513, 40, 0), heads, kv, d, max(sizes), 64, 64, sizes=sizes, seed=6)
    # a rotated value on the border between two bf16 numbers may round either way (the
    # angle's error): one step, 2^-7, on at most every element of q and k
    out, lse, tol, lse_tol = case.reference(theta=theta)
    got_out, got_lse = _verify(case, theta=theta)
    compare(got_out, got_lse, (out, lse, tol + 2.0 ** -6 * (np.abs(out).max() + 1), lse_tol + 2.0 ** -5))


@pytest.mark.parametrize("nodes", [1, 4, 40])
@pytest.mark.parametrize("spread,values", [(3.0, 1.0), (0.0, 1e-6), (0.0, 1e4)])
def test_scales(nodes, spread, values):
    """Scales over many powers of two, and tiny and large values."""
    case = Case((777, 50), 8, 2, 128, nodes, 32, 16, seed=7, scale_spread=spread, values=values, peak=0.5)
    compare(*_verify(case), case.reference())


@pytest.mark.parametrize("nodes", [1, 40])
def test_zero_scales(nodes):
    """Blocks whose values (or keys) are all zero, by scale 0: weightless values, score 0."""
    case = Case((300,), 8, 2, 128, nodes, 32, 16, seed=8)
    for w in "kv":
        case.scales[w][::2] = np.where(np.isnan(case.scales[w][::2]), np.nan, 0.0)
    out, lse, tol, lse_tol = case.reference()
    # a value scale of 0 counts as 2^-60: at most 448 * 2^-60
    compare(*_verify(case), (out, lse, tol + 448 * 2.0 ** -60, lse_tol))


@pytest.mark.parametrize("nodes,heads", [(1, 4), (1, 16), (64, 8)])
def test_spiked_scores(nodes, heads):
    """One key far above the rest, late in a long sequence: the maximum is raised there."""
    case = Case((3000,), heads, 1, 128, nodes, 64, 32, seed=9, peak=8.0)
    compare(*_verify(case), case.reference())


def test_many_sequences():
    """More sequences than the plan carries lengths for."""
    lens = [int(x) for x in np.random.default_rng(1).integers(0, 200, 40)]
    case = Case(lens, 8, 2, 64, 3, 16, 16, seed=10)
    compare(*_verify(case), case.reference())


@pytest.mark.parametrize("nodes", [2, 40])
def test_bad_tree_is_reported(nodes):
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case((100,), 8, 2, 128, nodes, 32, 16)
    case.parent[1] = 1
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(1, 8, 2, 128, nodes, cu_seqlens_host=case.cu)
    call(q, cache, kt, vt, par, cu)
    assert call.check() == 5


@pytest.mark.parametrize("nodes", [1, 40])
def test_length_mismatch_is_reported(nodes):
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case((100,), 8, 2, 128, nodes, 32, 16)
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(1, 8, 2, 128, nodes, cu_seqlens_host=[0, 90])
    call(q, cache, kt, vt, par, cu)
    assert call.check() == 7


@pytest.mark.parametrize("nodes", [1, 40])
def test_bad_pages_read_inside_the_cache(nodes):
    """A table that names pages outside the cache gives some result, and no fault."""
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case((500,), 8, 2, 128, nodes, 32, 16)
    case.table[0, 3:9] = [-1, 2 ** 31 - 1, -2 ** 31, case.num_pages, 10 ** 6, -5]
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(1, 8, 2, 128, nodes, cu_seqlens_host=case.cu)
    call(q, cache, kt, vt, par, cu)
    assert call.check() == 0


@pytest.mark.parametrize("nodes", [1, 64])
def test_same_bits_again_on_a_stream_and_in_a_graph(nodes):
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case((1500, 200), 16, 2, 128, nodes, 64, 32, seed=12)
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(2, 16, 2, 128, nodes, max_prefix_len=1500)
    first = [x.clone() for x in call(q, cache, kt, vt, par, cu)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = call(q, cache, kt, vt, par, cu)
    side.synchronize()
    out, lse = torch.empty_like(q), torch.empty_like(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(q, cache, kt, vt, par, cu, out, lse)
    for _ in range(2):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, again, (out, lse)):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_rows_behind_the_last_tree_are_left():
    """Rows of out past the last sequence's tree are not written."""
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case((50, 60), 8, 2, 64, 6, 16, 16, sizes=(2, 3))
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(2, 8, 2, 64, 6, cu_seqlens_host=case.cu, tree=case.opts())
    big = torch.full((9, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 8), 7.0, device="cuda")
    call(q, cache, kt, vt, par, cu, big[:5], lse[:5])
    torch.cuda.synchronize()
    assert (big[5:] == 7.0).all() and (lse[5:] == 7.0).all()
