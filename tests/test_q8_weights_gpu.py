"""How far rounding a weight together with its block's value scale, to f16, may move an output
element. With c_j = w_j s_j (w a row's weights, s the value scales) and M the largest c_j of the
row, the kernels round P_j = 2^9 c_j / M' for some M' <= M: relative 2^-11 while P_j is at least
2^-14, f16's least normal number, and by at most 2^-25 below it. So c_j moves by at most
max(2^-11 c_j, 2^-34 M). The cases hold one block whose scale is far above the others', and whose
values are zero in every dimension but one: in the other dimensions nothing hides the error."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from tests.q8_harness import BF16_HALF, EXP_ERR, F16_HALF, Case, f64

pytestmark = pytest.mark.gpu


def _scales_of(case, b, with_tree, group):
    """The value scale of each key of sequence b: its block's, or for tree nodes 2^-14 times the
    power of two below the largest magnitude of their group of nodes (of one kv head)."""
    n = case.lens[b]
    per_key = np.stack([case.scales["v"][case.table[b, j // case.page], j % case.page // case.block] for j in range(n)])
    if not with_tree:
        return per_key.astype(np.float64)
    s, e = case.cu_tree[b], case.cu_tree[b + 1]
    v = np.abs(f64(case.v_tree)[s:e])
    tree = np.stack([2.0 ** (np.floor(np.log2(v[i // group * group:(i // group + 1) * group].max((0, 2)))) - 14)
                     for i in range(e - s)])
    return np.concatenate([per_key.astype(np.float64), tree])


def _reference(case, with_tree, group):
    """(out, tolerance, tolerance of 2^-11 alone)"""
    scale, g = case.d ** -0.5, case.Hq // case.Hkv
    q, kt, vt = f64(case.q), f64(case.k_tree), f64(case.v_tree)
    outs, tols, plain = [], [], []
    for b, n in enumerate(case.lens):
        s, e = case.cu_tree[b], case.cu_tree[b + 1]
        k = oq.gather(case.codes["k"], case.scales["k"], case.table[b], n, case.page, case.block)
        v = oq.gather(case.codes["v"], case.scales["v"], case.table[b], n, case.page, case.block)
        see = np.ones((e - s, n), dtype=bool)
        if with_tree:
            k, v = np.concatenate([k, kt[s:e]]), np.concatenate([v, vt[s:e]])
            see = np.concatenate([see, oq.ancestors(case.parent[s:e])], 1)
        sv = _scales_of(case, b, with_tree, group)
        out, tol, tol11 = (np.zeros((e - s, case.Hq, case.d)) for _ in range(3))
        for h in range(case.Hq):
            kk, vv, ss = k[:, h // g], v[:, h // g], sv[:, h // g]
            x = np.where(see, scale * (q[s:e, h] @ kk.T), -np.inf)
            reach = (scale * (np.abs(q[s:e, h]) @ np.abs(kk).T)).max(1, keepdims=True)
            w = np.exp(x - x.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            # scores and exponentials, as in the harness; they move both sums
            rel = np.exp((case.d + 8) * 2.0 ** -23 * (reach + 1.0)) - 1 + EXP_ERR
            most = (w * ss).max(1, keepdims=True)
            # a tree value below 2^-17 of f16's range loses bits too: 2^-25 of its scale at most
            coarse = w * (ss * (np.arange(len(ss)) >= n)) * 2.0 ** -25
            off = np.where(w > 0, np.maximum(F16_HALF * w, 2.0 ** -34 * most / ss), 0.0)
            out[:, h], spread = w @ vv, w @ np.abs(vv)
            base = BF16_HALF * np.abs(out[:, h]) + 2.02 * rel * spread + 1e-30
            tol[:, h] = base + 1.02 * (off @ np.abs(vv) + coarse.sum(1, keepdims=True))
            tol11[:, h] = base + 1.02 * F16_HALF * spread
        outs.append(out), tols.append(tol), plain.append(tol11)
    return tuple(np.concatenate(x) for x in (outs, tols, plain))


def _case(ratio, heads, kv, d, nodes, seed):
    case = Case((700, 300), heads, kv, d, nodes, 32, 32, seed=seed, peak=0.5)
    for b, n in enumerate(case.lens):
        page = case.table[b, n // 64]  # in the middle
        case.scales["v"][page] *= np.float32(2.0 ** ratio)
        keep = case.codes["v"][page][..., 0].copy()
        case.codes["v"][page] = 0
        case.codes["v"][page][..., 0] = keep
    return case


# rows a kv head: up to 8, 16 and 32 (the kernel that streams through registers), 40 and 160
@pytest.mark.parametrize("heads,kv,d,nodes", [(8, 2, 128, 1), (4, 1, 64, 4), (8, 2, 128, 8), (8, 2, 128, 10), (8, 2, 64, 40)])
@pytest.mark.parametrize("ratio", [0, 12, 20, 26, 32, 40])
@pytest.mark.parametrize("with_tree", [False, True])
def test_outputs_stay_within_the_bound(ratio, heads, kv, d, nodes, with_tree):
    from tree_verification_attention_longspec_b200 import CrossAttnQ8, VerifyAttnQ8
    case = _case(ratio, heads, kv, d, nodes, seed=ratio + nodes)
    cache, q, kt, vt, par, cu = case.device()
    kind = VerifyAttnQ8 if with_tree else CrossAttnQ8
    call = kind(case.B, heads, kv, d, nodes, cu_seqlens_host=case.cu)
    out, lse = call(q, cache, kt, vt, par, cu) if with_tree else call(q, cache, cu)
    assert call.check() == 0
    rows = nodes * heads // kv
    want, tol, plain = _reference(case, with_tree, 16 if rows <= 32 else nodes)
    off = np.abs(f64(out) - want)
    print(f"ratio {ratio}: {(off / tol).max():.3f} of the bound, {(off / plain).max():.3f} of 2^-11 alone")
    assert (off <= tol).all(), ((off / tol).max(), np.unravel_index((off / tol).argmax(), off.shape))
    if ratio <= 12:  # products this close are all normal f16 numbers
        assert (off <= plain).all()
    # the row's sum is of fp32 weights: the scales cost it nothing
    ref_lse = case.reference(with_tree=with_tree)[1:4:2]
    assert (np.abs(f64(lse) - ref_lse[0]) <= ref_lse[1]).all()


def test_an_ordinary_spread_of_scales_keeps_eleven_bits():
    """Scales within 2^8 of one another, and weights within 2^11: 2^-11 for every element."""
    from tree_verification_attention_longspec_b200 import CrossAttnQ8
    for nodes in (1, 40):
        case = _case(8, 8, 2, 128, nodes, seed=nodes)
        cache, q, _, _, _, cu = case.device()
        out, _ = CrossAttnQ8(case.B, 8, 2, 128, nodes, cu_seqlens_host=case.cu)(q, cache, cu)
        want, _, plain = _reference(case, False, nodes)
        assert (np.abs(f64(out) - want) <= plain).all()
    torch.cuda.synchronize()
