"""The 8-bit cache's and the sampling calls' refusals, and the oracle's own pins (no GPU)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import q8 as oq

INVALID, UNSUPPORTED = 1, 2
# Addresses that no refused call reads: every check of an argument comes before any launch.
P = {name: (i + 1) << 20 for i, name in enumerate(
    ["q", "k_tree", "v_tree", "parent", "cu", "out", "lse", "table", "k_pages", "v_pages", "k_scale", "v_scale", "ws",
     "cu_new", "cu_out", "accept_len", "accept_path", "cu_tree", "k_new", "v_new", "logits", "uniform", "token", "draft",
     "next", "temperature", "top_k", "top_p", "min_p"])}


def _kv(**change):
    from tree_verification_attention_longspec_b200 import binding
    a = dict(page_size=64, scale_block=32, max_pages_per_seq=8, num_pages=20, page_table=P["table"],
             k_pages=P["k_pages"], v_pages=P["v_pages"], k_scale=P["k_scale"], v_scale=P["v_scale"])
    a.update(change)
    return binding.KvQ8(*a.values())


def _dims(**change):
    from tree_verification_attention_longspec_b200.binding import make_dims
    a = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, tree_size=4, max_prefix_len=512)
    a.update(change)
    return make_dims(**a)[0]


BAD_KV = [
    (dict(page_size=48, scale_block=16), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=0), UNSUPPORTED), (dict(page_size=-64), UNSUPPORTED), (dict(page_size=192), UNSUPPORTED),
    (dict(page_size=(1 << 20) + 128), UNSUPPORTED),
    (dict(scale_block=8), UNSUPPORTED), (dict(scale_block=0), UNSUPPORTED), (dict(scale_block=256), UNSUPPORTED),
    (dict(scale_block=48), UNSUPPORTED), (dict(scale_block=128), INVALID),
    (dict(page_size=384, scale_block=64, num_pages=6_000_000), UNSUPPORTED),
    (dict(num_pages=0), INVALID), (dict(num_pages=-1), INVALID), (dict(num_pages=1 << 25), UNSUPPORTED),
    (dict(num_pages=1 << 40), UNSUPPORTED), (dict(max_pages_per_seq=0), INVALID),
    (dict(max_pages_per_seq=1 << 26), UNSUPPORTED),
] + [({name: None}, INVALID) for name in ("page_table", "k_pages", "v_pages", "k_scale", "v_scale")] + [
    (dict(page_table=P["table"] + 2), INVALID), (dict(k_pages=P["k_pages"] + 8), INVALID),
    (dict(v_pages=P["v_pages"] + 1), INVALID), (dict(k_scale=P["k_scale"] + 2), INVALID),
    (dict(v_scale=P["v_scale"] + 1), INVALID)]


def _attend(lib, kv, dims, tree=None, **change):
    a = dict(q=P["q"], k_tree=P["k_tree"], v_tree=P["v_tree"], parent=P["parent"], cu=P["cu"], out=P["out"], lse=P["lse"])
    a.update(change)
    r = ctypes.byref
    return lib.ls_verify_attn_q8(a["q"], None if kv is None else r(kv), a["k_tree"], a["v_tree"], a["parent"], a["cu"],
                                 None if tree is None else r(tree), a["out"], a["lse"],
                                 None if dims is None else r(dims), P["ws"], 0, None)


def _cross(lib, kv, dims, **change):
    a = dict(q=P["q"], cu=P["cu"], out=P["out"], lse=P["lse"])
    a.update(change)
    r = ctypes.byref
    return lib.ls_cross_attn_q8(a["q"], None if kv is None else r(kv), a["cu"], a["out"], a["lse"],
                                None if dims is None else r(dims), P["ws"], 0, None)


def _append(lib, kv, dims, **change):
    a = dict(k=P["k_new"], v=P["v_new"], cu_new=P["cu_new"], total=10, most=8, cu=P["cu"], out=P["cu_out"])
    a.update(change)
    r = ctypes.byref
    return lib.ls_kv_append_q8(a["k"], a["v"], a["cu_new"], a["total"], a["most"], a["cu"], a["out"],
                               None if kv is None else r(kv), None if dims is None else r(dims), None)


def _commit(lib, kv, dims, **change):
    a = dict(k=P["k_tree"], v=P["v_tree"], cu_tree=None, nodes=0, length=P["accept_len"], path=P["accept_path"],
             cu=P["cu"], out=P["cu_out"])
    a.update(change)
    r = ctypes.byref
    return lib.ls_kv_commit_q8(a["k"], a["v"], a["cu_tree"], a["nodes"], a["length"], a["path"], a["cu"], a["out"],
                               None if kv is None else r(kv), None if dims is None else r(dims), None)


@pytest.mark.parametrize("change,want", BAD_KV)
def test_cache_descriptions_refused(cuda_lib, change, want):
    for call in (_attend, _cross, _append, _commit):
        assert call(cuda_lib, _kv(**change), _dims()) == want, call.__name__


def test_attention_arguments_refused(cuda_lib):
    from tree_verification_attention_longspec_b200.binding import TreeOpts
    for call in (_attend, _cross):
        assert call(cuda_lib, None, _dims()) == INVALID
        assert call(cuda_lib, _kv(), None) == INVALID
        for name, off in (("q", 8), ("cu", 2), ("out", 4), ("lse", 1)):
            assert call(cuda_lib, _kv(), _dims(), **{name: None}) == INVALID, name
            assert call(cuda_lib, _kv(), _dims(), **{name: P[name] + off}) == INVALID, name
        # a table shorter than the longest sequence, by either length
        assert call(cuda_lib, _kv(), _dims(max_prefix_len=513)) == INVALID
        assert call(cuda_lib, _kv(), _dims(max_prefix_len=0, cu_seqlens_host=[0, 1, 514])) == INVALID
        assert call(cuda_lib, _kv(), _dims(head_dim=96)) == UNSUPPORTED
        assert call(cuda_lib, _kv(), _dims(tree_size=129)) == UNSUPPORTED
        assert call(cuda_lib, _kv(), _dims(num_q_heads=7)) == INVALID
    for name, off in (("k_tree", 8), ("v_tree", 4), ("parent", 2)):
        assert _attend(cuda_lib, _kv(), _dims(), **{name: None}) == INVALID, name
        assert _attend(cuda_lib, _kv(), _dims(), **{name: P[name] + off}) == INVALID, name
    assert _attend(cuda_lib, _kv(), _dims(), TreeOpts(window=-1)) != 0
    assert _attend(cuda_lib, _kv(), _dims(), TreeOpts(cu_tree=P["cu_tree"], total_nodes=9)) != 0


def test_writers_arguments_refused(cuda_lib):
    for call in (_append, _commit):
        assert call(cuda_lib, None, _dims()) == INVALID
        assert call(cuda_lib, _kv(), None) == INVALID
        assert call(cuda_lib, _kv(), _dims(head_dim=256)) == UNSUPPORTED
        assert call(cuda_lib, _kv(), _dims(), cu=None) == INVALID
        assert call(cuda_lib, _kv(), _dims(), cu=P["cu"] + 1) == INVALID
        assert call(cuda_lib, _kv(), _dims(), out=P["cu_out"] + 2) == INVALID
        # the lengths after the call over those before it: the same array, or a part of it
        for off in (-8, -4, 0, 4, 8):
            assert call(cuda_lib, _kv(), _dims(), out=P["cu"] + off) == INVALID
        for name, off in (("k", 8), ("v", 2)):
            assert call(cuda_lib, _kv(), _dims(), **{name: None}) == INVALID
            assert call(cuda_lib, _kv(), _dims(), **{name: (1 << 24) + off}) == INVALID
    assert _append(cuda_lib, _kv(), _dims(), out=P["cu_new"]) == INVALID
    assert _append(cuda_lib, _kv(), _dims(), cu_new=None) == INVALID
    assert _append(cuda_lib, _kv(), _dims(), cu_new=P["cu_new"] + 2) == INVALID
    assert _append(cuda_lib, _kv(), _dims(), total=-1) == INVALID
    assert _append(cuda_lib, _kv(), _dims(), most=-1) == INVALID
    assert _commit(cuda_lib, _kv(), _dims(tree_size=0)) == INVALID
    assert _commit(cuda_lib, _kv(), _dims(tree_size=129)) == UNSUPPORTED
    assert _commit(cuda_lib, _kv(), _dims(batch=1 << 24, tree_size=128)) == UNSUPPORTED
    for name in ("length", "path"):
        assert _commit(cuda_lib, _kv(), _dims(), **{name: None}) == INVALID
        assert _commit(cuda_lib, _kv(), _dims(), **{name: P["accept_len"] + 2}) == INVALID
    assert _commit(cuda_lib, _kv(), _dims(), out=P["accept_len"]) == INVALID
    assert _commit(cuda_lib, _kv(), _dims(), out=P["accept_path"] + 16) == INVALID
    assert _commit(cuda_lib, _kv(), _dims(), out=P["cu_tree"], cu_tree=P["cu_tree"], nodes=8) == INVALID
    assert _commit(cuda_lib, _kv(), _dims(), cu_tree=P["cu_tree"], nodes=9) == INVALID  # more than 2 * 4
    assert _commit(cuda_lib, _kv(), _dims(), cu_tree=P["cu_tree"], nodes=-1) == INVALID
    assert _commit(cuda_lib, _kv(), _dims(), cu_tree=P["cu_tree"] + 2, nodes=8) == INVALID


def _sample(lib, **change):
    from tree_verification_attention_longspec_b200 import binding
    a = dict(logits=P["logits"], stride=1000, uniform=P["uniform"], out=P["out"], rows=4, vocab=1000,
             dtype=binding.LS_DTYPE_BF16)
    opts = {k: change.pop(k) for k in ("temperature", "top_k", "top_p", "min_p") if k in change}
    a.update(change)
    o = binding.SampleOpts(*[opts.get(k) for k in ("temperature", "top_k", "top_p", "min_p")])
    return lib.ls_sample(a["logits"], a["stride"], a["uniform"], ctypes.byref(o), a["out"], a["rows"], a["vocab"],
                         a["dtype"], None)


def _accept(lib, **change):
    from tree_verification_attention_longspec_b200 import binding
    a = dict(logits=P["logits"], uniform=P["uniform"], draft=P["draft"], parent=P["parent"], cu_tree=None, nodes=0,
             token=P["token"], length=P["accept_len"], path=P["accept_path"], after=P["next"])
    shape = dict(batch=2, tree_size=4, vocab=100, kind=binding.LS_DTYPE_F32)
    shape.update({k: change.pop(k) for k in list(change) if k in shape})
    a.update(change)
    d = binding.AcceptDims(*shape.values())
    return lib.ls_tree_accept_sample(a["logits"], a["uniform"], None, a["draft"], a["parent"], a["cu_tree"], a["nodes"],
                                     a["token"], a["length"], a["path"], a["after"], ctypes.byref(d), None)


def test_sampling_arguments_refused(cuda_lib):
    for name in ("logits", "uniform", "out"):
        assert _sample(cuda_lib, **{name: None}) == INVALID
        assert _sample(cuda_lib, **{name: P[name] + 1}) == INVALID
    for name in ("temperature", "top_k", "top_p", "min_p"):
        assert _sample(cuda_lib, **{name: P[name] + 2}) == INVALID
    assert _sample(cuda_lib, rows=-1) == INVALID
    assert _sample(cuda_lib, vocab=0) == INVALID
    assert _sample(cuda_lib, stride=999) == INVALID
    assert _sample(cuda_lib, dtype=7) == INVALID
    assert _sample(cuda_lib, vocab=(1 << 20) + 1, stride=1 << 21) == UNSUPPORTED
    assert _sample(cuda_lib, rows=(1 << 27) + 1) == UNSUPPORTED
    assert _sample(cuda_lib, rows=0, logits=None, uniform=None, out=None) == 0  # nothing to do


def test_sampled_acceptance_arguments_refused(cuda_lib):
    for name, off in (("logits", 2), ("uniform", 1), ("draft", 2), ("parent", 1), ("token", 2), ("length", 2),
                      ("path", 1), ("after", 2)):
        at = dict(logits=P["logits"], uniform=P["uniform"], draft=P["draft"], parent=P["parent"], token=P["token"],
                  length=P["accept_len"], path=P["accept_path"], after=P["next"])[name]
        assert _accept(cuda_lib, **{name: None}) == INVALID, name
        assert _accept(cuda_lib, **{name: at + off}) == INVALID, name
    for shape, want in ((dict(batch=0), INVALID), (dict(tree_size=0), INVALID), (dict(vocab=0), INVALID),
                        (dict(tree_size=129), UNSUPPORTED), (dict(vocab=(1 << 20) + 1), UNSUPPORTED),
                        (dict(batch=1 << 26), UNSUPPORTED), (dict(kind=5), INVALID)):
        assert _accept(cuda_lib, **shape) == want, shape
    assert _accept(cuda_lib, cu_tree=P["cu_tree"], nodes=9) == INVALID
    assert _accept(cuda_lib, cu_tree=P["cu_tree"], nodes=-1) == INVALID
    assert _accept(cuda_lib, cu_tree=P["cu_tree"] + 2, nodes=8) == INVALID


def test_python_calls_refuse_host_tensors_and_wrong_types():
    from tree_verification_attention_longspec_b200 import KVCacheQ8, sample, tree_accept_sample
    x = torch.zeros(2, 10)
    with pytest.raises(ValueError, match="CUDA"):
        sample(x, torch.zeros(2))
    with pytest.raises(TypeError, match="logits"):
        sample(x.half(), torch.zeros(2))
    with pytest.raises(TypeError, match="logits"):
        sample([[1.0, 2.0]], torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        tree_accept_sample(x, torch.zeros(2), torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 2)
    pages = torch.zeros(2, 16, 1, 64, dtype=torch.uint8)
    scale, table = torch.ones(2, 1, 1), torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages.*CUDA"):
        KVCacheQ8(pages, pages, scale, scale, table)
    with pytest.raises(TypeError, match="k_pages"):
        KVCacheQ8(pages.half(), pages, scale, scale, table)
    for page, block in ((64, 24), (48, 32), (16, 32), (100, None)):
        with pytest.raises(ValueError, match="scale_block"):
            KVCacheQ8.empty(2, page, 1, 64, table, scale_block=block)


# ---- the oracle

def test_oracle_e4m3_is_the_format():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oq.TABLE, want, equal_nan=True)
    # every value, every midpoint and its neighbours, from -448 to 448
    v = np.unique(want[~np.isnan(want)])
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), [1e-12, -1e-12]])
    got = oq.TABLE[oq.e4m3_encode(x)]
    assert np.array_equal(got, torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy())
    assert oq.TABLE[oq.e4m3_encode([449.0, 1e30, np.inf, -np.inf])].tolist() == [448.0, 448.0, 448.0, -448.0]
    assert np.isnan(oq.TABLE[oq.e4m3_encode([np.nan])]).all()


@pytest.mark.parametrize("amax,want", [(0.0, -60), (448.0, 0), (448.0000001, 1), (224.0, -1), (1.0, -8), (1.75, -8),
                                       (1.76, -7), (3e38, 64), (1e-30, -60)])
def test_oracle_scale_exponent(amax, want):
    e = oq.scale_exponent(amax)
    assert e == want
    assert amax <= 448 * 2.0 ** e or e == 64
    assert e == -60 or amax > 448 * 2.0 ** (e - 1)


def test_oracle_append_by_hand():
    """One head of two values, blocks of 16: token 0 at 1.0 gets scale 2^-8; a token at 500
    raises it to 2 and rounds the first one's code again."""
    pages, scale = np.full((1, 16, 1, 2), 0x7F, np.uint8), np.full((1, 1, 1), 5.0)
    table = np.zeros((1, 1), np.int32)
    pages, scale = oq.append(pages, scale, table, [0], [[np.array([[1.0, -0.5]])]], 16, 16)
    assert scale[0, 0, 0] == 2.0 ** -8 and (oq.TABLE[pages[0, 0, 0]] == [256.0, -128.0]).all()
    assert (pages[0, 1:] == 0x7F).all()
    pages, scale = oq.append(pages, scale, table, [1], [[np.array([[500.0, 1.0]])]], 16, 16)
    assert scale[0, 0, 0] == 2.0
    assert (oq.TABLE[pages[0, 0, 0]] * 2 == [1.0, -0.5]).all()     # 0.5 and -0.25: e4m3 has them
    assert (oq.TABLE[pages[0, 1, 0]] * 2 == [512.0, 1.0]).all()    # 250 rounds to 256


def test_oracle_sampling_by_hand():
    x = np.log([0.5, 0.2, 0.2, 0.1])
    draw = lambda u, **kw: oq.sample_row(x, u, **kw)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.49, 0.51, 0.71, 0.95)] == [0, 0, 1, 2, 3]
    assert [draw(u, k=1) for u in (0.0, 0.99)] == [0, 0]
    assert [draw(u, k=2) for u in (0.70, 0.73, 0.99)] == [0, 1, 1]           # 5/7, then the first of the two 0.2
    assert [draw(u, p=0.6) for u in (0.70, 0.73, 0.99)] == [0, 1, 1]         # 0.5 < 0.6: the next one too
    assert [draw(u, p=0.45) for u in (0.0, 0.99)] == [0, 0]
    assert [draw(u, p=0.0) for u in (0.0, 0.99)] == [0, 0]
    assert [draw(u, m=0.3) for u in (0.5, 0.6, 0.8, 0.99)] == [0, 1, 2, 2]   # 0.1 / 0.5 is below 0.3
    # p of what top-k left: 0.5 / 0.9 reaches 0.55, so the border is there and not at 0.5 / 1
    assert draw(0.99, k=3, p=0.55) == 0 and draw(0.99, k=3, p=0.56) == 1
    assert draw(0.99, t=0.0) == 0 and oq.sample_row(np.array([1.0, 2.0, 2.0]), 0.99, 0.0)[0] == 1
    # a temperature of 1/2 squares the weights: 25, 4, 4, 1
    assert [draw(u, t=0.5) for u in (24.9 / 34, 25.1 / 34, 29.1 / 34, 33.1 / 34)] == [0, 1, 2, 3]


def test_oracle_attention_by_hand():
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[5.0, 5.0]]])
    v = np.array([[[1.0, 2.0]], [[3.0, 4.0]], [[100.0, 100.0]]])
    q = np.array([[[np.log(3.0), 0.0], [0.0, 0.0]]])
    out, lse, spread, reach = oq.attention(q, k, v, np.array([[True, True, False]]), 1.0)
    assert np.allclose(out[0, 0], [1.5, 2.5]) and np.allclose(out[0, 1], [2.0, 3.0])  # weights 3:1 and 1:1
    assert np.allclose(lse[0], [np.log(4.0), np.log(2.0)])
    out, lse, _, _ = oq.attention(q, k, v, np.zeros((1, 3), bool), 1.0)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_oracle_walk_by_hand():
    parent, draft = [-1, 0, 0, 1, 2], [9, 5, 6, 7, 8]
    assert oq.walk([6, 0, 8, 0, 3], draft, parent) == (2, [0, 2, 4], 3)
    assert oq.walk([1, 0, 0, 0, 0], draft, parent) == (0, [0], 1)
    assert oq.walk([1], [1], [0]) == (-1, [], -1)
