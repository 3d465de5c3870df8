"""Calls of the 8-bit cache and of sampling at their edges: infinities in masked places, rows
of few or tiny values, offsets past 32 bits, shared pages, captured and concurrent steps."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from tests.q8_harness import Case, bf16, compare, f64
from tests.test_q8_cache_gpu import Pool
from tests.test_sample_gpu import _check, _sample

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("nodes,heads", [(4, 4), (24, 4), (40, 4), (70, 16)])
def test_an_infinite_tree_key_reaches_only_the_rows_that_see_it(nodes, heads):
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case((300, 40), heads, 2, 128, nodes, 32, 16, seed=nodes)
    leaf = nodes - 1  # no node's ancestor
    clean = case.reference()
    case.k_tree[leaf, :, 3] = float("inf")
    case.k_tree[nodes + leaf, :, 5] = float("nan")
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(2, heads, 2, 128, nodes, cu_seqlens_host=case.cu)
    out, lse = call(q, cache, kt, vt, par, cu)
    assert call.check() == 0
    rest = np.delete(np.arange(2 * nodes), [leaf, nodes + leaf])
    compare(out[_dev(rest)], lse[_dev(rest)], [x[rest] for x in clean])


def test_commit_of_a_path_longer_than_its_tree_leaves_room_for_the_others():
    """The first tree's path names nodes it does not have; the second's is committed whole."""
    pool = Pool((0, 5), (140, 30), 1, 64, 16, 16)
    cache = pool.device()
    T, k = 128, bf16(np.random.default_rng(2).standard_normal((4, 1, 64)))
    path = np.full((2, T), 9, dtype=np.int32)
    path[0, 0] = 0
    path[1, :3] = [0, 1, 2]
    cu = cache.commit(k.cuda(), k.cuda(), pool.cu, _dev(np.array([127, 2], np.int32)), _dev(path),
                      cu_tree=_dev(np.array([0, 1, 4], np.int32)))
    x = f64(k)
    rows = [[x[0]] + [None] * 127, [x[1], x[2], x[3]]]
    pool.expect({"k": rows, "v": rows}, cu, [128, 8])


@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
@pytest.mark.parametrize("d,page,block", [(64, 16, 16), (64, 128, 128), (128, 128, 32), (128, 64, 64), (128, 256, 128)])
def test_append_to_blocks_of_another_writers_scale(d, page, block, size):
    """Scales of 1.25 * 2^k: kept where they are large enough (the rows are divided by them), and
    else replaced. (8-bit values over 5 / 4 come no nearer to the middle of two codes, short of
    lying on it, than 2^-12 of themselves, so the kernel's division in fp32 rounds to the same.)"""
    r = np.random.default_rng(block)
    lens, new = (block - 1, block // 2 + 3, 5, 0), (block + 1, 2 * block, 1, block)
    pool = Pool(lens, [a + b for a, b in zip(lens, new)], 3, d, page, block, seed=d)
    for w in "kv":
        pool.scales[w] *= np.float32(1.25)
    cache = pool.device()
    cu_new = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = (bf16(size * r.standard_normal((sum(new), 3, d))) for _ in range(2))
    cu = cache.append(k.cuda(), v.cuda(), pool.cu, _dev(cu_new), max(new))
    split = [list(x) for x in np.split(f64(k), cu_new[1:-1])], [list(x) for x in np.split(f64(v), cu_new[1:-1])]
    pool.expect({"k": split[0], "v": split[1]}, cu, [a + b for a, b in zip(lens, new)])


def test_sequences_that_share_pages():
    """A common prompt's pages in every sequence's table."""
    case = Case((640, 640, 640), 8, 2, 128, 5, 64, 32, seed=4)
    case.table[1:, :6] = case.table[0, :6]
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(3, 8, 2, 128, 5, max_prefix_len=640)
    compare(*call(q, cache, kt, vt, par, cu), case.reference())


@pytest.mark.parametrize("nodes", [2, 48])
def test_a_cache_of_more_than_2_to_the_31_bytes(nodes):
    """Written and read in its last pages, with the answer of a small cache."""
    from tree_verification_attention_longspec_b200 import KVCacheQ8, VerifyAttnQ8
    kv, d, page, n = 8, 128, 64, 200
    pages = 2 ** 31 // (kv * d * page) + 40
    case = Case((n,), 16, kv, d, nodes, page, 64, seed=nodes)
    k, v = (bf16(np.random.default_rng(s).standard_normal((n, kv, d))).cuda() for s in (1, 2))
    zero, ends = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    got = []
    for total, at in ((8, (3, 0, 6, 1)), (pages, (pages - 1, 0, pages - 7, pages - 2))):
        cache = KVCacheQ8.empty(total, page, kv, d, torch.tensor([at], dtype=torch.int32, device="cuda"))
        cu = cache.append(k, v, zero, ends, n)
        call = VerifyAttnQ8(1, 16, kv, d, nodes, max_prefix_len=n)
        got.append(call(case.q.cuda(), cache, case.k_tree.cuda(), case.v_tree.cuda(), _dev(case.parent), cu))
        assert call.check() == 0
        del cache
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_rows_of_logits_more_than_2_to_the_31_elements_apart():
    from tree_verification_attention_longspec_b200 import sample
    stride, vocab = 2 ** 31 + 24, 5000
    store = torch.empty(stride + vocab, dtype=torch.bfloat16, device="cuda")
    far = store.as_strided((2, vocab), (stride, 1))
    far.copy_(torch.randn(2, vocab, generator=torch.Generator().manual_seed(1)) * 3)
    u = torch.tensor([0.3, 0.8], device="cuda")
    for opts in ({}, {"top_p": 0.9}, {"top_k": 30}):
        assert torch.equal(sample(far, u, **opts), sample(far.contiguous(), u, **opts))


def _filters(r, rows, vocab):
    return dict(temperature=r.choice([0.2, 0.7, 1.0, 3.0, 50.0], rows), top_k=r.choice([0, 1, 3, 40, vocab // 2], rows),
                top_p=r.choice([0.2, 0.9, 0.999, 1.0], rows), min_p=r.choice([0.0, 0.0, 0.05, 0.9], rows))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["negative", "tiny", "around zero", "zero tops", "wide", "narrow", "two values"])
@pytest.mark.parametrize("vocab", [50, 6000, 60000])
def test_rows_of_odd_values(kind, vocab, dtype):
    r = np.random.default_rng(len(kind) + vocab)
    rows = 24
    x = r.standard_normal((rows, vocab))
    if kind == "negative":
        x = -np.abs(x) * 5 - r.choice([0.0, 1e-3, 100.0], (rows, 1))
    elif kind == "tiny":
        x = x * 10.0 ** r.integers(-38, -3, (rows, 1))
    elif kind == "around zero":
        x = x * 10.0 ** r.integers(-12, 2, (rows, vocab))
    elif kind == "zero tops":
        x = np.where(r.random((rows, vocab)) < 0.2, 0.0, -np.abs(x) * 10.0 ** r.integers(-6, 2, (rows, vocab)))
    elif kind == "wide":
        x = x * 10.0 ** r.integers(0, 30, (rows, 1))
    elif kind == "narrow":
        x = 100.0 + x * 1e-3
    else:
        x = np.where(r.random((rows, vocab)) < 0.5, -3.0, 2.0)
    got, want, margin = _sample(x, r.random(rows), dtype, **_filters(r, rows, vocab))
    # a border of top-p that falls between two entries by rounding alone may move: u then
    # decides, and rows whose number lies near a border are left out
    bad = (got != want) & (margin > 1e-9)
    assert not bad.any(), (np.flatnonzero(bad), got[bad], want[bad])


def test_an_infinite_temperature_keeps_every_finite_logit():
    r = np.random.default_rng(9)
    x = r.standard_normal((8, 700))
    x[:, ::7] = -np.inf
    m = np.array([0.0, 0.5, 1.0, 2.0] * 2)
    with np.errstate(invalid="ignore"):
        _check(*_sample(x, r.random(8), temperature=np.full(8, np.inf), min_p=m))


def test_min_p_that_ends_before_the_other_filters():
    r = np.random.default_rng(11)
    x = r.standard_normal((40, 9000)) * 2
    for dtype in ("f32", "bf16"):
        _check(*_sample(x, r.random(40), dtype, min_p=r.uniform(0.3, 1.0, 40), top_p=np.full(40, 0.95)))
        _check(*_sample(x, r.random(40), dtype, min_p=r.uniform(0.3, 1.0, 40), top_k=np.full(40, 500)))


@pytest.mark.parametrize("small", [1e-6, 0.0, 2.0 ** -11])
@pytest.mark.parametrize("few", [3, 1000])
def test_top_k_that_ends_below_zero_with_tiny_logits_above(small, few):
    """top-p's border lies among the large values, and hangs on what top-k left of the low ones."""
    r = np.random.default_rng(few)
    x = np.concatenate([np.full(2000, 1.0), np.full(few, small), np.full(3000, -1.0)])
    rows = np.stack([r.permutation(x) for _ in range(40)])
    p = np.linspace(0.5, 0.82, 40)
    for dtype in ("f32", "bf16"):
        _check(*_sample(rows, r.random(40), dtype, top_k=np.full(40, 2000 + few + 500), top_p=p))


@pytest.mark.parametrize("vocab", [4000, 40000])
def test_borders_above_among_and_below_small_logits(vocab):
    """bf16 rows with zeros and logits too small to have a bin of their own, and thresholds of
    each kind on either side of them and among them."""
    r = np.random.default_rng(vocab)
    n = 48
    x = r.standard_normal((n, vocab)) * r.choice([0.3, 2.0], (n, 1))
    few = r.random((n, vocab)) < r.choice([0.001, 0.01, 0.3], (n, 1))
    x = np.where(few, r.choice([0.0, -0.0, 1e-5, -1e-5, 3e-4, -3e-4, 1e-30], (n, vocab)), x)
    half = (x > 1e-3).sum(1)
    low = (x > -1e-3).sum(1)
    at = r.choice([0.5, 0.9, 1.0, 1.02, 1.1, 1.5], n)
    for k in (np.zeros(n), half * at, low * at, np.full(n, 10)):
        for p in (np.ones(n), r.uniform(0.3, 1.0, n), np.full(n, 0.995)):
            for m in (np.zeros(n), np.exp(-x.max(1)) * r.choice([0.9, 1.0, 1.1], n)):
                _check(*_sample(x, r.random(n), "bf16", top_k=k.astype(int), top_p=p, min_p=m))


@pytest.mark.parametrize("scale", [0.1, 3.0, 12.0, 40.0])
def test_logits_inside_and_outside_the_plain_bins(scale):
    """bf16 logits below and above 32 in magnitude, and runs of small ones."""
    r = np.random.default_rng(int(scale * 10))
    x = r.standard_normal((24, 30000)) * scale
    x[::3, :400] *= 1e-4
    x[1::3, 0] = 32.0
    x[2::3, 5] = -32.0
    opts = dict(temperature=r.choice([0.3, 1.0, 5.0], 24), top_k=r.choice([0, 20, 3000], 24), top_p=r.choice([0.5, 0.95, 1.0], 24))
    _check(*_sample(x, r.random(24), "bf16", **opts))


def _step(state, call, cache, parts, gate):
    """One decoding step: attention with the new token, its logits, its choice, its append."""
    from tree_verification_attention_longspec_b200 import sample
    q, kt, vt, par, u, head = parts
    out, _ = call(q, cache, kt, vt, par, state["cu"], state["out"], state["lse"])
    token = sample(out.flatten(1) @ head, u, temperature=0.8, top_p=0.9, out=state["token"])
    cache.append(kt, vt, state["cu"], gate, 1, cu_seqlens_out=state["next"])
    state["cu"].copy_(state["next"])
    return token


def test_a_captured_decoding_step_follows_the_growing_cache():
    from tree_verification_attention_longspec_b200 import KVCacheQ8, VerifyAttnQ8
    B, kv, heads, d, page, vocab = 3, 2, 8, 64, 16, 300
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    parts = (rand(B, heads, d) * 2, rand(B, kv, d), rand(B, kv, d), torch.full((B,), -1, dtype=torch.int32, device="cuda"),
             torch.rand(B, generator=g).cuda(), rand(heads * d, vocab))
    table = torch.randperm(B * 8, generator=g).to(torch.int32).view(B, 8).cuda()
    gate = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    prompt, start = rand(60, kv, d), torch.tensor([0, 14, 14, 60], dtype=torch.int32, device="cuda")
    runs = []
    for captured in (False, True):
        cache = KVCacheQ8.empty(B * 8, page, kv, d, table)
        cu = cache.append(prompt, prompt, torch.zeros_like(start), start, 46)
        call = VerifyAttnQ8(B, heads, kv, d, 1, max_prefix_len=128)
        state = dict(cu=cu, next=torch.empty_like(cu), out=torch.empty_like(parts[0]),
                     lse=torch.empty(B, heads, device="cuda"), token=torch.empty(B, dtype=torch.int32, device="cuda"))
        seen = []
        if captured:
            keep = [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8), cache.k_scale,
                                        cache.v_scale, cu)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                _step(state, call, cache, parts, gate)  # warm-up of the library product
            torch.cuda.current_stream().wait_stream(side)
            for t, was in zip((cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8), cache.k_scale,
                               cache.v_scale, cu), keep):
                t.copy_(was)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                _step(state, call, cache, parts, gate)
        for _ in range(40):
            graph.replay() if captured else _step(state, call, cache, parts, gate)
            seen += [state["out"].clone(), state["lse"].clone(), state["token"].clone(), state["cu"].clone()]
            assert call.check() == 0
        seen += [cache.k_pages.view(torch.uint8).clone(), cache.v_scale.clone()]
        runs.append(seen)
    assert runs[0][-3].tolist() == [0, 54, 94, 180]
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_two_streams_at_once():
    """Calls with their own workspaces and outputs, on one cache, at the same time."""
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8, sample
    x = torch.randn(64, 50000, generator=torch.Generator().manual_seed(1)).cuda().to(torch.bfloat16)
    u = torch.rand(64, generator=torch.Generator().manual_seed(2)).cuda()
    want_tokens = sample(x, u, top_p=0.9)
    work = []
    cases = [Case((4000, 100), 16, 2, 128, n, 64, 32, seed=5) for n in (1, 64)]
    for case in cases:
        cache, q, kt, vt, par, cu = case.device()
        call = VerifyAttnQ8(2, 16, 2, 128, case.T, max_prefix_len=4000)
        work.append((call, (q, cache, kt, vt, par, cu), call(q, cache, kt, vt, par, cu)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(5):
        for (call, args, _), s in zip(work, streams):
            with torch.cuda.stream(s):
                got.append(call(*args))
        with torch.cuda.stream(streams[2]):
            tokens = sample(x, u, top_p=0.9)
            got.append((tokens,))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        want = (want_tokens,) if i % 3 == 2 else work[i % 3][2]
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_refusals_on_device_tensors():
    from tree_verification_attention_longspec_b200 import CrossAttnQ8, KVCacheQ8, VerifyAttnQ8, sample, tree_accept_sample
    from tree_verification_attention_longspec_b200.binding import LSError
    case = Case((100,), 8, 2, 128, 3, 32, 16)
    cache, q, kt, vt, par, cu = case.device()
    call = VerifyAttnQ8(1, 8, 2, 128, 3, cu_seqlens_host=case.cu)
    for bad in ((q[:2], kt, vt, par, cu), (q.float(), kt, vt, par, cu), (q, kt[:, :1], vt, par, cu), (q, kt, vt.cpu(), par, cu),
                (q, kt, vt, par.long(), cu), (q, kt, vt, par, cu[:1]), (q.transpose(0, 1).contiguous().transpose(0, 1), kt, vt, par, cu)):
        with pytest.raises((TypeError, ValueError)):
            call(bad[0], cache, *bad[1:])
    with pytest.raises(TypeError, match="cache"):
        call(q, None, kt, vt, par, cu)
    other = KVCacheQ8.empty(4, 32, 2, 64, torch.zeros(1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="head dimension"):
        call(q, other, kt, vt, par, cu)
    short = KVCacheQ8.empty(4, 32, 2, 128, torch.zeros(1, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(LSError):  # 100 tokens, and a table for 64
        call(q, short, kt, vt, par, cu)
    call.ws_bytes -= 1024
    with pytest.raises(LSError):
        call(q, cache, kt, vt, par, cu)
    with pytest.raises(ValueError, match="tree options"):
        CrossAttnQ8(1, 8, 2, 128, 3, tree=case.opts())
    with pytest.raises(LSError):  # the new lengths over the old ones
        cache.append(kt, vt, cu, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), 3, cu_seqlens_out=cu)
    with pytest.raises(ValueError, match="accept_path"):
        cache.commit(kt, vt, cu, par[:1], par)
    x, u = torch.zeros(6, 40, device="cuda"), torch.zeros(6, device="cuda")
    for kw in (dict(top_k=torch.zeros(6, device="cuda")), dict(top_p=torch.zeros(5, device="cuda")),
               dict(temperature=torch.zeros(6, dtype=torch.float64, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            sample(x, u, **kw)
    with pytest.raises(ValueError, match="rows"):
        sample(x.t(), torch.zeros(40, device="cuda"))
    with pytest.raises(ValueError, match="rows"):
        sample(x[:1].expand(6, 40), u)
    i = torch.zeros(6, dtype=torch.int32, device="cuda")
    for size in (0, 4, 129):
        with pytest.raises((ValueError, LSError)):
            tree_accept_sample(x, u, i, i, size)
    with pytest.raises(ValueError, match="contiguous"):
        tree_accept_sample(x[:, :20], u, i, i, 3)
