"""Sampling and sampled tree acceptance against the fp64 oracle: tokens must be equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import q8 as oq

pytestmark = pytest.mark.gpu

INF = np.inf


def _sample(x, u, dtype="f32", **opts):
    from tree_verification_attention_longspec_b200 import sample
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()
    if dtype == "bf16":
        t = t.to(torch.bfloat16)
    kw = {}
    for name, v in opts.items():
        kind = np.int32 if name == "top_k" else np.float32
        kw[name] = torch.from_numpy(np.ascontiguousarray(np.broadcast_to(np.asarray(v, dtype=kind), (len(x),)))).cuda()
    out = sample(t, torch.from_numpy(np.asarray(u, dtype=np.float32)).cuda(), **kw)
    host = t.double().cpu().numpy()
    u, kw = np.asarray(u, np.float32), {k: v.cpu().numpy() for k, v in kw.items()}
    want = [oq.sample_row(host[r], float(u[r]), float(kw["temperature"][r]) if "temperature" in kw else 1.0,
                          int(kw["top_k"][r]) if "top_k" in kw else 0, float(kw["top_p"][r]) if "top_p" in kw else 1.0,
                          float(kw["min_p"][r]) if "min_p" in kw else 0.0) for r in range(len(x))]
    return out.cpu().numpy(), np.array([w[0] for w in want]), np.array([w[1] for w in want])


def _check(got, want, margin):
    # weights are held to 2^-44 of the largest and 2^-46 of themselves: over V of them a border
    # moves by less than V * 2^-43 relative to the kept sum, which is at least the largest
    assert (margin > 1e-9).mean() > 0.99
    bad = (got != want) & (margin > 1e-9)
    assert not bad.any(), (np.flatnonzero(bad), got[bad], want[bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 64, 1000, 4099, 32000, 152064])
def test_sample(vocab, dtype):
    r = np.random.default_rng(vocab)
    rows = 60 if vocab < 10000 else 24
    x = r.standard_normal((rows, vocab)) * r.choice([0.5, 2.5, 6.0], (rows, 1))
    t = r.choice([0.0, 0.3, 0.7, 1.0, 1.6], rows)
    k = r.choice([0, 1, 2, 5, 50, 900, vocab, vocab + 5, -3], rows)
    p = r.choice([0.0, 0.01, 0.5, 0.9, 0.99, 1.0, 1.5], rows)
    m = r.choice([0.0, 0.0, 0.02, 0.3, 1.0], rows)
    _check(*_sample(x, r.random(rows), dtype, temperature=t, top_k=k, top_p=p, min_p=m))


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p", None])
def test_each_option_alone(name):
    r = np.random.default_rng(3)
    x = r.standard_normal((64, 5000)) * 3
    opts = {"temperature": r.uniform(0.1, 3, 64), "top_k": r.integers(1, 300, 64), "top_p": r.uniform(0.05, 0.999, 64),
            "min_p": r.uniform(0, 0.5, 64)}
    _check(*_sample(x, r.random(64), **({name: opts[name]} if name else {})))


@pytest.mark.parametrize("vocab", [10, 3000, 70000])
def test_ties(vocab):
    """Few distinct logits: what is cut falls inside a run of equal ones."""
    r = np.random.default_rng(vocab)
    x = r.integers(0, 3, (40, vocab)).astype(float)
    k = r.integers(1, vocab, 40)
    p = r.choice([0.3, 0.7, 1.0], 40)
    _check(*_sample(x, r.random(40), top_k=k, top_p=p))
    _check(*_sample(np.zeros((40, vocab)), r.random(40), top_k=k))
    _check(*_sample(np.zeros((40, vocab)), r.random(40), top_p=p * 0.99))
    got, want, _ = _sample(x, np.zeros(40), temperature=np.zeros(40))
    assert (got == want).all()


@pytest.mark.parametrize("vocab", [6, 9000])
@pytest.mark.parametrize("opts", [{}, {"top_k": 3}, {"top_p": 0.6}, {"min_p": 0.2}, {"top_k": 4, "top_p": 0.8}, {"temperature": 0.0}])
def test_odd_logits(vocab, opts):
    nan = np.nan
    head = [[-INF] * 6, [-INF, 2.0, -INF, 1.0, 2.0, 0.0], [nan, 1.0, nan, 2.0, -INF, 1.0], [nan] * 6,
            [INF, 0.0, INF, 1.0, -INF, INF], [-INF, -INF, -INF, -INF, 3.0, -INF], [1e38, -1e38, 3e38, 0.0, 3e38, -3e38],
            [-3e38, -3e38, -INF, -3.1e38, -3e38, nan], [0.0, -0.0, 0.0, -0.0, 1e-45, -1e-45], [INF] * 6]
    x = np.full((len(head), vocab), -INF)
    x[:, :6] = head
    if vocab > 6:
        x[::2, 6:] = np.nan
    for u in (0.0, 0.3, 0.9999999):
        got, want, _ = _sample(x, np.full(len(x), u), **opts)
        assert (got == want).all(), (u, got, want)


def test_uniform_outside_its_range():
    x = np.array([[0.0, 1.0, -INF]] * 4)
    got, want, _ = _sample(x, [-1.0, 1.0, 7.0, np.nan])
    assert got.tolist() == [0, 1, 1, 0]


def test_extreme_temperatures():
    r = np.random.default_rng(8)
    x = r.standard_normal((6, 3000))
    t = np.array([1e-40, 1e-3, 100.0, 1e30, INF, np.nan])
    got, want, margin = _sample(x, r.random(6), temperature=t)
    assert (got[margin > 1e-9] == want[margin > 1e-9]).all()
    _check(*_sample(x, r.random(6), temperature=np.full(6, 1e30), top_k=np.arange(1, 7) * 100, top_p=np.full(6, 0.5)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [333, 32000])
def test_strided_and_unaligned_rows(vocab, dtype):
    from tree_verification_attention_longspec_b200 import sample
    r = np.random.default_rng(vocab)
    wide = torch.from_numpy(r.standard_normal((9, vocab + 13)).astype(np.float32) * 3).cuda()
    wide = wide.to(torch.bfloat16) if dtype == "bf16" else wide
    u = torch.from_numpy(r.random(9).astype(np.float32)).cuda()
    part = wide[:, 5:5 + vocab]
    a, b = sample(part, u, top_p=0.9), sample(part.contiguous(), u, top_p=0.9)
    assert torch.equal(a, b)
    # every second row, a number for all rows
    a, b = sample(wide[::2, :vocab], u[::2].contiguous(), top_k=7), sample(wide[::2, :vocab].contiguous(), u[::2].contiguous(), top_k=7)
    assert torch.equal(a, b)


def test_large_vocabulary():
    r = np.random.default_rng(1)
    x = r.standard_normal((3, 1 << 20)).astype(np.float32) * 2
    _check(*_sample(x, r.random(3), "f32", temperature=np.ones(3), top_k=[0, 100000, 0], top_p=[1.0, 0.9, 0.7]))
    _check(*_sample(x, r.random(3), "bf16", temperature=np.ones(3), top_k=[0, 100000, 0], top_p=[1.0, 0.9, 0.7]))


def test_frequencies_follow_the_distribution():
    """Evenly spaced u: counts equal the kept weights' shares within one."""
    x = np.array([[1.0, 0.0, 2.0, -1.0, 0.5]])
    n = 1000
    u = (np.arange(n) + 0.5) / n
    got, _, _ = _sample(np.repeat(x, n, 0), u, top_k=4)
    w = np.exp(x[0] - 2.0)
    w[3] = 0
    assert np.abs(np.bincount(got, minlength=5) - n * w / w.sum()).max() <= 1.0


def test_no_rows():
    from tree_verification_attention_longspec_b200 import sample
    assert sample(torch.empty(0, 100, device="cuda"), torch.empty(0, device="cuda")).shape == (0,)


def _trees(sizes, vocab, seed, hit=0.8):
    r = np.random.default_rng(seed)
    n = sum(sizes)
    x = r.standard_normal((n, vocab)) * 2
    peak = r.integers(0, vocab, n)
    x[np.arange(n), peak] = 12.0
    parent, draft, at = [], np.zeros(n, dtype=np.int32), 0
    for size in sizes:
        i = np.arange(size)
        p = np.maximum(0, i - 3) + (r.random(size) * np.maximum(1, i - np.maximum(0, i - 3))).astype(int)
        p[0:1] = -1
        for j in range(1, size):
            draft[at + j] = peak[at + p[j]] if r.random() < hit else r.integers(0, vocab)
        parent.append(p)
        at += size
    return x, np.concatenate(parent).astype(np.int32), draft, r.random(n).astype(np.float32)


@pytest.mark.parametrize("sizes,uniform_size", [((1,), True), ((128,), True), ((20,) * 5, True), ((7, 0, 128, 1, 33), False)])
@pytest.mark.parametrize("vocab,dtype", [(100, "f32"), (20000, "bf16")])
def test_tree_accept(sizes, uniform_size, vocab, dtype):
    from tree_verification_attention_longspec_b200 import tree_accept_sample
    x, parent, draft, u = _trees(sizes, vocab, len(sizes))
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    t = t.to(torch.bfloat16) if dtype == "bf16" else t
    T = max(sizes)
    base = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    cu = None if uniform_size else torch.from_numpy(base).cuda()
    token, length, path, after = (y.cpu().numpy() for y in tree_accept_sample(
        t, torch.from_numpy(u).cuda(), torch.from_numpy(draft).cuda(), torch.from_numpy(parent).cuda(), T, cu_tree=cu,
        temperature=0.9, top_p=0.95))
    host = t.double().cpu().numpy()
    want = [oq.sample_row(host[i], float(u[i]), float(np.float32(0.9)), 0, float(np.float32(0.95))) for i in range(len(u))]
    assert all(g == w or m < 1e-9 for g, (w, m) in zip(token, want))
    for b in range(len(sizes)):
        s, e = base[b], base[b + 1]
        n, p, nxt = oq.walk(token[s:e], draft[s:e], parent[s:e])
        assert (length[b], after[b]) == (n, nxt)
        assert path[b].tolist() == p + [-1] * (T - len(p))


def test_tree_accept_at_temperature_zero_is_the_greedy_call():
    from tree_verification_attention_longspec_b200 import binding, tree_accept_sample
    x, parent, draft, u = _trees((40, 40), 3333, 4)
    t = torch.from_numpy(x.astype(np.float32)).cuda()
    tok, par = torch.from_numpy(draft).cuda(), torch.from_numpy(parent).cuda()
    _, length, path, after = tree_accept_sample(t, torch.from_numpy(u).cuda(), tok, par, 40, temperature=0.0)
    dims = binding.AcceptDims(2, 40, 3333, binding.LS_DTYPE_F32)
    wsb = binding.accept_workspace_size(dims, 80)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    l2, p2, n2 = (torch.full(s, -1, dtype=torch.int32, device="cuda") for s in ((2,), (2, 40), (2,)))
    assert binding.call_accept_raw(t.data_ptr(), tok.data_ptr(), par.data_ptr(), None, 80, l2.data_ptr(), p2.data_ptr(),
                                   n2.data_ptr(), dims, ws.data_ptr(), wsb, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(length, l2) and torch.equal(path, p2) and torch.equal(after, n2)


def test_tree_accept_bad_trees():
    from tree_verification_attention_longspec_b200 import tree_accept_sample
    x, parent, draft, u = _trees((6, 6, 6), 50, 5)
    parent[1], parent[6] = 1, 0
    args = [torch.from_numpy(a).cuda() for a in (x.astype(np.float32), u, draft, parent)]
    _, length, path, after = tree_accept_sample(*args, 6)
    assert length.tolist()[:2] == [-1, -1] and after.tolist()[:2] == [-1, -1] and (path[:2] == -1).all()
    assert length[2] >= 0
    cu = torch.tensor([0, 6, 30, 18], dtype=torch.int32, device="cuda")
    _, length, _, after = tree_accept_sample(*args, 6, cu_tree=cu)
    assert length.tolist()[1:] == [-1, -1] and after.tolist()[1:] == [-1, -1]


def test_streams_and_graphs():
    from tree_verification_attention_longspec_b200 import sample, tree_accept_sample
    x, parent, draft, u = _trees((30, 30), 9000, 6)
    args = [torch.from_numpy(a).cuda() for a in (x.astype(np.float32), u, draft, parent)]
    knobs = dict(temperature=torch.full((60,), 0.8, device="cuda"), top_k=torch.full((60,), 40, dtype=torch.int32, device="cuda"))
    want = tree_accept_sample(*args, 30, **knobs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = tree_accept_sample(*args, 30, **knobs)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tree_accept_sample(*args, 30, **knobs)
        alone = sample(args[0], args[1], **knobs)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, again, got))
    assert torch.equal(alone, want[0])
