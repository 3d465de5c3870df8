"""Writing the 8-bit paged cache: codes, scales and lengths must equal the oracle's."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from tests.q8_harness import bf16, compare, f64

pytestmark = pytest.mark.gpu


class Pool:
    def __init__(self, lens, room, kv, d, page, block, seed=0):
        r = np.random.default_rng(seed)
        need = [(n + page - 1) // page for n in room]
        self.page, self.block, self.lens = page, block, list(lens)
        pages = sum(need) + 3
        order = r.permutation(pages)
        self.table = np.full((len(lens), max(1, max(need))), -3, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.codes = {w: r.integers(0, 127, (pages, page, kv, d)).astype(np.uint8) for w in "kv"}
        self.scales = {w: 2.0 ** r.integers(-9, -3, (pages, page // block, kv)).astype(np.float32) for w in "kv"}

    def device(self):
        from tree_verification_attention_longspec_b200 import KVCacheQ8

        def put(a):
            return torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.cache = KVCacheQ8(put(self.codes["k"]), put(self.codes["v"]), put(self.scales["k"]),
                               put(self.scales["v"]), put(self.table))
        self.cu = put(np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32))
        return self.cache

    def expect(self, rows, cu_after, lens_after):
        """rows[w][b]: appended rows. Compares the device's cache, and keeps it."""
        for w, codes, scale in (("k", self.cache.k_pages, self.cache.k_scale), ("v", self.cache.v_pages, self.cache.v_scale)):
            want, want_scale = oq.append(self.codes[w], self.scales[w], self.table, self.lens, rows[w], self.page, self.block)
            got = codes.view(torch.uint8).cpu().numpy()
            assert np.array_equal(scale.cpu().numpy().astype(np.float64), want_scale)
            # -0 and 0 are one value; the codes' values are compared (NaN with NaN)
            assert np.array_equal(oq.TABLE[got], oq.TABLE[want], equal_nan=True)
            self.codes[w], self.scales[w] = got, scale.cpu().numpy()
        assert cu_after.cpu().tolist() == [0] + list(np.cumsum(lens_after))
        self.lens, self.cu = list(lens_after), cu_after


def _split(x, cu):
    return [list(x[cu[b]:cu[b + 1]]) for b in range(len(cu) - 1)]


@pytest.mark.parametrize("lens,new,kv,d,page,block", [
    ((0,), (1,), 1, 64, 16, 16),
    ((5, 0, 31), (1, 1, 1), 2, 128, 32, 16),
    ((0, 15, 16, 17), (0, 3, 40, 16), 3, 64, 16, 16),
    ((100, 0), (29, 300), 2, 128, 128, 128),
    ((63, 64, 65), (129, 1, 64), 8, 128, 64, 64),
    ((7, 250), (505, 6), 1, 64, 384, 128),
    ((33,), (260,), 4, 128, 256, 32),
])
def test_append(lens, new, kv, d, page, block):
    r = np.random.default_rng(len(lens) + d)
    pool = Pool(lens, [a + b for a, b in zip(lens, new)], kv, d, page, block)
    cache = pool.device()
    cu_new = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    size = np.exp(2 * r.standard_normal((sum(new), kv, 1)))
    k, v = bf16(size * r.standard_normal((sum(new), kv, d))), bf16(r.standard_normal((sum(new), kv, d)) / 64)
    cu = cache.append(k.cuda(), v.cuda(), pool.cu, torch.from_numpy(cu_new).cuda(), max(new))
    pool.expect({"k": _split(f64(k), cu_new), "v": _split(f64(v), cu_new)}, cu, [a + b for a, b in zip(lens, new)])


def test_append_token_by_token_then_one_more_chunk():
    """A block that grows: its scale is raised as larger tokens come, never lowered."""
    r = np.random.default_rng(5)
    pool = Pool((0, 9), (80, 80), 2, 64, 32, 32)
    cache = pool.device()
    for step in range(40):
        x = r.standard_normal((2, 2, 64)) * 2.0 ** (step % 7 - 3)
        k, v = bf16(x), bf16(-x / 3)
        cu_new = np.array([0, 1, 2], dtype=np.int32)
        cu = cache.append(k.cuda(), v.cuda(), pool.cu, torch.from_numpy(cu_new).cuda(), 1)
        pool.expect({"k": _split(f64(k), cu_new), "v": _split(f64(v), cu_new)}, cu, [n + 1 for n in pool.lens])


@pytest.mark.parametrize("values", ["zero", "tiny", "huge", "nan", "inf", "border"])
def test_append_odd_values(values):
    x = np.random.default_rng(2).standard_normal((20, 1, 64)).astype(np.float64)
    if values == "zero":
        x[:] = 0.0
    elif values == "tiny":
        x *= 2.0 ** -125
    elif values == "huge":
        x *= 2.0 ** 100
    elif values == "nan":
        x[3, 0, 5] = x[17, 0, 0] = np.nan
    elif values == "inf":
        x[4, 0, 1], x[18, 0, 2] = np.inf, -np.inf
    else:  # the largest of a scale, the next bf16 above it, and ties between two codes
        x[:10] = 1.0
        x[0, 0, 0] = 448.0
        x[16, 0, 0] = 450.0
        x[1, 0, :8] = [17.0, 19.0, 21.0, 23.0, -17.0, -19.0, 2.0 ** -10, 3 * 2.0 ** -10]
    pool = Pool((0,), (20,), 1, 64, 16, 16)
    cache = pool.device()
    k, cu_new = bf16(x), np.array([0, 20], dtype=np.int32)
    cu = cache.append(k.cuda(), k.cuda(), pool.cu, torch.from_numpy(cu_new).cuda(), 20)
    rows = _split(f64(k), cu_new)
    pool.expect({"k": rows, "v": rows}, cu, [20])


def test_append_drops_what_has_no_room():
    """Rows past max_new, past the table, and of pages that are not the cache's."""
    pool = Pool((20, 3, 0, 30), (32, 32, 32, 32), 2, 64, 16, 16)
    pool.table = pool.table[:, :2]
    pool.table[1] = [2 ** 31 - 1, -9]
    cache = pool.device()
    new = (30, 5, 9, 1)
    cu_new = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    x = bf16(np.random.default_rng(3).standard_normal((45, 2, 64)))
    cu = cache.append(x.cuda(), x.cuda(), pool.cu, torch.from_numpy(cu_new).cuda(), 8)
    rows = [z[:8] for z in _split(f64(x), cu_new)]
    pool.expect({"k": rows, "v": rows}, cu, [28, 8, 8, 31])


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("d,page,block", [(64, 16, 16), (128, 128, 64)])
def test_commit(ragged, d, page, block):
    r = np.random.default_rng(d)
    lens, T = (0, 30, 63, 5), 12
    sizes = (12, 3, 0, 7) if ragged else (T,) * 4
    base = np.concatenate([[0], np.cumsum(sizes)])
    length = np.array([4, 0, -1, 2], dtype=np.int32)
    path = np.full((4, T), -1, dtype=np.int32)
    path[0, :5], path[1, :1], path[3, :3] = [0, 2, 3, 9, 11], [0], [0, 5, 6]
    pool = Pool(lens, [n + T for n in lens], 2, d, page, block)
    cache = pool.device()
    k, v = (bf16(r.standard_normal((base[-1], 2, d))) for _ in range(2))
    cu_tree = torch.from_numpy(base.astype(np.int32)).cuda() if ragged else None
    cu = cache.commit(k.cuda(), v.cuda(), pool.cu, torch.from_numpy(length).cuda(), torch.from_numpy(path).cuda(), cu_tree=cu_tree)
    rows = {w: [[f64(x)[base[b] + i] for i in path[b, :length[b] + 1]] for b in range(4)] for w, x in (("k", k), ("v", v))}
    pool.expect(rows, cu, [n + int(a) + 1 for n, a in zip(lens, length)])


def test_commit_skips_path_entries_that_are_no_node():
    pool = Pool((3,), (20,), 1, 64, 16, 16)
    cache = pool.device()
    path = np.array([[0, 7, -4, 2]], dtype=np.int32)
    k = bf16(np.random.default_rng(1).standard_normal((4, 1, 64)))
    cu = cache.commit(k.cuda(), k.cuda(), pool.cu, torch.tensor([3], dtype=torch.int32, device="cuda"), torch.from_numpy(path).cuda())
    x = f64(k)
    pool.expect({"k": [[x[0], None, None, x[2]]], "v": [[x[0], None, None, x[2]]]}, cu, [7])


def test_append_in_a_graph_and_on_a_stream():
    pool = Pool((10,), (40,), 2, 128, 16, 16)
    cache = pool.device()
    x = bf16(np.random.default_rng(4).standard_normal((13, 2, 128))).cuda()
    cu_new, after = torch.tensor([0, 13], dtype=torch.int32, device="cuda"), torch.empty_like(pool.cu)
    cache.append(x, x, pool.cu, cu_new, 13, cu_seqlens_out=after)
    want = [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_scale, after)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(x, x, pool.cu, cu_new, 13, cu_seqlens_out=after)
    after.zero_()
    graph.replay()  # the same rows at the same place: nothing changes
    torch.cuda.synchronize()
    for a, b in zip(want, (cache.k_pages.view(torch.uint8), cache.v_scale, after)):
        assert torch.equal(a, b)
