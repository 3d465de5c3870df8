"""The greedy acceptance call and the sampled one at temperature 0 are one walk."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import q8 as oq

pytestmark = pytest.mark.gpu


def _trees(sizes, vocab, seed):
    """Trees whose siblings often hold the same draft token, most of them the parent's argmax."""
    r = np.random.default_rng(seed)
    n = sum(sizes)
    x = r.standard_normal((n, vocab)).astype(np.float32)
    best, parent, draft, at = x.argmax(1), [], np.zeros(n, dtype=np.int32), 0
    for size in sizes:
        i = np.arange(size)
        p = np.maximum(0, i - 1 - r.integers(0, 5, size))
        p[:1] = -1
        for j in range(1, size):
            draft[at + j] = best[at + p[j]] if r.random() < 0.8 else r.integers(0, vocab)
        parent.append(p)
        at += size
    return x, draft, np.concatenate(parent).astype(np.int32)


@pytest.mark.parametrize("sizes", [(1,), (128, 128), (5, 0, 128, 1, 64, 2), (17,) * 40])
@pytest.mark.parametrize("vocab,dtype", [(3, torch.float32), (5000, torch.bfloat16)])
@pytest.mark.parametrize("broken", [False, True])
def test_same_paths(sizes, vocab, dtype, broken):
    from tree_verification_attention_longspec_b200 import binding, tree_accept_sample
    x, draft, parent = _trees(sizes, vocab, len(sizes) + vocab)
    base = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    B, T, N = len(sizes), max(sizes), int(base[-1])
    if broken:
        parent[base[B // 2]:base[B // 2] + 1] = 0  # a root with a parent
    lg = torch.from_numpy(x).cuda().to(dtype)
    tok, par, cu = (torch.from_numpy(a).cuda() for a in (draft, parent, base))
    node, length, path, after = tree_accept_sample(lg, torch.zeros(N, device="cuda"), tok, par, T, cu_tree=cu, temperature=0.0)
    dims = binding.AcceptDims(B, T, vocab, binding.LS_DTYPE_F32 if dtype == torch.float32 else binding.LS_DTYPE_BF16)
    wsb = binding.accept_workspace_size(dims, N)
    ws = torch.empty(wsb, dtype=torch.uint8, device="cuda")
    l2, p2, n2 = (torch.full(s, -1, dtype=torch.int32, device="cuda") for s in ((B,), (B, T), (B,)))
    assert binding.call_accept_raw(lg.data_ptr(), tok.data_ptr(), par.data_ptr(), cu.data_ptr(), N, l2.data_ptr(),
                                   p2.data_ptr(), n2.data_ptr(), dims, ws.data_ptr(), wsb,
                                   torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(length, l2) and torch.equal(path, p2) and torch.equal(after, n2)
    node = node.cpu().numpy()
    for b in range(B):
        s, e = base[b], base[b + 1]
        n, p, nxt = oq.walk(node[s:e], draft[s:e], parent[s:e])
        assert (int(length[b]), int(after[b]), path[b].tolist()) == (n, nxt, p + [-1] * (T - len(p)))
