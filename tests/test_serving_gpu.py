"""The serving operators as they are used together: prompts appended, trees verified over
the 8-bit cache, accepted by sampling and committed, step after step."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from tests.q8_harness import Case, bf16, compare, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes,heads,kv,d", [(1, 8, 2, 128), (6, 8, 4, 64), (24, 16, 2, 128)])
def test_steps(nodes, heads, kv, d):
    from tree_verification_attention_longspec_b200 import KVCacheQ8, VerifyAttnQ8, tree_accept_sample
    r = np.random.default_rng(nodes)
    B, page, vocab, most = 3, 16, 500, 256
    table = torch.from_numpy(r.permutation(B * 16).reshape(B, 16).astype(np.int32)).cuda()
    cache = KVCacheQ8.empty(B * 16, page, kv, d, table)
    lens = [40, 0, 17]
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu_new = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)).cuda()
    prompt = [bf16(r.standard_normal((sum(lens), kv, d))) for _ in range(2)]
    cu = cache.append(prompt[0].cuda(), prompt[1].cuda(), cu, cu_new, max(lens))
    call = VerifyAttnQ8(B, heads, kv, d, nodes, max_prefix_len=most)
    accepted = 0
    for step in range(6):
        case = Case(lens, heads, kv, d, nodes, page, page, seed=100 + step)
        case.table = table.cpu().numpy()
        case.codes = {"k": cache.k_pages.view(torch.uint8).cpu().numpy(), "v": cache.v_pages.view(torch.uint8).cpu().numpy()}
        case.scales = {"k": cache.k_scale.cpu().numpy(), "v": cache.v_scale.cpu().numpy()}
        case.num_pages = B * 16
        q, kt, vt, par = (t.cuda() for t in (case.q, case.k_tree, case.v_tree, torch.from_numpy(case.parent)))
        out, lse = call(q, cache, kt, vt, par, cu)
        assert call.check() == 0
        compare(out, lse, case.reference())
        x = r.standard_normal((B * nodes, vocab)) * 2
        likely = r.integers(0, vocab, B * nodes)
        x[np.arange(B * nodes), likely] = 11.0
        base = np.repeat(np.arange(B) * nodes, nodes)
        draft = likely[base + np.maximum(case.parent, 0)].astype(np.int32)
        u = r.random(B * nodes).astype(np.float32)
        token, length, path, after = tree_accept_sample(
            torch.from_numpy(x.astype(np.float32)).cuda(), torch.from_numpy(u).cuda(), torch.from_numpy(draft).cuda(), par, nodes, top_k=50)
        cu = cache.commit(kt, vt, cu, length, path)
        n = length.cpu().numpy()
        lens = [a + int(b) + 1 for a, b in zip(lens, n)]
        accepted += int(n.sum())
        assert cu.cpu().tolist() == [0] + list(np.cumsum(lens))
        # the committed rows are the path's, to the cache's precision: 2^-4 of a value, and
        # half of e4m3's smallest step, 2^-10, of the block's scale
        for b in range(B):
            got = oq.gather(cache.k_pages.view(torch.uint8).cpu().numpy(), cache.k_scale.cpu().numpy(),
                            table.cpu().numpy()[b], lens[b], page, page)[-(int(n[b]) + 1):]
            want = f64(case.k_tree)[b * nodes + path[b, :int(n[b]) + 1].cpu().numpy()]
            unit = cache.k_scale.max().item()
            assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * unit).all()
    assert nodes == 1 or accepted > 0
