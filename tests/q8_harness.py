"""Builds cases of the 8-bit cache for the GPU tests: seeded host arrays, the oracle's
answer, and the package's."""
from __future__ import annotations

import numpy as np
import torch

from oracle import q8 as oq
from oracle import tree_positions as tp

EXP_ERR = 2.0 ** -22      # a hardware 2^x: relative error 2^-22.5, and the argument's rounding
F16_HALF = 2.0 ** -11     # half a step of f16
BF16_HALF = 2.0 ** -8     # half a step of bf16
F32_HALF = 2.0 ** -24


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """A cache of random codes, trees and queries; garbage wherever nothing may be read."""

    def __init__(self, lens, heads, kv_heads, dim, nodes, page, block, *, sizes=None, seed=0, peak=2.0, spare=2,
                 scale_spread=0.0, values=1.0):
        r = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.d, self.T = list(lens), heads, kv_heads, dim, nodes
        self.page, self.block, self.B = page, block, len(lens)
        self.sizes = [nodes] * self.B if sizes is None else list(sizes)
        self.ragged = sizes is not None
        need = [(n + page - 1) // page for n in lens]
        self.num_pages = sum(need) + spare
        order = r.permutation(self.num_pages)
        # unused table entries name pages that do not exist
        self.table = np.where(np.arange(max(1, max(need)) + 1)[None] >= 0,
                              r.choice([-7, self.num_pages, 2 ** 31 - 1], (self.B, max(1, max(need)) + 1)), 0).astype(np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.num_pages, page, kv_heads, dim)
        self.codes, self.scales = {}, {}
        for w in "kv":
            c = oq.e4m3_encode(r.standard_normal(shape) * 100.0)
            s = (0.01 * np.exp(scale_spread * r.standard_normal((self.num_pages, page // block, kv_heads)))).astype(np.float32)
            if w == "v":
                s *= np.float32(values)
            used = np.zeros((self.num_pages, page), dtype=bool)
            for b, n in enumerate(self.lens):
                for i in range(need[b]):
                    used[self.table[b, i], :min(page, n - i * page)] = True
            c[~used] = 0x7F                                       # NaN codes behind every sequence
            s[~used.reshape(self.num_pages, -1, block).any(-1)] = np.nan
            self.codes[w], self.scales[w] = c, s
        n = sum(self.sizes)
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        self.cu_tree = np.concatenate([[0], np.cumsum(self.sizes)]).astype(np.int32)
        par = []
        for size in self.sizes:
            i = np.arange(size)
            p = np.maximum(0, i - 4) + (r.random(size) * np.maximum(1, i - np.maximum(0, i - 4))).astype(int)
            p[0:1] = -1
            par.append(p)
        self.parent = np.concatenate(par).astype(np.int32) if par else np.zeros(0, np.int32)
        self.q = bf16(peak * r.standard_normal((n, heads, dim)))
        self.k_tree = bf16(r.standard_normal((n, kv_heads, dim)))
        self.v_tree = bf16(values * r.standard_normal((n, kv_heads, dim)))

    def device(self, dev="cuda"):
        from tree_verification_attention_longspec_b200 import KVCacheQ8

        def put(a):
            return torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        cache = KVCacheQ8(put(self.codes["k"]), put(self.codes["v"]), put(self.scales["k"]), put(self.scales["v"]),
                          put(self.table))
        return cache, self.q.to(dev), self.k_tree.to(dev), self.v_tree.to(dev), put(self.parent), put(self.cu)

    def opts(self, window=0, theta=0.0, dev="cuda", wait_ns=0):
        from tree_verification_attention_longspec_b200.binding import TreeOpts
        self.cu_tree_dev = torch.from_numpy(self.cu_tree).to(dev)
        return TreeOpts(cu_tree=self.cu_tree_dev.data_ptr() if self.ragged else None,
                        total_nodes=int(self.cu_tree[-1]) if self.ragged else 0, window=window, rope_theta=theta,
                        wait_limit_ns=wait_ns)

    def reference(self, with_tree=True, window=0, theta=0.0, scale=None):
        """(out, lse, out tolerance, lse tolerance), rows as the tensors'."""
        scale = self.d ** -0.5 if scale is None else scale
        q, kt, vt = f64(self.q), f64(self.k_tree), f64(self.v_tree)
        if theta:
            pos = tp.tree_positions(self.parent, self.cu, self.cu_tree)
            q = tp.round_to_bf16(tp.rope_rotate(q, pos, theta))
            kt = tp.round_to_bf16(tp.rope_rotate(kt, pos, theta))
        parts = []
        for b, n in enumerate(self.lens):
            s, e = self.cu_tree[b], self.cu_tree[b + 1]
            k = oq.gather(self.codes["k"], self.scales["k"], self.table[b], n, self.page, self.block)
            v = oq.gather(self.codes["v"], self.scales["v"], self.table[b], n, self.page, self.block)
            see = np.ones((e - s, n), dtype=bool)
            par = self.parent[s:e]
            if window:
                depth = tp.tree_depth_walk(par)
                see = np.arange(n)[None] > n + depth[:, None] - window
            if with_tree:
                k, v = np.concatenate([k, kt[s:e]]), np.concatenate([v, vt[s:e]])
                see = np.concatenate([see, oq.ancestors(par)], 1)
            parts.append(oq.attention(q[s:e], k, v, see, scale))
        out, lse, spread, reach = (np.concatenate(x) for x in zip(*parts))
        # A score's error: d products summed in fp32 (each addition off by at most 2^-23 of the
        # sum of magnitudes, the tensor core truncating), then the score and its exponent
        # rounded a few times; a weight's: that, the exponential's, and half a step of f16.
        score = (self.d + 8) * 2.0 ** -23 * (reach + 1.0)
        weight = (np.exp(score) - 1 + EXP_ERR + F16_HALF)[..., None]
        # out = sum w v / sum w: both sums move by `weight`, relative to sum w |v|; then bf16
        tol = BF16_HALF * np.abs(out) + 2.02 * weight * spread + 1e-30
        # the sums stay in fp32: score errors, exponentials, and the sums of n terms (in order
        # within a lane, at most n / 16 of them, then a few merges)
        n = max(self.lens) + self.T
        with np.errstate(invalid="ignore"):
            lse_tol = score + EXP_ERR + (n / 16 + 64) * F32_HALF + 4 * F32_HALF * np.abs(np.where(np.isinf(lse), 0, lse))
        return out, lse, tol, lse_tol


def compare(got_out, got_lse, ref):
    out, lse, tol, lse_tol = ref
    o, l = f64(got_out), f64(got_lse)
    assert np.isfinite(o).all()
    off = np.abs(o - out) / tol
    assert off.max(initial=0.0) <= 1.0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    empty = np.isinf(lse)
    assert (np.isneginf(l) == empty).all()
    off = np.abs(np.where(empty, 0, l) - np.where(empty, 0, lse)) / lse_tol
    assert off.max(initial=0.0) <= 1.0, (off.max(), np.unravel_index(off.argmax(), off.shape))
