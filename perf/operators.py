"""The serving operators around tree verification over an 8-bit paged cache, as cases.

Four operators of one verification step:

- "attend": tree-verification attention (or prefix-only attention) whose cached keys and
  values are held in 8 bits (e4m3) with one scale for each block of tokens and kv head;
- "append": new keys and values written into that cache, quantised, with the scale of a
  block that already holds tokens raised where the new ones need it;
- "sample": one token for each row of logits, by temperature, top-k, top-p and min-p from
  a given uniform number;
- "accept": every node of the draft trees sampled that way and the walk from each root.

`run` computes them in elementary torch operations, or, where `own` is set, makes the calls
that a program makes of the package.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 64  # exponents of the block scales that the append writes


def ints(text):
    return [int(x) for x in str(text).split(",")]


def listed():
    return [
        # one new token of a long document: the step of a decoder without a draft
        dict(name="attend_token_L64k", op="attend", heads=28, kv_heads=4, dim=128, nodes=1, lens="65536", page=64,
             block=64, tree=True, peak=2.0),
        # the draft model's token of every running sequence over the target's cache
        dict(name="attend_prefix_b8", op="attend", heads=32, kv_heads=8, dim=128, nodes=1,
             lens="4099,32768,20011,9001,15000,27777,6400,12345", page=32, block=32, tree=False, peak=2.0),
        # the smallest verification: a short prompt, a small tree, one kv head
        dict(name="attend_tree16_L1k", op="attend", heads=4, kv_heads=1, dim=64, nodes=16, lens="1024", page=16,
             block=16, tree=True, peak=1.0),
        # a tree of four candidates for several sequences
        dict(name="attend_tree4_b4", op="attend", heads=32, kv_heads=8, dim=128, nodes=4, lens="16384,777,9000,4097",
             page=128, block=128, tree=True, peak=2.0),
        # the ordinary verification of a 64-node tree
        dict(name="attend_tree64_L16k", op="attend", heads=32, kv_heads=8, dim=128, nodes=64, lens="16384", page=64,
             block=32, tree=True, peak=2.0),
        # the same over a long document
        dict(name="attend_tree64_L64k", op="attend", heads=28, kv_heads=4, dim=128, nodes=64, lens="65536", page=256,
             block=64, tree=True, peak=2.0),
        # a batch of prompts, two of them continuing what is cached
        dict(name="append_prompts", op="append", kv_heads=8, dim=128, lens="0,1000,0,17", new="8192,4096,3001,1095",
             page=64, block=32, path=False),
        # the accepted paths of a verification step, committed to the cache
        dict(name="append_paths", op="append", kv_heads=8, dim=128, lens="4099,32768,20011,9001,15000,27777,6400,12345",
             new="3,1,5,0,2,4,7,1", page=64, block=64, path=True),
        # the tokens of a few sequences, small vocabulary
        dict(name="sample_8x32000", op="sample", rows=8, vocab=32000, dtype="f32", how="mixed"),
        # a large batch, nucleus sampling alone
        dict(name="sample_256x128256", op="sample", rows=256, vocab=128256, dtype="bf16", how="topp"),
        # one verified tree
        dict(name="accept_64x152064", op="accept", trees="64", vocab=152064, dtype="bf16", how="mixed"),
        # trees of several sequences, of their own sizes
        dict(name="accept_534x128256", op="accept", trees="16,128,77,40,101,31,64,77", vocab=128256, dtype="bf16",
             how="mixed"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "sample", "accept"])
    if op == "attend":
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8])
        nodes = _log(rng, 1, 128)
        batch = _log(rng, 1, 8)
        page = rng.choice([16, 32, 64, 128, 256])
        block = rng.choice([b for b in (16, 32, 64, 128) if page % b == 0])
        tree = rng.random() < 0.7
        most = min(65536, int(64 * 28 * 65536 * 128 / (nodes * kv * group * dim * batch)))
        lens = [_log(rng, 1, max(2, most)) for _ in range(batch)]
        if tree and batch > 1 and rng.random() < 0.3:
            lens[rng.randrange(batch)] = 0
        return dict(op=op, heads=kv * group, kv_heads=kv, dim=dim, nodes=nodes, lens=",".join(map(str, lens)),
                    page=page, block=block, tree=tree, peak=rng.choice([0.5, 1.0, 2.0, 3.0]))
    if op == "append":
        batch = _log(rng, 1, 32)
        page = rng.choice([16, 32, 64, 128, 256])
        path = rng.random() < 0.5
        most = max(2, 16384 // batch)
        new = [rng.randrange(0, 17) if path else _log(rng, 1, most) for _ in range(batch)]
        new[0] = max(1, new[0])
        return dict(op=op, kv_heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128]),
                    lens=",".join(str(rng.choice([0, _log(rng, 1, 8192)])) for _ in range(batch)),
                    new=",".join(map(str, new)),
                    page=page, block=rng.choice([b for b in (16, 32, 64, 128) if page % b == 0]), path=path)
    vocab = _log(rng, 1000, 152064)
    dtype = rng.choice(["bf16", "f32"])
    how = rng.choice(["mixed", "mixed", "topp", "topk", "plain"])
    rows = _log(rng, 1, max(1, min(534, 534 * 128256 // vocab // (2 if dtype == "f32" else 1))))
    if op == "sample":
        return dict(op=op, rows=rows, vocab=vocab, dtype=dtype, how=how)
    trees = []
    while len(trees) < 8 and sum(trees) < rows:
        trees.append(min(rng.randrange(1, 129), rows - sum(trees)))
    return dict(op=op, trees=",".join(map(str, trees)), vocab=vocab, dtype=dtype, how=how)


# ------------------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _parents(sizes, seed):
    """Local parents of packed trees: -1 for a root, else one of the eight nodes before."""
    r = np.random.default_rng(seed + 1)
    out = []
    for n in sizes:
        i = np.arange(n)
        lo = np.maximum(0, i - 8)
        p = lo + (r.random(n) * np.maximum(1, i - lo)).astype(np.int64)
        p[0:1] = -1
        out.append(p)
    return torch.from_numpy(np.concatenate(out).astype(np.int32)).to(DEV)


def _cu(sizes):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEV)


def _table(lens, page, seed, spare=0):
    """A page table of pages in random order, and the number of pages."""
    need = [max(1, (n + page - 1) // page) for n in lens]
    total = sum(need) + spare
    order = np.random.default_rng(seed + 2).permutation(total)[:sum(need)]
    table = np.zeros((len(lens), max(need)), dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).to(DEV), total


def _cache(pages, page, block, kv, dim, g, power_of_two):
    """Cached keys or values: normal values, quantised by block and head."""
    x = torch.randn(pages, page // block, block, kv, dim, generator=g, device=DEV)
    x *= 0.5 + torch.rand(pages, page // block, 1, kv, 1, generator=g, device=DEV)
    amax = x.abs().amax(dim=(2, 4))
    scale = amax / E4M3_MAX
    if power_of_two:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    codes = (x / scale[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes.view(pages, page, kv, dim), scale.contiguous()


def _sampling(rows, how, g):
    u = torch.rand(rows, generator=g, device=DEV)
    pick = torch.rand(rows, 4, generator=g, device=DEV)
    temperature = 0.6 + 0.7 * pick[:, 0]
    top_k = torch.zeros(rows, dtype=torch.int32, device=DEV)
    top_p = torch.ones(rows, device=DEV)
    min_p = torch.zeros(rows, device=DEV)
    if how == "topp":
        top_p = 0.8 + 0.19 * pick[:, 1]
    elif how == "topk":
        top_k = (1 + 99 * pick[:, 1]).to(torch.int32)
    elif how == "mixed":
        # what the requests of one batch ask for: greedy rows, top-k, top-p, min-p and pairs of them
        temperature = torch.where(pick[:, 0] < 0.1, torch.zeros_like(temperature), temperature)
        top_k = torch.where(pick[:, 1] < 0.4, (1 + 200 * pick[:, 1]).to(torch.int32), top_k)
        top_p = torch.where(pick[:, 2] < 0.5, 0.7 + 0.5 * pick[:, 2], top_p)
        min_p = torch.where(pick[:, 3] < 0.3, 0.1 * pick[:, 3], min_p)
    return dict(uniform=u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)


def _logits(rows, vocab, dtype, g):
    x = torch.randn(rows, vocab, generator=g, device=DEV)
    x *= 2.5
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "attend":
        lens = ints(case["lens"])
        batch, n, d, kv, h = len(lens), case["nodes"], case["dim"], case["kv_heads"], case["heads"]
        s["table"], pages = _table(lens, case["page"], seed)
        s["k"], s["k_scale"] = _cache(pages, case["page"], case["block"], kv, d, g, False)
        s["v"], s["v_scale"] = _cache(pages, case["page"], case["block"], kv, d, g, False)
        s["q"] = (torch.randn(batch * n, h, d, generator=g, device=DEV) * case["peak"]).to(torch.bfloat16)
        s["cu"], s["max_len"], s["batch"] = _cu(lens), max(lens), batch
        if case["tree"]:
            s["k_tree"] = torch.randn(batch * n, kv, d, generator=g, device=DEV).to(torch.bfloat16)
            s["v_tree"] = torch.randn(batch * n, kv, d, generator=g, device=DEV).to(torch.bfloat16)
            s["parent"] = _parents([n] * batch, seed)
        if own:
            from tree_verification_attention_longspec_b200 import CrossAttnQ8, KVCacheQ8, VerifyAttnQ8
            s["cache"] = KVCacheQ8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
            make = VerifyAttnQ8 if case["tree"] else CrossAttnQ8
            s["call"] = make(batch, h, kv, d, n, cu_seqlens_host=np.concatenate([[0], np.cumsum(lens)]), device=DEV)
    elif op == "append":
        lens, new = ints(case["lens"]), ints(case["new"])
        batch, d, kv = len(lens), case["dim"], case["kv_heads"]
        s["batch"], s["cu"] = batch, _cu(lens)
        s["table"], pages = _table([a + b for a, b in zip(lens, new)], case["page"], seed, spare=1)
        s["k"], s["k_scale"] = _cache(pages, case["page"], case["block"], kv, d, g, True)
        s["v"], s["v_scale"] = _cache(pages, case["page"], case["block"], kv, d, g, True)
        if case["path"]:
            # trees of 64 nodes; the accepted path of each is `new` nodes long (0: no node)
            nodes = 64
            s["nodes"], s["max_new"] = nodes, nodes
            r = np.random.default_rng(seed + 3)
            path = np.full((batch, nodes), -1, dtype=np.int32)
            for b, n in enumerate(new):
                if n:
                    path[b, :n] = np.concatenate([[0], 1 + np.sort(r.permutation(nodes - 1)[:n - 1])])
            s["path"] = torch.from_numpy(path).to(DEV)
            s["accepted"] = torch.from_numpy(np.array(new, dtype=np.int32) - 1).to(DEV)
            rows = batch * nodes
        else:
            s["cu_new"], s["max_new"] = _cu(new), max(new)
            rows = sum(new)
        size = 0.5 + 2.0 * torch.rand(rows, kv, 1, generator=g, device=DEV)
        s["k_new"] = (torch.randn(rows, kv, d, generator=g, device=DEV) * size).to(torch.bfloat16)
        s["v_new"] = (torch.randn(rows, kv, d, generator=g, device=DEV) * size).to(torch.bfloat16)
        if own:
            from tree_verification_attention_longspec_b200 import KVCacheQ8
            s["cache"] = KVCacheQ8(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"])
    elif op == "sample":
        s["logits"] = _logits(case["rows"], case["vocab"], case["dtype"], g)
        s |= _sampling(case["rows"], case["how"], g)
    else:
        sizes = ints(case["trees"])
        rows = sum(sizes)
        s["sizes"] = torch.tensor(sizes, device=DEV)
        s["batch"], s["nodes"], s["cu_tree"] = len(sizes), max(sizes), _cu(sizes)
        s["parent"] = _parents(sizes, seed)
        s["logits"] = _logits(rows, case["vocab"], case["dtype"], g)
        s |= _sampling(rows, case["how"], g)
        # peaked rows; a draft guesses its parent's likeliest token three times in four
        peak = torch.randint(case["vocab"], (rows,), generator=g, device=DEV)
        at = torch.arange(rows, device=DEV)
        s["logits"][at, peak] = 16.0
        base = torch.repeat_interleave(s["cu_tree"][:-1], s["sizes"])
        above = (base + s["parent"].clamp(min=0)).long()
        other = torch.randint(case["vocab"], (rows,), generator=g, device=DEV)
        hit = torch.rand(rows, generator=g, device=DEV) < 0.75
        s["draft"] = torch.where(hit, peak[above], other).to(torch.int32)
    return s


# ------------------------------------------------------------------------------ plain forms


def _rows_of(table, page, positions):
    """Cache rows of positions [B, n] of each sequence."""
    at = torch.clamp(positions // page, max=table.shape[1] - 1)
    return torch.gather(table.long(), 1, at) * page + positions % page


def _values(s, which, rows):
    """The cached values of rows [B, n] in fp32: code times scale."""
    codes = s[which].view(-1, s["kv_heads"], s["dim"])[rows].float()
    scale = s[which + "_scale"].view(-1, s["kv_heads"])[rows // s["block"]]
    return codes * scale[..., None]


def _ancestors(parent, count):
    """[B, T, T]: whether node j is node i or an ancestor of it, of padded parents."""
    up = torch.nn.functional.one_hot(parent.long().clamp(min=0), count).double()
    up = up * (parent >= 0)[..., None] + torch.eye(count, device=DEV, dtype=torch.float64)
    return torch.linalg.matrix_power(up, count) > 0


def _plain_attend(s):
    b, n, kv, d = s["batch"], s["nodes"], s["kv_heads"], s["dim"]
    group = s["heads"] // kv
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    pos = torch.arange(max(1, s["max_len"]), device=DEV)[None].expand(b, -1)
    rows = _rows_of(s["table"], s["page"], pos)
    k, v = _values(s, "k", rows), _values(s, "v", rows)
    seen = (pos < lens[:, None])[:, None].expand(b, n, -1)
    v = torch.where((pos < lens[:, None])[..., None, None], v, 0.0)
    if s["tree"]:
        k = torch.cat([k, s["k_tree"].float().view(b, n, kv, d)], 1)
        v = torch.cat([v, s["v_tree"].float().view(b, n, kv, d)], 1)
        seen = torch.cat([seen, _ancestors(s["parent"].view(b, n), n)], 2)
    q = s["q"].float().view(b, n, kv, group, d).permute(0, 2, 1, 3, 4).reshape(b, kv, n * group, d)
    score = (q @ k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    score = torch.where(seen[:, None, :, None].expand(b, 1, n, group, -1).reshape(b, 1, n * group, -1), score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3.0e38)
    w = torch.exp(score - top)
    total = w.sum(-1, keepdim=True)
    out = (w @ v.permute(0, 2, 1, 3)) / total
    lse = (top + torch.log(total))[..., 0]
    out = out.view(b, kv, n, group, d).permute(0, 2, 1, 3, 4).reshape(b * n, kv * group, d)
    lse = lse.view(b, kv, n, group).permute(0, 2, 1, 3).reshape(b * n, kv * group)
    return out.to(torch.bfloat16), lse


def _plain_append(s):
    b, kv, d, block, page = s["batch"], s["kv_heads"], s["dim"], s["block"], s["page"]
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(s["max_new"], device=DEV)[None]
    if s["path"].__class__ is torch.Tensor:
        count = (s["accepted"] + 1).long()
        source = torch.arange(b, device=DEV)[:, None] * s["nodes"] + s["path"].long().clamp(min=0)
    else:
        count = (s["cu_new"][1:] - s["cu_new"][:-1]).long()
        source = s["cu_new"][:-1, None].long() + i
    there = i < count[:, None]
    source, to = source[there], _rows_of(s["table"], page, lens[:, None] + i)[there]
    blocks = to // block
    # the first block of a sequence keeps its older tokens where it has some
    held = (lens % block)[:, None].expand_as(there)
    first = (lens[:, None] + i) // block == (lens // block)[:, None]
    old = torch.zeros(s["k_scale"].numel() // kv, dtype=torch.bool, device=DEV)
    old[blocks] = ((held > 0) & first)[there]
    total = (lens + count).to(torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), torch.cumsum(total, 0).to(torch.int32)])
    _plain_quantise(s, "k", source, to, blocks, old, lens)
    _plain_quantise(s, "v", source, to, blocks, old, lens)
    return s["k"], s["v"], s["k_scale"], s["v_scale"], cu


def _plain_quantise(s, which, source, to, blocks, old, lens):
    kv, d, block = s["kv_heads"], s["dim"], s["block"]
    x = s[which + "_new"][source].double()
    scale = s[which + "_scale"].view(-1, kv)
    amax = torch.zeros(scale.shape[0], kv, dtype=torch.float64, device=DEV)
    amax.scatter_reduce_(0, blocks[:, None].expand(-1, kv), x.abs().amax(-1), "amax")
    part, power = torch.frexp(amax)  # amax = part * 2^power, part in [0.5, 1); 448 = 0.875 * 2^9
    power = torch.where(part > 0.875, power - 8, power - 9)
    power = torch.where(amax > 0, power, MIN_EXP).clamp(MIN_EXP, MAX_EXP)
    need = torch.exp2(power.double())
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV)
    touched[blocks] = True
    now = torch.where(old[:, None], torch.maximum(scale.double(), need), need)
    now = torch.where(touched[:, None], now, scale.double())
    codes = s[which].view(-1, block, kv, d)
    again = codes.double() * (scale.double() / now)[:, None, :, None]
    again = again.to(torch.float8_e4m3fn)
    # only the older tokens of a raised block are written again
    at = lens // block
    held = torch.arange(block, device=DEV)[None] < (lens % block)[:, None]
    home = _rows_of(s["table"], s["page"], (at * block)[:, None])[:, 0] // block
    keep = torch.zeros(codes.shape[0], block, dtype=torch.bool, device=DEV)
    keep.index_put_((home,), held, accumulate=True)
    keep = keep & old[:, None]
    bits, new_bits = codes.view(torch.uint8), again.view(torch.uint8)
    bits.copy_(torch.where(keep[:, :, None, None], new_bits, bits))
    y = (x / now[blocks][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    s[which].view(-1, kv, d).view(torch.uint8)[to] = y.view(torch.uint8)
    scale.copy_(now)


def _plain_sample(s):
    logits = s["logits"].double()
    top = logits.amax(-1, keepdim=True)
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, 1.0, s["temperature"].double())[:, None]
    w, order = torch.sort((logits - top) / t, dim=-1, descending=True, stable=True)
    w = torch.exp(w)
    rank = torch.arange(w.shape[1], device=DEV)[None]
    k = s["top_k"].long()[:, None]
    keep = (k <= 0) | (rank < k)
    w = torch.where(keep, w, 0.0)
    before = torch.cumsum(w, -1) - w
    p = s["top_p"].double()[:, None]
    keep = keep & ((p >= 1) | (before < p * w.sum(-1, keepdim=True)) | (rank == 0))
    keep = keep & (w >= s["min_p"].double()[:, None])
    w = torch.where(keep, w, 0.0)
    w = torch.zeros_like(w).scatter_(1, order, w)  # back to the order of the vocabulary
    total = torch.cumsum(w, -1)
    past = total <= s["uniform"].double()[:, None] * total[:, -1:]
    token = past.sum(-1)
    last = w.shape[1] - 1 - (w > 0).flip(-1).int().argmax(-1)
    token = torch.minimum(token, last)
    return torch.where(greedy, order[:, 0], token).to(torch.int32)


def _plain_accept(s):
    token = _plain_sample(s)
    b, n = s["batch"], s["nodes"]
    i = torch.arange(n, device=DEV)[None].expand(b, n)
    there = i < s["sizes"][:, None]
    at = torch.clamp(s["cu_tree"][:-1, None].long() + i, max=token.numel() - 1)
    parent = torch.where(there, s["parent"][at], 0)
    parent = torch.where(i == 0, -1, parent)
    chosen, draft = token[at], s["draft"][at]
    match = there & (i > 0) & (draft == torch.gather(chosen, 1, parent.long().clamp(min=0)))
    first = torch.full((b, n), n, dtype=torch.int64, device=DEV)
    first.scatter_reduce_(1, parent.long().clamp(min=0), torch.where(match, i, n), "amin")
    on = match & (i == torch.gather(first, 1, parent.long().clamp(min=0)))
    miss = (~(on | (i == 0))).double()
    on = there & ((_ancestors(parent, n).double() @ miss[..., None])[..., 0] == 0)
    length = on.sum(-1) - 1
    path = torch.sort(torch.where(on, i, n), -1).values
    after = torch.gather(chosen, 1, torch.gather(path, 1, length[:, None]))[:, 0]
    path = torch.where(path == n, -1, path)
    return token, length.to(torch.int32), path.to(torch.int32), after


def run(s):
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "sample": _plain_sample, "accept": _plain_accept}[s["op"]](s)
    if s["op"] == "attend":
        if s["tree"]:
            return s["call"](s["q"], s["cache"], s["k_tree"], s["v_tree"], s["parent"], s["cu"])
        return s["call"](s["q"], s["cache"], s["cu"])
    if s["op"] == "append":
        if s["path"] is False:
            cu = s["cache"].append(s["k_new"], s["v_new"], s["cu"], s["cu_new"], s["max_new"])
        else:
            cu = s["cache"].commit(s["k_new"], s["v_new"], s["cu"], s["accepted"], s["path"])
        return s["k"], s["v"], s["k_scale"], s["v_scale"], cu
    from tree_verification_attention_longspec_b200 import sample, tree_accept_sample
    knobs = dict(temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    if s["op"] == "sample":
        return sample(s["logits"], s["uniform"], **knobs)
    return tree_accept_sample(s["logits"], s["uniform"], s["draft"], s["parent"], s["nodes"], cu_tree=s["cu_tree"], **knobs)


def work(case):
    op = case["op"]
    if op == "attend":
        lens = ints(case["lens"])
        n, d, kv, h, batch = case["nodes"], case["dim"], case["kv_heads"], case["heads"], len(lens)
        extra = n if case["tree"] else 0
        size = 2 * sum(lens) * kv * d + 2 * 4 * kv * sum((x + case["block"] - 1) // case["block"] for x in lens)
        size += 2 * 2 * batch * extra * kv * d + batch * n * h * (2 * 2 * d + 4)
        return dict(bytes=size, flops=sum(4 * n * h * d * (x + extra) for x in lens))
    if op == "append":
        tokens = sum(ints(case["new"]))
        values = 2 * tokens * case["kv_heads"] * case["dim"]
        return dict(bytes=3 * values, flops=2 * values)
    rows = case["rows"] if op == "sample" else sum(ints(case["trees"]))
    return dict(bytes=rows * case["vocab"] * (2 if case["dtype"] == "bf16" else 4), flops=rows * case["vocab"])


# ------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    """From the definitions, one sequence (one row) at a time, in 64 bits."""
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "sample": _exact_sample, "accept": _exact_accept}[case["op"]](s)


def _exact_attend(s):
    kv, d, n, page, block = s["kv_heads"], s["dim"], s["nodes"], s["page"], s["block"]
    group = s["heads"] // kv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    lens, table = ints(s["lens"]), s["table"].cpu().tolist()
    deq = {}
    for w in "kv":
        codes = s[w].double().view(-1, block, kv, d)
        deq[w] = (codes * s[w + "_scale"].double().view(-1, 1, kv, 1)).view(-1, page, kv, d)
    for b, length in enumerate(lens):
        use = table[b][:(length + page - 1) // page]
        key, val = (deq[w][use].reshape(-1, kv, d)[:length] for w in "kv")
        visible = torch.ones(n, length, dtype=torch.bool, device=DEV)
        if s["tree"]:
            here = slice(b * n, (b + 1) * n)
            key, val = torch.cat([key, s["k_tree"][here].double()]), torch.cat([val, s["v_tree"][here].double()])
            parent = s["parent"][here].cpu().tolist()
            own_tree = np.zeros((n, n), dtype=bool)
            for i in range(n):
                if i:
                    own_tree[i] = own_tree[parent[i]]
                own_tree[i, i] = True
            visible = torch.cat([visible, torch.from_numpy(own_tree).to(DEV)], 1)
        for h in range(s["heads"]):
            score = s["q"][b * n:(b + 1) * n, h].double() @ key[:, h // group].T / math.sqrt(d)
            score = score.masked_fill(~visible, -math.inf)
            norm = torch.logsumexp(score, -1)
            lse[b * n:(b + 1) * n, h] = norm
            out[b * n:(b + 1) * n, h] = torch.exp(score - norm[:, None]) @ val[:, h // group]
    return out, lse


def _exact_append(s):
    kv, d, page, block = s["kv_heads"], s["dim"], s["page"], s["block"]
    lens, new, table = ints(s["lens"]), s["new"], s["table"].cpu().tolist()
    new = ints(new)
    out = {}
    for w in "kv":
        codes = s[w].float().cpu().double().view(-1, page, kv, d).clone()
        scale = s[w + "_scale"].cpu().double().clone()
        data = s[w + "_new"].cpu().double()
        at = 0
        for b, (length, count) in enumerate(zip(lens, new)):
            if s["path"] is False:
                rows = data[at:at + count]
                at += count
            else:
                rows = data[(b * s["nodes"] + s["path"][b, :count].cpu().long())]
            pos = length
            while pos < length + count:
                start, end = pos // block * block, min(length + count, (pos // block + 1) * block)
                p, o = table[b][start // page], start % page
                x = rows[pos - length:end - length]
                amax = x.abs().amax((0, 2))
                for h in range(kv):
                    a = float(amax[h])
                    e = MIN_EXP
                    while a > E4M3_MAX * 2.0 ** e and e < MAX_EXP:
                        e += 1
                    unit = 2.0 ** e
                    if pos > start:
                        before = float(scale[p, o // block, h])
                        unit = max(unit, before)
                        codes[p, o:o + pos - start, h] = _e4m3(codes[p, o:o + pos - start, h] * before / unit)
                    scale[p, o // block, h] = unit
                    codes[p, o + pos - start:o + end - start, h] = _e4m3(x[:, h] / unit)
                pos = end
        out[w], out[w + "_scale"] = codes, scale
    total = np.concatenate([[0], np.cumsum([a + b for a, b in zip(lens, new)])])
    return out["k"], out["v"], out["k_scale"], out["v_scale"], torch.from_numpy(total.astype(np.int32))


def _e4m3(x):
    """The nearest e4m3 value, ties to even: steps of 2^-3 of the value's power of two, 2^-9 at least."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_sample(s):
    tokens = []
    host = {k: s[k].cpu().tolist() for k in ("uniform", "temperature", "top_k", "top_p", "min_p")}
    for r in range(s["logits"].shape[0]):
        x = s["logits"][r].double().cpu().numpy()
        if host["temperature"][r] <= 0:
            tokens.append(int(np.argmax(x)))
            continue
        order = np.argsort(-x, kind="stable")
        w = np.exp((x[order] - x[order[0]]) / host["temperature"][r])
        if host["top_k"][r] > 0:
            w[host["top_k"][r]:] = 0
        if host["top_p"][r] < 1:
            before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
            cut = before >= host["top_p"][r] * w.sum()
            cut[0] = False
            w[cut] = 0
        w[w < host["min_p"][r]] = 0
        back = np.zeros_like(w)
        back[order] = w
        total = np.cumsum(back)
        tokens.append(int(min(np.searchsorted(total, host["uniform"][r] * total[-1], side="right"), np.flatnonzero(back)[-1])))
    return torch.tensor(tokens, dtype=torch.int32)


def _exact_accept(s):
    token = _exact_sample(s)
    cu, parent, draft, chosen = (x.cpu().tolist() for x in (s["cu_tree"], s["parent"], s["draft"], token))
    lengths, paths, after = [], [], []
    for b in range(s["batch"]):
        base, n = cu[b], cu[b + 1] - cu[b]
        path = [0]
        while True:
            here = path[-1]
            step = [i for i in range(here + 1, n) if parent[base + i] == here and draft[base + i] == chosen[base + here]]
            if not step:
                break
            path.append(step[0])
        lengths.append(len(path) - 1)
        after.append(chosen[base + path[-1]])
        paths.append(path + [-1] * (s["nodes"] - len(path)))
    return token, torch.tensor(lengths, dtype=torch.int32), torch.tensor(paths, dtype=torch.int32), torch.tensor(after, dtype=torch.int32)
