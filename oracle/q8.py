"""The 8-bit paged cache, attention over it, and sampling, in fp64 — TEST INFRASTRUCTURE ONLY.

Only ``tests/`` and the smoke check may import this module; the CUDA path never does and
shares no code with it. Written as plain loops over sequences, blocks and rows from the
definitions:

- e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; exponent 0 is subnormal (steps of
  2^-9); 0x7f and 0xff are NaN, there is no infinity, the largest value is 448.
- a cached value is its code's value times the scale of its block of tokens and head;
- the append's scales are powers of two (``scale_exponent``), a block with earlier tokens
  keeps the larger of its scale and the new rows' own, its earlier codes rounded again;
- sampling weighs exp((l - top) / t), filters by top-k, top-p and min-p in the order of
  larger logit, then smaller index, and takes the first kept index whose inclusive sum
  exceeds u times the kept sum.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 64


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        elif e == 0:
            out[c] = s * m * 2.0 ** -9
        else:
            out[c] = s * (8 + m) * 2.0 ** (e - 10)
    return out


TABLE = e4m3_table()
_POSITIVE = TABLE[:127]  # 0 .. 448, increasing


def e4m3_encode(x) -> np.ndarray:
    """Codes of x: nearest, ties to the even code, saturated, NaN to 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), E4M3_MAX)
    hi = np.searchsorted(_POSITIVE, a)  # first value >= a
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), code).astype(np.uint8)


def scale_exponent(amax: float) -> int:
    """The least e in [-60, 64] with amax <= 448 * 2^e."""
    e = MIN_EXP
    while e < MAX_EXP and amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return e


def gather(pages, scale, table, length, page_size, scale_block):
    """[length, H, d] values of one sequence: pages [num_pages, page_size, H, d] codes,
    scale [num_pages, page_size / scale_block, H], table the sequence's row."""
    rows = []
    for key in range(length):
        p, o = int(table[key // page_size]), key % page_size
        rows.append(TABLE[pages[p, o]] * np.asarray(scale[p, o // scale_block], dtype=np.float64)[:, None])
    H, d = pages.shape[2:]
    return np.array(rows).reshape(length, H, d)


def attention(q, k, v, visible, scale):
    """One sequence: q [n, Hq, d], k / v [x, Hkv, d], visible [n, x]. Returns out [n, Hq, d],
    lse [n, Hq] (0 and -inf for a row that sees nothing), spread [n, Hq, d] = sum of w |v|,
    and reach [n, Hq] = the largest scale * sum |q_i k_i| of a visible key."""
    n, Hq, d = q.shape
    g = Hq // k.shape[1] if k.shape[1] else 1
    out, spread = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, reach = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for h in range(Hq):
        kk, vv = k[:, h // g], v[:, h // g]
        s = scale * (q[:, h] @ kk.T)
        r = scale * (np.abs(q[:, h]) @ np.abs(kk).T)
        for i in range(n):
            see = visible[i]
            if not see.any():
                continue
            x = s[i, see]
            top = x.max()
            w = np.exp(x - top)
            lse[i, h] = top + np.log(w.sum())
            w /= w.sum()
            out[i, h], spread[i, h] = w @ vv[see], w @ np.abs(vv[see])
            reach[i, h] = r[i, see].max()
    return out, lse, spread, reach


def ancestors(parent) -> np.ndarray:
    n = len(parent)
    see = np.zeros((n, n), dtype=bool)
    for i in range(n):
        x = i
        while x >= 0:
            see[i, x] = True
            x = int(parent[x])
    return see


def append(pages, scale, table, lens, rows_of, page_size, scale_block):
    """Copies of (pages, scale) with rows_of[b] ([n_b, H, d] values, a row of None kept as it
    is) appended to sequence b."""
    pages, scale = pages.copy(), np.asarray(scale, dtype=np.float64).copy()
    for b, rows in enumerate(rows_of):
        room = table.shape[1] * page_size - lens[b]
        rows = rows[:max(0, room)]
        end = lens[b] + len(rows)
        for first in range(lens[b] // scale_block * scale_block, end, scale_block):
            p0, p1 = max(first, lens[b]), min(end, first + scale_block)
            if p0 >= p1:
                continue
            page, o = int(table[b, first // page_size]), first % page_size
            if not 0 <= page < pages.shape[0]:
                continue
            at = (page, o // scale_block)
            for h in range(pages.shape[2]):
                new = [(p, rows[p - lens[b]][h]) for p in range(p0, p1) if rows[p - lens[b]] is not None]
                mags = np.abs(np.concatenate([x for _, x in new])) if new else np.zeros(1)
                mags = mags[~np.isnan(mags)]
                unit = 2.0 ** scale_exponent(float(mags.max()) if mags.size else 0.0)
                if p0 > first:
                    old = scale[at + (h,)]
                    if old < unit:
                        held = slice(o, o + p0 - first)
                        pages[page, held, h] = e4m3_encode(TABLE[pages[page, held, h]] * (old / unit))
                    unit = max(unit, old)
                scale[at + (h,)] = unit
                for p, x in new:
                    pages[page, o + p - first, h] = e4m3_encode(x / unit)
    return pages, scale


def sample_row(logits, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, margin): margin is how far u * Z lies from the nearest border of the token's
    interval, relative to Z (inf where no border was computed)."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return 0, np.inf
    if not t > 0:
        return int(np.argmax(x)), np.inf
    order = np.argsort(-x, kind="stable")
    with np.errstate(invalid="ignore"):
        w = np.where(x == top, 1.0, np.where((x == -np.inf) | (top == np.inf), 0.0, np.exp((x - top) / t)))[order]
    keep = np.ones(len(w), dtype=bool)
    if 0 < k < len(w):
        keep[k:] = False
    w = np.where(keep, w, 0.0)
    if p < 1.0:
        before = np.cumsum(w) - w
        keep &= before < p * w.sum()
        keep[0] = True
    if m > 0:
        keep &= w >= min(m, 1.0)
    back = np.zeros(len(w))
    back[order] = np.where(keep, w, 0.0)
    total = np.cumsum(back)
    target = (u if u > 0 else 0.0) * total[-1]
    i = int(np.searchsorted(total, target, side="right"))
    i = min(i, int(np.flatnonzero(back)[-1]))
    low = total[i - 1] if i else -np.inf
    return i, min(abs(target - low), abs(total[i] - target)) / total[-1]


def walk(token, draft, parent):
    """(accepted, path, next token) of one tree from the tokens drawn at its nodes."""
    n = len(parent)
    if n == 0 or parent[0] != -1 or any(not 0 <= parent[i] < i for i in range(1, n)):
        return -1, [], -1
    path = [0]
    while True:
        here = path[-1]
        step = [c for c in range(here + 1, n) if parent[c] == here and draft[c] == token[here]]
        if not step:
            return len(path) - 1, path, int(token[here])
        path.append(step[0])


__all__ = ["E4M3_MAX", "MIN_EXP", "MAX_EXP", "TABLE", "e4m3_encode", "scale_exponent", "gather", "attention",
           "ancestors", "append", "sample_row", "walk"]
