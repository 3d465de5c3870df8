"""Codes written at scales that are no powers of two (another writer's, amax / 448): each is the
nearest to the exact quotient or product, also where that lies next to the middle of two codes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import q8 as oq
from tests.q8_harness import bf16, f64
from tests.test_q8_cache_gpu import Pool

LARGEST = np.array([8.5, 9.0, 9.5, 10.5, 11.0, 11.5, 12.5, 13.0, 13.5, 7.0 + 2.0 ** -6, 14.0 - 2.0 ** -7])
SCALES = LARGEST.astype(np.float32) / np.float32(448.0)
HEADS = len(SCALES)


def _quotients():
    """Every positive bf16 from 2^-7 to 7: below the largest that these scales are kept for."""
    x = torch.arange(0x3C00, 0x40E1, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    return x.double().numpy()


def test_the_values_include_quotients_and_products_that_two_roundings_get_wrong():
    """(On the CPU.) Rounding to fp32 first gives other codes for some of them."""
    x = _quotients()
    wrong = 0
    for s in SCALES:
        once = oq.e4m3_encode(x / np.float64(s))
        wrong += int((oq.e4m3_encode(x.astype(np.float32) / s) != once).sum())
    assert wrong >= HEADS
    wrong = 0
    codes = oq.TABLE[:127]
    for s in SCALES:
        ratio = s * np.float32(2.0 ** 5)
        once = oq.e4m3_encode(codes * np.float64(ratio))
        wrong += int((oq.e4m3_encode(codes.astype(np.float32) * ratio) != once).sum())
    assert wrong >= HEADS


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _append(pool, cache, rows, n_new):
    k, v = bf16(rows), bf16(-rows)
    cu = cache.append(k.cuda(), v.cuda(), pool.cu, _dev(np.array([0, n_new], dtype=np.int32)), n_new)
    pool.expect({"k": [list(f64(k))], "v": [list(f64(v))]}, cu, [pool.lens[0] + n_new])


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,block", [(64, 128, 128), (128, 64, 64), (64, 16, 16)])
def test_rows_divided_by_a_kept_scale(d, page, block):
    r = np.random.default_rng(d)
    n_new = block - 1
    pool = Pool((1,), (block,), HEADS, d, page, block)
    for w in "kv":
        pool.scales[w][:] = SCALES
    cache = pool.device()
    rows = r.choice(_quotients(), (n_new, HEADS, d)) * r.choice([-1.0, 1.0], (n_new, HEADS, d))
    every = np.resize(_quotients(), (n_new, d)) if n_new * d >= len(_quotients()) else rows[:, 0]
    rows[:, :] = np.where(r.random((n_new, 1, d)) < 0.5, rows, every[:, None])
    rows[0, :, 0] = 0.515625  # times 448 / 11 next to 21, between the codes of 20 and 22
    _append(pool, cache, rows, n_new)
    assert np.array_equal(pool.scales["k"][pool.table[0, 0], 0], SCALES)


@pytest.mark.gpu
@pytest.mark.parametrize("d,page,block", [(64, 128, 128), (128, 64, 64), (64, 16, 16)])
def test_codes_rounded_again_from_such_a_scale(d, page, block):
    r = np.random.default_rng(d + 1)
    held = block - 1
    pool = Pool((held,), (block,), HEADS, d, page, block)
    for w in "kv":
        pool.scales[w][:] = SCALES
        pool.codes[w] = (pool.codes[w] | r.choice([0, 128], pool.codes[w].shape)).astype(np.uint8)
    cache = pool.device()
    rows = r.standard_normal((1, HEADS, d))
    rows[:, :, 5] = 14.0  # 448 * 2^-5: the scale becomes 2^-5
    _append(pool, cache, rows, 1)
    assert (pool.scales["k"][pool.table[0, 0], 0] == 2.0 ** -5).all()


@pytest.mark.gpu
def test_odd_values_at_a_kept_scale():
    """Infinities saturate, NaN stays, zeros keep their value, and what overflows saturates."""
    pool = Pool((3,), (16,), HEADS, 64, 16, 16)
    for w in "kv":
        pool.scales[w][:] = SCALES * np.float32(2.0 ** 58)  # kept for infinities too (2^64 is the largest unit)
        pool.scales[w][:, :, ::2] = np.float32(1.25 * 2.0 ** 64)
    cache = pool.device()
    x = np.random.default_rng(3).standard_normal((5, HEADS, 64))
    x[0, :, 0], x[1, :, 1], x[2, :, 2], x[3, :, 3] = np.inf, -np.inf, np.nan, 0.0
    x[4, :, 4], x[4, :, 5] = 3e38, -1e-38
    _append(pool, cache, x, 5)
