"""Temperatures at the ends of fp32's range: logits further apart than its largest number that all
weigh something, and subnormal ones that are told apart by a temperature as small."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_sample_gpu import _check, _sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [7, 3000, 60000])
@pytest.mark.parametrize("t", [2e36, 1e38, 3e38, np.inf])
def test_differences_beyond_fp32(t, vocab, dtype):
    r = np.random.default_rng(vocab)
    rows = 24
    x = r.choice([3.2e38, 1e38, 0.0, -1e38, -3.3e38, -np.inf, 2.0], (rows, vocab))
    x[:, :2] = [3.2e38, -3.2e38]
    u = r.random(rows)
    full = np.full(rows, t)
    with np.errstate(all="ignore"):
        _check(*_sample(x, u, dtype, temperature=full))
        _check(*_sample(x, u, dtype, temperature=full, top_k=r.integers(1, vocab, rows)))
        _check(*_sample(x, u, dtype, temperature=full, top_p=r.choice([0.3, 0.9, 0.99], rows)))
        _check(*_sample(x, u, dtype, temperature=full, min_p=np.full(rows, 0.1), top_p=np.full(rows, 0.95)))


def test_just_below_the_limit_differences_that_overflow_weigh_nothing():
    r = np.random.default_rng(2)
    x = r.choice([3.2e38, 3.199e38, -3.3e38, -np.inf], (16, 500))
    x[:, 0] = 3.2e38
    for t in (1e35, 9e35):
        for opts in ({}, {"top_p": np.full(16, 0.7)}, {"top_k": np.full(16, 100)}):
            with np.errstate(all="ignore"):
                _check(*_sample(x, r.random(16), "f32", temperature=np.full(16, t), **opts))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [5, 3000, 60000])
@pytest.mark.parametrize("t", [1e-45, 9.2e-41, 1e-39, 2.9e-39, 3e-39, 1e-38])
def test_subnormal_temperatures(t, vocab, dtype):
    r = np.random.default_rng(vocab + 1)
    rows = 24
    x = r.choice([9.2e-41, -9.2e-41, 0.0, 3e-40, 1e-39, -2e-39, -np.inf, -1.0], (rows, vocab))
    u = r.random(rows)
    full = np.full(rows, t)
    with np.errstate(all="ignore"):
        for opts in ({}, {"top_k": r.integers(1, vocab, rows)}, {"top_p": r.choice([0.3, 0.9, 0.99], rows)},
                     {"min_p": np.full(rows, 0.1), "top_p": np.full(rows, 0.95)}):
            got, want, margin = _sample(x, u, dtype, temperature=full, **opts)
            bad = (got != want) & (margin > 1e-9)
            assert not bad.any(), (opts, np.flatnonzero(bad), got[bad], want[bad])
