"""bf16 rows in which top-k ends inside a run of zeros, with positive logits above them that are
too small to have a bin of their own: what top-k keeps of each decides top-p's border."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_sample_gpu import _check, _sample

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1.0, 4.0])
@pytest.mark.parametrize("high,small,zeros,low", [(2000, 30000, 30000, 100), (300, 900, 5000, 0), (50, 400, 400, 3000)])
@pytest.mark.parametrize("at", [0.01, 0.5, 1.0])
def test_top_k_that_ends_among_zeros(high, small, zeros, low, at, t):
    r = np.random.default_rng(high + low)
    rows = 120
    x = np.concatenate([np.full(high, 1.0), np.full(small, 8e-5), np.zeros(zeros), np.full(low, -1.0)])
    x[high + small:high + small + zeros:2] = -0.0
    x = np.stack([r.permutation(x) for _ in range(rows)])
    k = np.full(rows, high + small + max(1, int(at * zeros)))
    z = high * np.exp(0.0) + (k[0] - high) * np.exp(-1.0 / t)
    # top-p's border among the large values, for the most part
    p = r.uniform(0.2, 1.1, rows) * high / z
    _check(*_sample(x, r.random(rows), "bf16", temperature=np.full(rows, t), top_k=k, top_p=np.minimum(p, 0.999)))


@pytest.mark.parametrize("few", [1, 500])
def test_top_k_that_ends_among_zeros_with_small_logits_on_both_sides(few):
    r = np.random.default_rng(few)
    rows, big, zeros = 48, 700, 3000
    x = np.concatenate([np.full(big, 2.0), np.full(few, 1e-5), np.zeros(zeros), np.full(few, -1e-5), np.full(400, -2.0)])
    x = np.stack([r.permutation(x) for _ in range(rows)])
    for k in (big + 1, big + few, big + few + 1, big + few + zeros // 2, big + few + zeros, big + 2 * few + zeros):
        _check(*_sample(x, r.random(rows), "bf16", top_k=np.full(rows, k), top_p=r.uniform(0.05, 0.95, rows)))
