"""The smoke check launches every kind of kernel that the package offers."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_smoke_reaches_the_serving_kernels(capsys):
    from torch.profiler import ProfilerActivity, profile

    import __graft_entry__
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        __graft_entry__.smoke()
        torch.cuda.synchronize()
    assert capsys.readouterr().out.count("smoke ok") == 2
    names = " ".join(e.name for e in p.events())
    if "kernel" not in names:
        pytest.skip("the profiler sees no kernels here")
    for kernel in ("partials_tc_kernel", "combine_kernel", "q8_rows_kernel", "q8_tc_kernel", "q8_append_kernel",
                   "sample_kernel", "sampled_walk_kernel"):
        assert kernel in names, kernel
