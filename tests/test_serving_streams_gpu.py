"""A call object that is dropped while its call still runs on a stream of its own."""
from __future__ import annotations

import pytest
import torch

from tests.q8_harness import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nodes", [1, 40])
def test_the_workspace_outlives_the_object_on_another_stream(nodes):
    from tree_verification_attention_longspec_b200 import VerifyAttnQ8
    case = Case((900, 30), 8, 2, 128, nodes, 64, 32, seed=nodes)
    args = case.device()
    q, rest = args[1], (args[0], *args[2:])
    want = VerifyAttnQ8(2, 8, 2, 128, nodes, max_prefix_len=900)(q, *rest)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    call = VerifyAttnQ8(2, 8, 2, 128, nodes, max_prefix_len=900)
    place, size = call.workspace.data_ptr(), call.ws_bytes
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # about a tenth of a second: the call has not run when the object goes
        call(q, *rest, out, lse)
    del call
    again = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() != place
    again.fill_(0xFF)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
