"""A call whose plan the host has no memory for is refused: no exception leaves a C entry."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A child process, so that its limit is its own: 2^28 sequences want 1 GB for their block counts.
CHILD = r"""
import ctypes, re, resource
import torch
from tree_verification_attention_longspec_b200 import binding
torch.zeros(1, device="cuda")
lib = binding.load_library()
small = binding.make_dims(4, 8, 2, 64, 2, max_prefix_len=100)[0]
want = lib.ls_verify_attn_q8_workspace_size(ctypes.byref(small), None)
assert want > 0
used = int(re.search(r"VmSize:\s+(\d+) kB", open("/proc/self/status").read()).group(1)) * 1024
resource.setrlimit(resource.RLIMIT_AS, (used + (256 << 20), resource.getrlimit(resource.RLIMIT_AS)[1]))
big = binding.make_dims(1 << 28, 1, 1, 64, 1, max_prefix_len=1)[0]
ref = ctypes.byref(big)
sizes = [lib.ls_verify_attn_workspace_size(ref), lib.ls_verify_attn_ex_workspace_size(ref, None),
         lib.ls_cross_attn_workspace_size(ref), lib.ls_verify_attn_q8_workspace_size(ref, None),
         lib.ls_cross_attn_q8_workspace_size(ref)]
assert sizes == [0] * 5, sizes
assert lib.ls_verify_attn_plan(ref, None, None, None) == 2
assert lib.ls_verify_attn_check(ref, None, None) == 2
assert lib.ls_verify_attn_q8_workspace_size(ctypes.byref(small), None) == want
print("refused")
"""


def test_a_batch_without_host_memory_is_refused():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "refused" in r.stdout, (r.returncode, r.stdout, r.stderr[-2000:])


def test_the_status_of_many_combine_ctas_is_read_whole():
    """Words past the first piece that the check copies count too."""
    from tree_verification_attention_longspec_b200 import binding
    B, T, H = 700, 64, 8  # 89,600 CTAs of the combine kernel
    dims = binding.make_dims(B, H, H, 64, T, max_prefix_len=16)[0]
    ws = torch.zeros(binding.workspace_size(dims), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    words = ws.view(torch.int32)
    n = B * T * H // 4
    for at, code, want in ((0, 1, 5), (65535, 4, 6), (65536, 2, 7), (n - 1, 1, 5)):
        words.zero_()
        assert binding.check(dims, ws.data_ptr(), stream) == 0
        words[at] = code
        assert binding.check(dims, ws.data_ptr(), stream) == want
    words.zero_()
    words[n] = 1  # not a status
    assert binding.check(dims, ws.data_ptr(), stream) == 0
