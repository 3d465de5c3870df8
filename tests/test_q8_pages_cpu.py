"""Looking up the 8-bit cache's pages at the ends of the index range (no GPU)."""
from __future__ import annotations

import os
import subprocess

from tests.test_serving_cpu import INVALID, UNSUPPORTED, _append, _attend, _commit, _cross, _dims, _kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tree_verification_attention_longspec_b200", "csrc")


def test_every_key_is_looked_up_inside_the_cache(tmp_path):
    exe = tmp_path / "q8_pages_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC,
                    os.path.join(ROOT, "tests", "q8_pages_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_tables_of_too_many_tokens_are_refused(cuda_lib):
    most = 2 ** 31 - 2 ** 21
    for call in (_attend, _cross, _append, _commit):
        for page in (64, 128, 1 << 20):
            kv = _kv(page_size=page, scale_block=64, num_pages=4, max_pages_per_seq=most // page + 1)
            assert call(cuda_lib, kv, _dims()) == UNSUPPORTED
            # (one page less is accepted, and the call goes on to fail for want of a workspace or a GPU)
            kv = _kv(page_size=page, scale_block=64, num_pages=4, max_pages_per_seq=most // page)
            if call in (_attend, _cross):
                assert call(cuda_lib, kv, _dims(), q=None) == INVALID
