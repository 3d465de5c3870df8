"""How many keys a windowed call is planned for when only a bound on the lengths is given (no GPU)."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tree_verification_attention_longspec_b200", "csrc")


def test_the_plan_of_a_bound_holds_every_shorter_sequence(tmp_path):
    exe = tmp_path / "window_plan_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, os.path.join(ROOT, "tests", "window_plan_check.cpp"),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
