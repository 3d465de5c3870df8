"""How a row is split over CTAs: it fits, and on any number of SMs no more run than have a place."""
from __future__ import annotations

import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tree_verification_attention_longspec_b200", "csrc")
BF16, FP32 = 38912, 19456  # entries that a CTA's shared memory holds


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    exe = tmp_path_factory.mktemp("plan") / "sample_plan_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, os.path.join(ROOT, "tests", "sample_plan_check.cpp"),
                    "-o", str(exe)], check=True)

    def ask(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
        return [(int(a), int(b)) for a, b in zip(out[::2], out[1::2])]
    return ask


def test_known_splits(split):
    assert split([(8, 32000, FP32, 148), (32, 32000, FP32, 148), (256, 128256, BF16, 148), (64, 152064, BF16, 148),
                  (1, 1, BF16, 148), (1, 1000, FP32, 148), (1, 1 << 20, FP32, 148)]) == [
        (8, 4000), (8, 4000), (4, 32064), (4, 38016), (1, 8), (1, 1000), (8, 131072)]


def test_fewer_sms_have_fewer_places(split):
    # 32 rows in 2 places each of 148, 64 and 16 SMs: 8, 4 and (the row needs two) 2 CTAs a row
    assert [c for c, _ in split([(32, 32000, FP32, n) for n in (148, 64, 16)])] == [8, 4, 2]


def test_every_split_holds_its_row(split):
    r = np.random.default_rng(0)
    cases = [(int(2 ** r.uniform(0, 27)), int(2 ** r.uniform(0, 20)), int(r.choice([BF16, FP32])), int(r.integers(1, 200)))
             for _ in range(2000)]
    for (rows, vocab, cap, sms), (c, share) in zip(cases, split(cases)):
        assert c in (1, 2, 4, 8) and share * c >= vocab and share % 8 == 0 and share <= 1 << 17
        fewest = next(n for n in (1, 2, 4, 8) if -(-vocab // n) <= cap - 8 or n == 8)
        assert c == fewest or (c > fewest and rows * c <= 2 * sms)
