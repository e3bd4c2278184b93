"""The routing scores' divisions go through reciprocals: 1 / x as r + r (1 - x r) and e / total as q + r (e - q total),
q = RN(e r), with fused multiply-adds.  This checks in IEEE binary32 on the CPU what that gives: the reciprocal is
correctly rounded for every significand from a correctly rounded start, and for all but 32 from one that is an ulp
off (the GPU test of the keys' bits takes those); the quotient is correctly rounded at the numerators next to rounding
midpoints and at random ones."""
import os
import subprocess

import pytest


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    src = os.path.join(os.path.dirname(__file__), "helpers", "score_div_check.c")
    exe = str(tmp_path_factory.mktemp("score") / "score_div_check")
    # -ffp-contract=off: every product and sum rounds on its own, as in the library's sources
    subprocess.run(["gcc", "-O2", "-ffp-contract=off", "-std=c11", src, "-o", exe, "-lm"], check=True)
    return exe


def test_scores_by_reciprocals_equal_division(checker):
    out = subprocess.run([checker, "3", "9", "20000000"], capture_output=True, text=True, check=True).stdout.split()
    exact, off, hard, random = [(int(out[i]), int(out[i + 1])) for i in range(0, 8, 2)]
    assert exact == (1 << 23, 0)
    assert off == (1 << 24, 33)  # 32 significands, one of them (all ones) from both sides
    assert hard[0] > 10_000_000 and hard[1] == 0
    assert random == (20_000_000, 0)
