"""Shares of a ragged product's reduction (tests/host/ragged_shares.cpp, a host program), up to the
row limit of the interface."""
import math
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_shares_up_to_the_row_limit(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "ragged_shares")
    csrc = os.path.join(ROOT, "routing_dispatch_expert_router_gb300", "csrc")
    trap = "signed-integer-overflow,float-cast-overflow"
    r = subprocess.run([cxx, "-std=c++17", "-O1", f"-fsanitize={trap}", "-fsanitize-undefined-trap-on-error",
                        "-I", csrc, os.path.join(ROOT, "tests", "host", "ragged_shares.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout.splitlines()[-1:])
    rows = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert max(nk for _, nk, _, _ in rows) > 2 ** 25
    for most, nk, tile, got in rows:
        least = max(2, int(math.sqrt(nk * tile * 0.02)))
        want = 1 if nk < 24 else min(max(nk // least, 1), most)
        # (the root in 32 bits may lie the other side of a whole number)
        near = {min(max(nk // max(2, least + d), 1), most) for d in (-1, 0, 1)} if nk >= 24 else {1}
        assert got == want or got in near, (most, nk, tile, got, want)
