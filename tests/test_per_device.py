"""What the launchers set up once per device (tests/host/per_device.cpp, a host program)."""
import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routing_dispatch_expert_router_gb300", "csrc")


def test_a_value_per_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "per_device")
    src = os.path.join(ROOT, "tests", "host", "per_device.cpp")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, src, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_launchers_keep_nothing_for_all_devices_at_once():
    """A plain static set at the first launch would hold for every device of the process."""
    for path in glob.glob(os.path.join(CSRC, "grouped_gemm*.cu")):
        with open(path) as f:
            text = f.read()
        assert not re.search(r"static (bool|int) \w+ = (false|0);", text), path
