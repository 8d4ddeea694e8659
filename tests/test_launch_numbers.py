"""The numbers that tag a launch's words in shared scratch, on the host (no
GPU): tests/launch_number_check.cpp against scratch_state.hpp with g++."""
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_launch_numbers():
    src = os.path.join(ROOT, "tests", "launch_number_check.cpp")
    inc = os.path.join(ROOT, "prefix_scan_amd", "csrc")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "launch_number_check")
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", inc, "-o", exe, src], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr + r.stdout
