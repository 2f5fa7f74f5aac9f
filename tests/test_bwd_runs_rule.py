"""Which layout the pre-mapping's backward takes for 16-bit x, on the host (tests/bwd_runs_check.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_faster_layout_is_taken(tmp_path):
    exe = tmp_path / "bwd_runs_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "mhc_hyper_connection_amd", "csrc"),
                    os.path.join(ROOT, "tests", "bwd_runs_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout
