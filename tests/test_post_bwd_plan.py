"""The launches of hc_post's backward, replayed on the host (tests/post_bwd_plan_check.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_size_taken_can_be_launched(tmp_path):
    exe = tmp_path / "post_bwd_plan_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "mhc_hyper_connection_amd", "csrc"),
                    os.path.join(ROOT, "tests", "post_bwd_plan_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout
