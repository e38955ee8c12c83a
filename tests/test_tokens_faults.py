"""The token side (include/tbe_tokens.h) where it once went wrong, as far as the host shows it."""
import os
import subprocess

from bwd_tbe_fwd_gb300 import build as tbe_build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_sort_takes_a_cluster_that_can_run(tmp_path):
    """Where no cluster of 8 CTAs (or of 16) can run, a smaller one sorts, or the tokens are sorted through memory: a lookup's
    gradient is not refused for it."""
    exe = tmp_path / "sort_plans"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-x", "c++", "-I", tbe_build.CSRC,
                    os.path.join(HERE, "sanitize", "sort_plans.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "plans ok\n", r.stdout[-2000:] + r.stderr[-2000:]
