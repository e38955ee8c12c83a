"""The token side (include/tbe_tokens.h) where it once went wrong, as far as the host shows it."""
import ctypes
import os
import subprocess

from bwd_tbe_fwd_gb300 import build as tbe_build
from bwd_tbe_fwd_gb300 import tbe, tokens

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_sort_takes_a_cluster_that_can_run(tmp_path):
    """Where no cluster of 8 CTAs (or of 16) can run, a smaller one sorts, or the tokens are sorted through memory: a lookup's
    gradient is not refused for it."""
    exe = tmp_path / "sort_plans"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-x", "c++", "-I", tbe_build.CSRC,
                    os.path.join(HERE, "sanitize", "sort_plans.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "plans ok\n", r.stdout[-2000:] + r.stderr[-2000:]


def test_the_loss_refuses_what_the_header_does():
    """tokens * rows up to 2^45."""
    tbe_build.build()
    lib = tokens._bind(tbe.load())

    def problem(n, rows):
        return ctypes.byref(tokens.SoftmaxProblem(n, rows, 8, 8, 8, 8, 8, tbe.TBE_BF16, tbe.TBE_I64, 1.0))

    for n, rows in ((1 << 24, 1 << 21), (1 << 15, 1 << 30), ((1 << 14) + 1, (1 << 31) - (1 << 17) - (1 << 16))):
        assert lib.tbe_softmax_loss_workspace_size(problem(n, rows)) > 0
    A = ctypes.c_void_p(1 << 16)  # stands for an aligned buffer; the call does not get as far as using it
    for n, rows in ((1 << 24, (1 << 21) + 1), ((1 << 15) + 1, 1 << 30)):
        assert lib.tbe_softmax_loss_workspace_size(problem(n, rows)) == 0
        assert lib.tbe_softmax_loss_forward(problem(n, rows), A, A, A, A, A, A, A, 1 << 50, None, None) == tbe.TBE_ERR_UNSUPPORTED


def test_the_losss_workspace_does_not_grow_with_the_logits():
    """What the forward keeps of the logits is 256 MB or 16 bytes a token at the most, beside a copy of hidden; more tokens
    never take less."""
    tbe_build.build()
    lib = tokens._bind(tbe.load())
    for dim in (8, 64):
        for rows in (1000, 131072, 1 << 21, 1 << 24):
            last = 0
            for n in (1, 100, 256, 257, 1000, 8192, 32768, 131072, 1 << 20, 1 << 21):
                size = lib.tbe_softmax_loss_workspace_size(
                    ctypes.byref(tokens.SoftmaxProblem(n, rows, dim, dim, dim, dim, dim, tbe.TBE_BF16, tbe.TBE_I64, 1.0)))
                assert last <= size <= max(256 << 20, 16 * n) + (2 * dim + 64) * (n + 256) + 4096, (dim, rows, n)
                last = size
