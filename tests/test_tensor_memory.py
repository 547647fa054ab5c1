"""CTAs that share an SM never want more tensor memory than it has.

An allocation of tensor memory waits without a limit, so CTAs of clusters could wait for each other for ever; the constants
that decide it (shared memory and columns of a CTA) are checked when the kernels are compiled.  Here they are changed in a
copy of the sources, which must not compile.  Nothing of it is run.  Runs on CPU.
"""
import os
import re
import shutil
import subprocess

import pytest

from submanifold_sparse_convolution_gb300 import build as build_mod

PACKAGE = os.path.dirname(os.path.abspath(build_mod.__file__))


@pytest.mark.parametrize("source,constant,changed", [
    ("dense_blocks.cu", r"kSmallRing = R == 16 && !DUAL \? kFewRing / 2 : kFewRing;", "kSmallRing = kFewRing / 2;"),
    ("dense_blocks.cu", r"constexpr int kFewRing = 100 \* 1024;", "constexpr int kFewRing = 66 * 1024;"),
    ("dense_blocks.cu", r"constexpr int kMaxAcc = 4;", "constexpr int kMaxAcc = 16;"),
])
def test_a_change_that_wants_too_much_does_not_compile(tmp_path, source, constant, changed):
    try:
        nvcc = build_mod.nvcc()
    except RuntimeError:
        pytest.skip("nvcc not available")
    csrc = tmp_path / "package" / "csrc"
    shutil.copytree(os.path.join(PACKAGE, "csrc"), csrc)
    shutil.copytree(os.path.join(os.path.dirname(PACKAGE), "include"), tmp_path / "include")
    text = (csrc / source).read_text()
    text, count = re.subn(constant, changed, text)
    assert count == 1, "the constant is written otherwise now"
    (csrc / source).write_text(text)
    r = subprocess.run([nvcc, *build_mod.NVCC_FLAGS, "-ptx", str(csrc / source), "-o", os.devnull], capture_output=True, text=True)
    assert r.returncode != 0 and "TMEM of an SM" in r.stdout + r.stderr
