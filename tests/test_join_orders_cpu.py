"""The selection of the join over bounded tiles in any order of its threads.

Builds tests/csrc/sparse_join.cpp (host code only) against the kernel's own header and
runs it: token lists that overflow once and many times, the threads of a token one at a
time between barriers, in rising, falling and shuffled order. Every order has to give the
largest keys within the stated number of passes."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_order_of_threads_selects_the_same(tmp_path):
    gpp = shutil.which("g++")
    if gpp is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "sparse_join")
    r = subprocess.run([gpp, "-O2", "-std=c++17", "-pthread", "-Wall", "-Wextra",
                        "-Wno-unknown-pragmas",
                        os.path.join(ROOT, "tests", "csrc", "sparse_join.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr
    assert "the same alternatives in every order" in r.stdout
