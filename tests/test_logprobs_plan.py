"""What the log probabilities' launches write stays within their workspace.

Builds tests/csrc/logprobs_plan.cpp (host code only) against the library's own planner and
runs it over counts of rows, vocabularies, types and alternatives on both sides of every
rule that splits a call."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "lm_head_linear_amd", "csrc")


def test_launches_within_the_workspace(tmp_path):
    gpp = shutil.which("g++")
    if gpp is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "logprobs_plan")
    r = subprocess.run([gpp, "-O2", "-std=c++17", "-Wall", "-Wextra", "-I",
                        os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "csrc", "logprobs_plan.cpp"),
                        os.path.join(CSRC, "ops_check.cpp"), os.path.join(CSRC, "flce_check.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = {k: v for k, v in os.environ.items() if k != "FLCE_VCHUNK"}
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr
    assert "all launches within their workspace" in r.stdout
