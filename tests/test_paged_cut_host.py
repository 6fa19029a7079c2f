"""Host check of how bw_attn_paged_prefill cuts a call (prefill_cut() in
bw_paged_plan.cuh, the code that the launch runs), without a GPU: the plan
over many shapes and device sizes."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

@pytest.fixture(scope="module")
def check(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("cut") / "paged_cut_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "bit_gemv_bitlinear_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "paged_cut_check.cpp"),
                    "-o", exe], check=True)

    def run(*args):
        r = subprocess.run([exe] + [str(a) for a in args], capture_output=True,
                           text=True, timeout=120)
        assert r.returncode == 0, r.stdout
        return r.stdout.split()
    return run


def test_cuts_fit_their_workspace_and_device(check):
    assert check()[0] == "ok"
