"""Host check of how bw_attn_paged_prefill cuts a call (prefill_cut() in
bw_paged_plan.cuh, the code that the launch runs), without a GPU: the plan
over many shapes and device sizes, and that the cases of
test_gpu_paged_paths.py go the way that they name on a device of 152 SMs."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

pytest.importorskip("torch")


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


def test_cases_go_the_way_they_name(check):
    import test_gpu_paged_paths as paths

    def path(n_tokens, n_seqs, H, Hkv, longest, window, sinks):
        return check(n_tokens, n_seqs, H // Hkv, Hkv, longest, window, sinks,
                     152)[0]

    def table(lens, page):  # the width that Cache makes
        return (-(-max(lens) // page) + 1) * page

    for name, H, Hkv, n, new, _ in paths.JUMPS:
        assert path(new, 1, H, Hkv, table([n], 64), 0, 0) == name, (H, n, new)
    for name, H, Hkv, n, new, window, sinks in paths.ODD:
        assert path(new, 1, H, Hkv, table([n], 64), window, sinks) == name
    for name, H, Hkv, page, lens, new, window, sinks in paths.RANDOM:
        assert path(sum(new) + 2 * paths.LEAD, len(lens), H, Hkv,
                    table(lens, page), window, sinks) == name, (H, lens, new)
    for H, Hkv, lens, tokens, window, sinks in paths.CAPTURED:
        assert path(tokens, len(lens), H, Hkv, table(lens, 64), window,
                    sinks) == "parts"


def test_20_mib_are_enough_for_every_call():
    import ctypes

    from conftest import build_lib
    lib = ctypes.CDLL(build_lib())
    decode, prefill = (lib.bw_attn_paged_decode_workspace_bytes,
                       lib.bw_attn_paged_prefill_workspace_bytes)
    decode.restype = prefill.restype = ctypes.c_size_t
    most = 0
    for D in (64, 128):
        for Hkv in (1, 2, 3, 5, 8, 19, 38, 64):
            for G in range(1, 17):
                most = max(most, decode(4096, G * Hkv, Hkv, D))
                TQ2 = 2 * (128 // G)
                for k in (1, 2, 3, 5, 10, 19, 38, 50, 76, 152, 500):
                    for n in (k * TQ2 - 1, k * TQ2):
                        for seqs in (1, 2, 7, 4096):
                            need = prefill(n, seqs, G * Hkv, Hkv, D)
                            assert need > 0
                            most = max(most, need)
    assert most <= 20 << 20, most
