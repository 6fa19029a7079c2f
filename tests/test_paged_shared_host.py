"""Host-side checks of the attention over a shared prefix, without a GPU: the
argument checks of the C ABI and the plan of its parts."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT, build_lib
from test_paged_host import A, INVALID, KV, MISALIGNED, SHAPE, F, I, L, P, Z, kv


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(build_lib())
    lib.bw_attn_paged_shared.argtypes = [P, L, I, P, P, I, P, F, P, L, P, Z, P]
    lib.bw_attn_paged_shared_workspace_bytes.restype = Z
    lib.bw_attn_paged_decode_workspace_bytes.restype = Z
    return lib


def call(lib, cache=None, **kw):
    a = dict(q=A, q_ld=1024, H=8, table=A, pages=3, length=A, scale=0.1,
             out=2 * A, out_ld=1024, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    c = cache if cache is not None else kv()
    return lib.bw_attn_paged_shared(
        a["q"], a["q_ld"], a["H"], ctypes.byref(c) if isinstance(c, KV) else None,
        a["table"], a["pages"], a["length"], a["scale"], a["out"], a["out_ld"],
        a["ws"], a["ws_bytes"], None)


def test_checks(lib):
    assert call(lib, False) == INVALID
    for name in ("q", "table", "length", "out", "ws"):
        assert call(lib, **{name: None}) == INVALID
    for name in ("k_pages", "v_pages", "page_table", "kv_len"):
        assert call(lib, kv(**{name: None})) == INVALID
    assert call(lib, pages=0) == INVALID
    assert call(lib, pages=-1) == INVALID
    assert call(lib, pages=(1 << 20) + 1) == SHAPE
    assert call(lib, kv(page_size=48)) == SHAPE
    assert call(lib, kv(head_dim=96)) == SHAPE
    assert call(lib, kv(n_seqs=4097)) == SHAPE
    assert call(lib, H=7) == INVALID
    assert call(lib, H=34) == SHAPE
    assert call(lib, q_ld=1016) == INVALID
    assert call(lib, out_ld=1016) == INVALID
    assert call(lib, q_ld=1028) == MISALIGNED
    assert call(lib, out_ld=1028) == MISALIGNED
    assert call(lib, q_ld=1 << 31) == INVALID
    assert call(lib, out=A) == INVALID  # q itself
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, scale=scale) == INVALID
    for name, off in (("q", 8), ("table", 2), ("length", 2), ("ws", 8)):
        assert call(lib, **{name: A + off}) == MISALIGNED
    assert call(lib, out=2 * A + 8) == MISALIGNED
    need = lib.bw_attn_paged_shared_workspace_bytes(4, 8, 2, 128)
    assert call(lib, ws_bytes=need - 1) == INVALID


def test_workspace(lib):
    ws = lib.bw_attn_paged_shared_workspace_bytes
    assert ws(0, 20, 5, 128) == ws(4097, 20, 5, 128) == 0
    assert ws(4, 20, 3, 128) == ws(4, 20, 5, 96) == ws(4, 34, 2, 128) == 0
    for n in (1, 64, 4096):
        assert ws(n, 20, 5, 128) > n * 20 * 130 * 4


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_plan(tmp_path):
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-o", exe, os.path.join(
        ROOT, "tests", "paged_shared_check.cpp")], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r
    assert "plans" in r.stdout
