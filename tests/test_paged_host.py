"""Host-side checks of the paged-cache calls that need no GPU: every argument
check of the C ABI, before any CUDA call, and the tile plans
(bw_paged_plan.cuh), compiled by the host compiler into
tests/paged_plan_check.cpp.  The W2A8 kernel page's §六 item 2 keeps a
preallocated KV cache whose position is read on the device; what the device
reads is checked there and tested on a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

from conftest import ROOT, build_lib

OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
P, I, L, F, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                 ctypes.c_float, ctypes.c_size_t)
A = 0x10000  # a never-dereferenced device address with every alignment


class KV(ctypes.Structure):
    _fields_ = [("k_pages", P), ("v_pages", P), ("page_table", P),
                ("kv_len", P), ("page_stride", L), ("n_pages", I),
                ("page_size", I), ("n_kv_heads", I), ("head_dim", I),
                ("n_seqs", I), ("max_pages", I)]


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(build_lib())
    lib.bw_qk_norm_rope_append.argtypes = [P, L, I, P, I, P, P, F, F, P, P, L, P]
    lib.bw_attn_paged_decode.argtypes = [P, L, I, P, F, I, I, P, L, I, P, Z, P]
    lib.bw_attn_paged_prefill.argtypes = [P, L, I, P, I, P, F, I, I, P, L, P, Z, P]
    lib.bw_attn_paged_decode_workspace_bytes.restype = Z
    lib.bw_attn_paged_prefill_workspace_bytes.restype = Z
    return lib


def kv(**kw):
    f = dict(k_pages=A, v_pages=A, page_table=A, kv_len=A,
             page_stride=2 * 16 * 128, n_pages=3, page_size=16, n_kv_heads=2,
             head_dim=128, n_seqs=4, max_pages=5)
    f.update(kw)
    return KV(**f)


def append(lib, cache=None, **kw):
    a = dict(qkv=A, qkv_ld=12 * 128, n=4, q_start=None, H=8, gq=None, gk=None,
             eps=1e-5, theta=1e4, q_out=2 * A, q_ld=8 * 128)
    a.update(kw)
    c = cache if cache is not None else kv()
    return lib.bw_qk_norm_rope_append(
        a["qkv"], a["qkv_ld"], a["n"], a["q_start"], a["H"], a["gq"], a["gk"],
        a["eps"], a["theta"], ctypes.byref(c) if c else None, a["q_out"],
        a["q_ld"], None)


def decode(lib, cache=None, **kw):
    a = dict(q=A, q_ld=1024, H=8, scale=0.1, window=0, sinks=0, out=2 * A,
             out_ld=1024, bf16=0, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    c = cache if cache is not None else kv()
    return lib.bw_attn_paged_decode(
        a["q"], a["q_ld"], a["H"], ctypes.byref(c) if c else None, a["scale"],
        a["window"], a["sinks"], a["out"], a["out_ld"], a["bf16"], a["ws"],
        a["ws_bytes"], None)


def prefill(lib, cache=None, **kw):
    a = dict(q=A, q_ld=1024, n=9, q_start=A, H=8, scale=0.1, window=0, sinks=0,
             out=2 * A, out_ld=1024, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    c = cache if cache is not None else kv()
    return lib.bw_attn_paged_prefill(
        a["q"], a["q_ld"], a["n"], a["q_start"], a["H"],
        ctypes.byref(c) if c else None, a["scale"], a["window"], a["sinks"],
        a["out"], a["out_ld"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [append, decode, prefill])
def test_cache_checks(lib, call):
    assert call(lib, False) == INVALID  # no cache
    for name in ("k_pages", "v_pages", "page_table", "kv_len"):
        assert call(lib, kv(**{name: None})) == INVALID
        bad = A + (8 if "pages" in name else 2)
        assert call(lib, kv(**{name: bad})) == MISALIGNED
    for name in ("n_pages", "max_pages", "n_seqs", "page_size", "n_kv_heads",
                 "head_dim"):
        assert call(lib, kv(**{name: 0})) == INVALID
        assert call(lib, kv(**{name: -1})) == INVALID
    assert call(lib, kv(page_size=8, max_pages=1)) == SHAPE
    assert call(lib, kv(page_size=48)) == SHAPE
    assert call(lib, kv(page_size=512)) == SHAPE
    assert call(lib, kv(head_dim=96)) == SHAPE
    assert call(lib, kv(head_dim=256)) == SHAPE
    assert call(lib, kv(n_seqs=4097)) == SHAPE
    assert call(lib, kv(max_pages=(1 << 20) + 1)) == SHAPE
    assert call(lib, kv(max_pages=2 ** 31 - 1)) == SHAPE
    assert call(lib, kv(n_kv_heads=65), H=65) == SHAPE
    assert call(lib, kv(page_stride=2 * 16 * 128 - 8)) == INVALID
    assert call(lib, kv(page_stride=1 << 38)) == INVALID
    assert call(lib, kv(page_stride=2 * 16 * 128 + 4)) == MISALIGNED
    assert call(lib, H=7) == INVALID       # 2 key heads do not divide it
    assert call(lib, H=0) == INVALID
    assert call(lib, H=-8) == INVALID
    assert call(lib, H=34) == SHAPE        # 17 query heads to a key head


def test_append_checks(lib):
    assert append(lib, qkv=None) == INVALID
    assert append(lib, q_out=None) == INVALID
    assert append(lib, n=0) == INVALID
    assert append(lib, n=3) == INVALID                 # one row per sequence
    assert append(lib, n=(1 << 20) + 1, q_start=A) == SHAPE
    assert append(lib, qkv_ld=12 * 128 - 8) == INVALID
    assert append(lib, q_ld=8 * 128 - 8) == INVALID
    assert append(lib, qkv_ld=1 << 31) == INVALID
    assert append(lib, qkv_ld=12 * 128 + 4) == MISALIGNED
    assert append(lib, q_ld=8 * 128 + 4) == MISALIGNED
    assert append(lib, qkv=A + 8) == MISALIGNED
    assert append(lib, q_out=A + 8) == MISALIGNED
    assert append(lib, q_start=A + 2) == MISALIGNED
    assert append(lib, gq=A + 4) == MISALIGNED
    assert append(lib, gk=A + 4) == MISALIGNED
    assert append(lib, eps=-1.0) == INVALID
    assert append(lib, eps=float("nan")) == INVALID
    assert append(lib, theta=0.5) == INVALID
    assert append(lib, theta=float("inf")) == INVALID
    assert append(lib, theta=float("nan")) == INVALID
    assert append(lib, q_out=A) == INVALID             # in place, other stride


@pytest.mark.parametrize("call", [decode, prefill])
def test_attention_checks(lib, call):
    assert call(lib, q=None) == INVALID
    assert call(lib, out=None) == INVALID
    assert call(lib, ws=None) == INVALID
    assert call(lib, ws_bytes=0) == INVALID
    assert call(lib, ws=A + 8) == MISALIGNED
    assert call(lib, q=A + 8) == MISALIGNED
    assert call(lib, out=A + 8) == MISALIGNED
    assert call(lib, q_ld=1016) == INVALID
    assert call(lib, out_ld=1016) == INVALID
    assert call(lib, q_ld=1028) == MISALIGNED
    assert call(lib, out_ld=1028) == MISALIGNED
    assert call(lib, q_ld=1 << 31) == INVALID
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert call(lib, scale=bad) == INVALID
    assert call(lib, window=-1) == INVALID
    assert call(lib, sinks=-1) == INVALID


def test_prefill_checks(lib):
    assert prefill(lib, q_start=None) == INVALID
    assert prefill(lib, q_start=A + 2) == MISALIGNED
    assert prefill(lib, n=0) == INVALID
    assert prefill(lib, n=(1 << 20) + 1) == SHAPE
    assert prefill(lib, out=A) == INVALID  # q itself


@pytest.mark.parametrize("bf16", [0, 1])
def test_decode_checks(lib, bf16):
    assert decode(lib, out=A, bf16=bf16) == INVALID  # q itself


def test_workspace_sizes(lib):
    d, p = (lib.bw_attn_paged_decode_workspace_bytes,
            lib.bw_attn_paged_prefill_workspace_bytes)
    assert d(1, 20, 5, 128) > 0 and p(9, 1, 20, 5, 128) > 0
    assert d(0, 20, 5, 128) == 0 and d(4097, 20, 5, 128) == 0
    for bad in ((20, 3, 128), (20, 0, 128), (17, 1, 128), (20, 5, 80),
                (65, 65, 64)):
        assert d(1, *bad) == 0 and p(9, 1, *bad) == 0
    assert p(0, 1, 20, 5, 128) == 0 and p((1 << 20) + 1, 1, 20, 5, 128) == 0


def test_tile_plans_hold_what_is_seen(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "paged_plan_check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-I", os.path.join(ROOT, "bit_gemv_bitlinear_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "paged_plan_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("ok "), r.stdout
