"""Host-side checks of the calls between a served layer's projections, without
a GPU: every argument check of the C ABI comes before any CUDA call."""
import ctypes

import pytest

from conftest import build_lib

OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
P, I, L, F, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                 ctypes.c_float, ctypes.c_size_t)
A = 0x10000  # a never-dereferenced device address with every alignment


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(build_lib())
    lib.bw_add_rms_norm_quant.argtypes = [P, I, L, P, P, P, F, I, I, P, P, P]
    lib.bw_relu2_rms_norm_quant.argtypes = [P, L, P, F, I, I, P, P, P]
    lib.bw_lora_workspace_bytes.restype = Z
    lib.bw_lora_add.argtypes = [P] * 6 + [I] * 5 + [P, L, P, L, P, Z, P]
    return lib


def norm(lib, **kw):
    a = dict(x=A, bf16=1, ld=64, h=2 * A, h_out=2 * A, gamma=A, eps=1e-5, M=4,
             K=64, q=A, s=A)
    a.update(kw)
    return lib.bw_add_rms_norm_quant(
        a["x"], a["bf16"], a["ld"], a["h"], a["h_out"], a["gamma"], a["eps"],
        a["M"], a["K"], a["q"], a["s"], None)


def gate(lib, **kw):
    a = dict(x=A, ld=128, gamma=A, eps=1e-5, M=4, K=64, q=A, s=A)
    a.update(kw)
    return lib.bw_relu2_rms_norm_quant(a["x"], a["ld"], a["gamma"], a["eps"],
                                       a["M"], a["K"], a["q"], a["s"], None)


@pytest.mark.parametrize("call", [norm, gate])
def test_norm_checks(lib, call):
    for name in ("x", "gamma", "q", "s"):
        assert call(lib, **{name: None}) == INVALID
    for name in ("M", "K"):
        assert call(lib, **{name: 0}) == INVALID
        assert call(lib, **{name: -1}) == INVALID
    assert call(lib, M=4097) == SHAPE
    assert call(lib, K=65537, ld=1 << 18) == SHAPE
    assert call(lib, ld=63) == INVALID
    assert call(lib, ld=1 << 31) == INVALID
    assert call(lib, ld=-64) == INVALID
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(lib, eps=eps) == INVALID
    assert call(lib, gamma=A + 2) == MISALIGNED
    assert call(lib, s=A + 2) == MISALIGNED
    assert call(lib, x=A + 1) == MISALIGNED


def test_norm_residual_checks(lib):
    assert norm(lib, h=None) == INVALID          # h_out without h
    assert norm(lib, h_out=None) == INVALID      # and h without h_out
    assert norm(lib, h_out=A, x=A) == INVALID    # x is not h_out
    assert norm(lib, bf16=0, x=A + 2) == MISALIGNED
    assert norm(lib, h=2 * A + 2) == MISALIGNED
    assert norm(lib, h_out=2 * A + 2) == MISALIGNED
    assert gate(lib, ld=127) == INVALID          # gate and up


def lora(lib, **kw):
    a = dict(x=A, s=A, A=A, B=A, scale=A, adapter=A, n=3, M=4, N=40, K=64, R=16,
             y=A, y_ld=40, out=2 * A, out_ld=40, ws=A, ws_bytes=1 << 30)
    a.update(kw)
    return lib.bw_lora_add(
        a["x"], a["s"], a["A"], a["B"], a["scale"], a["adapter"], a["n"],
        a["M"], a["N"], a["K"], a["R"], a["y"], a["y_ld"], a["out"],
        a["out_ld"], a["ws"], a["ws_bytes"], None)


def test_lora_checks(lib):
    for name in ("x", "s", "A", "B", "adapter", "y", "out", "ws"):
        assert lora(lib, **{name: None}) == INVALID
    for name in ("n", "M", "N", "K", "R"):
        assert lora(lib, **{name: 0}) == INVALID
        assert lora(lib, **{name: -8}) == INVALID
    assert lora(lib, M=4097) == SHAPE
    assert lora(lib, N=(1 << 24) + 1, y_ld=1 << 25, out_ld=1 << 25) == SHAPE
    assert lora(lib, K=65540) == SHAPE
    assert lora(lib, K=66) == SHAPE
    assert lora(lib, R=12) == SHAPE
    assert lora(lib, R=136) == SHAPE
    assert lora(lib, n=65537) == SHAPE
    for name in ("y_ld", "out_ld"):
        assert lora(lib, **{name: 39}) == INVALID
        assert lora(lib, **{name: 1 << 31}) == INVALID
    assert lora(lib, out=A, out_ld=48) == INVALID  # in place: one stride
    need = lib.bw_lora_workspace_bytes(4, 16)
    assert need == 4 * 16 * 4
    assert lora(lib, ws_bytes=need - 1) == INVALID
    for name, off in (("x", 2), ("s", 2), ("A", 8), ("B", 8), ("scale", 2),
                      ("adapter", 2), ("y", 1), ("out", 1), ("ws", 8)):
        base = 2 * A if name == "out" else A
        assert lora(lib, **{name: base + off}) == MISALIGNED


def test_lora_workspace(lib):
    ws = lib.bw_lora_workspace_bytes
    assert ws(0, 16) == ws(-1, 16) == ws(4097, 16) == 0
    assert ws(1, 0) == ws(1, 12) == ws(1, 136) == 0
    assert ws(1, 8) == 64 and ws(4096, 128) == 4096 * 128 * 4


def test_binding_refuses_before_the_call():
    torch = pytest.importorskip("torch")
    build_lib()
    import bit_gemv_bitlinear_gb300 as bw
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        bw.bw_add_rms_norm_quant(x, torch.ones(64))
    with pytest.raises(TypeError):
        bw.bw_add_rms_norm_quant(None, torch.ones(64))
    with pytest.raises(ValueError):
        bw.bw_relu2_rms_norm_quant(x.bfloat16(), torch.ones(32))
    with pytest.raises(ValueError):
        bw.bw_lora_add(x.bfloat16(), x.to(torch.int8), x[:, 0], x, x, x)
    assert bw.bw_lora_workspace_bytes(2, 16) == 128
