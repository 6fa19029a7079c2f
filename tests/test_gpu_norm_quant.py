"""The residual's addition with the RMS norm and 8-bit codes, and its gated
form, on a GB300 against plain 64-bit forms.

Tolerances (u = 2^-24): v = h + x and relu(g)^2 u are fp32 (h + x exact to one
rounding, so h_out is compared bit for bit; the product has two: 2 u).  The sum
of squares adds at most 64 values of a thread and 10 exchanges: 74 u, half of
it after the root; the root, the mean, eps, the quotient and gamma's product
add less than 8 u more: a scale is off by at most 50 u of its value, and t s by
as much twice: a code is within 1/2 + 127 x 100 u of it.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
CODE = 0.5 + 127 * 100 * U


@pytest.fixture(scope="module")
def bw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_lib
    build_lib()
    import bit_gemv_bitlinear_gb300 as bw
    return bw


def f64(t):
    return t.double().cpu().numpy()


def check(q, s, v, gamma, eps, more=0.0):
    """q, s of rows v (64 bits); more: what v's own rounding adds, in u."""
    rms = np.sqrt((v * v).mean(1, keepdims=True) + eps)
    t = np.divide(v, rms, out=np.zeros_like(v), where=rms > 0) * gamma
    scale = 127.0 / np.maximum(np.abs(t).max(1, keepdims=True), 1e-5)
    got = f64(s)[:, None]
    assert (np.abs(got - scale) <= (50 + more) * U * scale).all()
    assert (np.abs(f64(q) - t * scale) <= CODE + 127 * 2 * more * U).all()


def normals(seed, *shape):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()


WIDTHS = [1, 3, 4, 32, 33, 127, 128, 1021, 2560, 4096, 4100, 6912, 8192, 16384,
          16388, 65536]


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(bw, K, kind, residual):
    M = 5
    x = normals(K, M, K).to(kind)
    gamma = 1.0 + 0.25 * normals(K + 1, K)
    h = 3.0 * normals(K + 2, M, K) if residual else None
    before = h.clone() if residual else None
    q, s = bw.bw_add_rms_norm_quant(x, gamma, h=h, eps=1e-5)
    assert q.dtype is torch.int8 and tuple(q.shape) == (M, K)
    v = x.float()
    if residual:
        v = before + v
        assert torch.equal(h, v)  # in place
    check(q, s, f64(v), f64(gamma), 1e-5)


@pytest.mark.parametrize("M", [1, 2, 97, 4096])
def test_rows(bw, M):
    K = 260
    x = normals(M, M, K)
    gamma = normals(1, K)
    h = normals(M + 7, M, K)
    out = torch.full_like(h, 5.0)
    kept = h.clone()
    q, s = bw.bw_add_rms_norm_quant(x, gamma, h=h, h_out=out, eps=0.0)
    assert torch.equal(h, kept) and torch.equal(out, h + x)
    check(q, s, f64(h + x), f64(gamma), 0.0)


@pytest.mark.parametrize("F", [1, 2, 31, 64, 1021, 6912, 8192, 16384, 65536])
def test_gate(bw, F):
    gu = normals(F, 3, 2 * F).bfloat16()
    gamma = 1.0 + 0.25 * normals(F + 1, F)
    q, s = bw.bw_relu2_rms_norm_quant(gu, gamma, eps=1e-6)
    g, u = f64(gu)[:, :F], f64(gu)[:, F:]
    check(q, s, np.maximum(g, 0) ** 2 * u, f64(gamma), 1e-6, more=4)


@pytest.mark.parametrize("off,pad", [(0, 8), (1, 0), (1, 7), (4, 4)])
def test_strided_rows(bw, off, pad):
    """Rows of a wider buffer, at places that vectors do not fit; the codes of
    other rows and what lies around them stay as they are."""
    M, K = 7, 132
    gamma = normals(2, K)
    for kind in (torch.bfloat16, torch.float32):
        x = normals(3, M, off + K + pad).to(kind)[:, off:off + K]
        h = normals(4, M * K + 1)[1:].view(M, K)
        q = torch.full((M * K + 2,), 77, dtype=torch.int8, device="cuda")
        want = h + x.float()
        _, s = bw.bw_add_rms_norm_quant(x, gamma, h=h, q=q[1:-1].view(M, K))
        assert torch.equal(h, want)
        check(q[1:-1].view(M, K), s, f64(want), f64(gamma), 1e-5)
        assert q[0] == 77 and q[-1] == 77
    gu = normals(5, M, off + 2 * K + pad).bfloat16()[:, off:off + 2 * K]
    q, s = bw.bw_relu2_rms_norm_quant(gu, gamma)
    g, u = f64(gu)[:, :K], f64(gu)[:, K:]
    check(q, s, np.maximum(g, 0) ** 2 * u, f64(gamma), 1e-5, more=4)


@pytest.mark.parametrize("K", [64, 67])
@pytest.mark.parametrize("size", [2.0 ** -126, 1e-30, 1e-12, 1e12, 2.0 ** 63, 1e37])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_range(bw, K, size, eps):
    """Squares that leave fp32's range on either side."""
    x = normals(6, 3, K).clamp(-3, 3) * size
    x[1] = 0.0
    x[1, K // 2] = size
    gamma = 1.0 + 0.25 * normals(7, K)
    q, s = bw.bw_add_rms_norm_quant(x, gamma, eps=eps)
    check(q, s, f64(x), f64(gamma), eps)


@pytest.mark.parametrize("K", [64, 67])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_rows_of_zeros(bw, K, eps):
    x = torch.zeros(3, K, device="cuda")
    x[1] = 1.0
    q, s = bw.bw_add_rms_norm_quant(x, torch.ones(K, device="cuda"), eps=eps)
    assert (q[0] == 0).all() and (q[2] == 0).all() and (q[1] == 127).all()
    assert float(s[0]) == pytest.approx(127e5, rel=1e-6)


@pytest.mark.parametrize("K", [64, 67])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite(bw, K, bad):
    """A scale of NaN and codes of 0 in that row alone; the sum is kept."""
    x = normals(8, 4, K)
    h = normals(9, 4, K)
    x[1, 5] = bad
    h[3, K - 1] = bad
    gamma = torch.ones(K, device="cuda")
    out = torch.empty_like(h)
    q, s = bw.bw_add_rms_norm_quant(x, gamma, h=h, h_out=out)
    assert s.isnan().tolist() == [False, True, False, True]
    assert (q[1] == 0).all() and (q[3] == 0).all()
    assert torch.equal(out.nan_to_num(7.0), (h + x).nan_to_num(7.0))
    check(q[::2], s[::2], f64(h + x)[::2], f64(gamma), 1e-5)
    gu = normals(10, 4, 2 * K).bfloat16()
    gu[0, 3] = bad
    gu[2, K + 3] = bad
    gu[2, 3] = 1.0
    gu[3, 7], gu[3, K + 7] = 3e38, 3.0  # a product beyond fp32
    q, s = bw.bw_relu2_rms_norm_quant(gu, gamma)
    # relu(-inf) is 0, and 0 u is 0
    assert s.isnan().tolist() == [bad != float("-inf"), False, True, True]
    assert (q[2] == 0).all() and (q[3] == 0).all()


def test_feeds_the_projection(bw):
    """What bw_quant_act gives for the norm in fp32 differs by a code at most."""
    x = normals(11, 6, 2560)
    gamma = 1.0 + 0.1 * normals(12, 2560)
    t = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * gamma
    q, s = bw.bw_add_rms_norm_quant(x, gamma)
    q2, s2 = bw.bw_quant_act(t)
    assert int((q.int() - q2.int()).abs().max()) <= 1
    assert torch.allclose(s, s2, rtol=100 * U, atol=0.0)


def test_captured_and_on_another_stream(bw):
    x = normals(13, 9, 640)
    gamma = 1.0 + 0.1 * normals(14, 640)
    h = normals(15, 9, 640)
    q = torch.zeros(9, 640, dtype=torch.int8, device="cuda")
    s = torch.zeros(9, device="cuda")
    out = torch.zeros_like(h)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    bw.bw_add_rms_norm_quant(x, gamma, h=h, h_out=out, q=q, s=s, stream=side)
    side.synchronize()
    with torch.cuda.graph(graph):
        bw.bw_add_rms_norm_quant(x, gamma, h=h, h_out=out, q=q, s=s)
    for seed in (16, 17):
        x.copy_(normals(seed, 9, 640))
        graph.replay()
        check(q, s, f64(h + x), f64(gamma), 1e-5)


def test_refusals(bw):
    x, g = normals(1, 2, 64), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        bw.bw_add_rms_norm_quant(x, g[:63])
    with pytest.raises(ValueError):
        bw.bw_add_rms_norm_quant(x.t(), torch.ones(2, device="cuda"))
    with pytest.raises(TypeError):
        bw.bw_add_rms_norm_quant(x.half(), g)
    with pytest.raises(ValueError):
        bw.bw_add_rms_norm_quant(x, g, h_out=x.clone())
    with pytest.raises(ValueError):
        bw.bw_add_rms_norm_quant(x, g, h=normals(2, 3, 64))
    with pytest.raises(ValueError):
        bw.bw_relu2_rms_norm_quant(x[:, :63].bfloat16(), g)
    with pytest.raises(bw.BwError):
        bw.bw_add_rms_norm_quant(x, g, eps=-1.0)
    with pytest.raises(bw.BwError):
        bw.bw_add_rms_norm_quant(x, g, h=normals(2, 2, 64), h_out=x)
    with pytest.raises(ValueError):
        bw.bw_add_rms_norm_quant(x, g, q=torch.zeros(2, 65, dtype=torch.int8, device="cuda"))
    assert bw.bw_device_error() == 0
