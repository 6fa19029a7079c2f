"""The norms with 8-bit codes (GB300) where they could give way: a residual
stream that is updated in place, scales of the largest values, products that leave
fp32's range.

Forms and tolerances are those of test_gpu_norm_quant.py.
"""
import numpy as np
import pytest

from test_gpu_norm_quant import bw, check, f64, normals  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("K", [260, 2564, 2880, 3840, 5760, 6912, 11008, 13824])
@pytest.mark.parametrize("M", [5, 4096])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_in_place_is_as_into_another_buffer(bw, M, K, kind):  # noqa: F811
    """Bit for bit, on fresh inputs, at widths that leave threads without a
    vector.  A row's largest values are its last four, and x has h's sign there:
    to add x twice would show in the scale."""
    gamma = torch.ones(K, device="cuda")
    for seed in range(4):
        h = normals(seed, M, K).clamp(-3, 3)
        x = normals(seed + 50, M, K).clamp(-3, 3)
        h[:, -4:] = 8.0 + h[:, -4:].abs()
        x[:, -4:] = 8.0 + x[:, -4:].abs()
        x = x.to(kind)
        out = torch.empty_like(h)
        q, s = bw.bw_add_rms_norm_quant(x, gamma, h=h, h_out=out)
        q2, s2 = bw.bw_add_rms_norm_quant(x, gamma, h=h)
        assert torch.equal(h, out)
        assert torch.equal(s, s2) and torch.equal(q, q2)


@pytest.mark.parametrize("K", [64, 67])
@pytest.mark.parametrize("top", [2.0 ** 125, 2.0 ** 126, 1e38, 2.0 ** 127, 3.3e38])
def test_values_up_to_the_largest(bw, K, top):  # noqa: F811
    """A row that is finite has a scale, however large its values are."""
    x = normals(1, 3, K).sign()
    gamma = 1.0 + 0.25 * normals(2, K)
    gamma[K // 2] = top
    gamma[3] = -0.4 * top
    q, s = bw.bw_add_rms_norm_quant(x, gamma, eps=0.0)
    check(q, s, f64(x), f64(gamma), 0.0)
    assert (q[:, K // 2].abs() == 127).all()


def test_the_scale_is_the_quantisers(bw):  # noqa: F811
    """Rows whose norm is 1 (64 values of 1 and -1, eps 0: every step is exact):
    the same quotient as bw_quant_act's, to the bit."""
    x = normals(3, 400, 64).sign()
    for seed in range(20):
        gamma = normals(seed + 10, 64) * 10.0 ** (seed % 7 - 3)
        rows = x[seed:seed + 20]
        _, s = bw.bw_add_rms_norm_quant(rows, gamma, eps=0.0)
        _, want = bw.bw_quant_act((rows * gamma).contiguous())
        assert torch.equal(s, want)


@pytest.mark.parametrize("K", [64, 67])
@pytest.mark.parametrize("size,gain", [(2.0 ** 55, 2.0 ** 75), (2.0 ** 62, 2.0 ** 70),
                                       (2.0 ** 61, 2.0 ** 110), (1e37, 1e30),
                                       (2.0 ** 20, 2.0 ** 110)])
def test_large_rows_of_large_gains(bw, K, size, gain):  # noqa: F811
    """Their product leaves fp32's range; what the norm makes of it does not."""
    x = normals(4, 3, K).clamp(-3, 3) * size
    gamma = (1.0 + 0.25 * normals(5, K)) * gain
    q, s = bw.bw_add_rms_norm_quant(x, gamma, eps=1e-5)
    check(q, s, f64(x), f64(gamma), 1e-5)


@pytest.mark.parametrize("F", [64, 67])
@pytest.mark.parametrize("g,u", [(80, -100), (100, -120), (-75, 120), (-70, 125),
                                 (63, -120), (-66, 100)])
def test_squares_of_the_gate_beyond_the_range(bw, F, g, u):  # noqa: F811
    """relu(g)^2 u is in fp32's range where relu(g)^2 is not, on either side."""
    gu = torch.cat((normals(6, 3, F).clamp(-3, 3) * 2.0 ** g,
                    normals(7, 3, F).clamp(-3, 3) * 2.0 ** u), 1).bfloat16()
    gamma = 1.0 + 0.25 * normals(8, F)
    q, s = bw.bw_relu2_rms_norm_quant(gu, gamma, eps=0.0)
    v = np.maximum(f64(gu)[:, :F], 0) ** 2 * f64(gu)[:, F:]
    check(q, s, v, f64(gamma), 0.0, more=4)
