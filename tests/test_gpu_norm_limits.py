"""The norms with 8-bit codes (GB300) where they could give way: a residual
stream that is updated in place.

Forms and tolerances are those of test_gpu_norm_quant.py.
"""
import pytest

from test_gpu_norm_quant import bw, normals  # noqa: F401

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
