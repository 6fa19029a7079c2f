"""The shared prefix's weights keep the bits that the decode call's have (GB300).

Tolerance (u = 2^-24): that of test_gpu_paged_shared.py with weights of two bf16
values, the first one cut off (what is left is below 2^-7 of the weight) and the
second one rounded (2^-8 of that): 2^-15 of the mean of |v| in the place of 2^-8;
and sums of 2 n terms, each step rounded or truncated: 4 n u.
"""
import pytest

from test_gpu_paged import U, bw  # noqa: F401
from test_gpu_paged_shared import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 64), (8, 2, 128), (16, 1, 64),
                                     (5, 5, 128), (12, 4, 128)])
@pytest.mark.parametrize("n", [1, 3, 40, 70])
@pytest.mark.parametrize("shared", [70, 128, 300, 2050])
def test_weights_of_two_values(bw, H, Hkv, D, n, shared):  # noqa: F811
    c = Batch(n + shared, shared, [b % 3 for b in range(n)], H, Hkv, D, 32)
    c.q = c.q * 2.0  # uneven weights
    got = c.run(bw)
    assert bw.bw_device_error() == 0
    for b, length in enumerate(c.lens):
        q = c.q[b].double().cpu().view(Hkv, H // Hkv, D)
        k, v = c.k[b].transpose(0, 1), c.v[b].transpose(0, 1)
        w = torch.softmax(q @ k.transpose(1, 2) / D ** 0.5, 2)
        mass = (q.abs() @ k.abs().transpose(1, 2)).amax(2, keepdim=True) / D ** 0.5
        want = w @ v
        rel = (D + 4) * 2 * U * mass + (8 + 4 * length) * U
        tol = 2 * rel * v.abs().amax(1, keepdim=True)
        tol = tol + 2.0 ** -15 * (w @ v.abs()) + 2.0 ** -8 * want.abs()
        off = (got[b].double().cpu().view_as(want) - want).abs()
        assert (off <= tol).all(), (b, length, float((off / tol).max()))
