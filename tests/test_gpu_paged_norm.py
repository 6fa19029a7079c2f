"""The norm of bw_qk_norm_rope_append (GB300) over all of bf16's range: heads
whose squares leave fp32's range, with and without eps, next to ordinary ones,
against 64 bits.  Tolerance as in test_gpu_paged.py: 2^-8 of the value for its
rounding and 2^-19 of the pair."""
import numpy as np
import pytest

from test_gpu_paged import THETA, as_bf16, bw, f64, norm_rope  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SIZES = [1.0, 0.0, 1e-40, 1e-38, 1e-30, 1e-22, 3e-18, 1e-15, 1e-12, 1e-5, 1e4,
         1e12, 1e18, 3e19, 1e25, 1e34, 2e37]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-33, 1e-20, 1e-5, 1e30])
@pytest.mark.parametrize("tokens", [1, 600, 2100])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_of_small_and_large_heads(bw, D, eps, tokens, in_place):
    """tokens: four warps a token, two and one.  (A head of zeros has no norm
    without eps: NaN, 0 times infinity, as the formula says.)"""
    H = Hkv = len(SIZES)
    rng = np.random.default_rng(191)
    x = rng.standard_normal((tokens, 3, H, D)) * np.array(SIZES)[:, None]
    x[:, :, 5, 3] *= 1e6  # one large value in a small head
    qkv = as_bf16(x.reshape(tokens, -1)).cuda()
    x = f64(qkv).reshape(tokens, 3, H, D)
    page = 64
    n_pages = -(-tokens // page)
    kp = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    gamma = rng.uniform(0.5, 1.5, D).astype(np.float32)
    g = torch.from_numpy(gamma).cuda()
    q = bw.bw_qk_norm_rope_append(qkv, kp, vp, table, lens, H, q_start=start,
                                  q_gamma=g, k_gamma=g, eps=eps, theta=THETA,
                                  q_out=qkv.unflatten(1, (3 * H, D))[:, :H]
                                  if in_place else None)
    assert bw.bw_device_error() == 0
    k = f64(kp.transpose(1, 2).reshape(-1, Hkv, D)[:tokens])
    e32 = float(np.float32(eps))
    for t in range(0, tokens, 1 if tokens < 9 else 97):
        for got, want in ((f64(q[t]), x[t, 0]), (k[t], x[t, 1])):
            with np.errstate(invalid="ignore"):
                z, pair = norm_rope(want, t, gamma.astype(np.float64), e32, THETA)
            if eps == 0.0:
                assert np.isnan(got[1]).all()
                got[1], z[1], pair[1] = 0.0, 0.0, 0.0
            err = np.abs(got - z)
            # below bf16's smallest normal number its steps are 2^-133
            tol = 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * pair + 2.0 ** -134
            # Values below fp32's smallest normal number against a larger eps:
            # z is r (y0 a - y1 b), a product and an fma on multiples of
            # 2^-149, each off by half of that at most, times r = 1 / sqrt(ms).
            # (Heads whose ms is below 1e-30 are brought up first.)
            ms = (want ** 2).mean(-1, keepdims=True) + e32
            with np.errstate(divide="ignore"):
                tol = tol + np.where(ms >= 1e-30, 2.0 ** -149 / np.sqrt(ms), 0.0)
            assert (err <= tol).all(), (t, np.argwhere(err > tol)[:4])
