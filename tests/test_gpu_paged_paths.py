"""bw_attn_paged_prefill (GB300) by the way a call is cut: items of one query
tile ("one"), items of two ("two"), and items of two whose key axis is cut into
parts that a second kernel joins ("parts").  The tolerances are those of
test_gpu_paged.py, whose caches these are.
"""
import numpy as np
import pytest

from test_gpu_paged import Cache, as_bf16, bw, f64  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# ---------------------------------------------------------------------------
# a score far above all before it
# ---------------------------------------------------------------------------

JUMPS = [
    # path, H, Hkv, positions, new tokens, the position that stands out: tile
    # 1's first half and second half; the same; a part's second tile (12000
    # positions are 94 tiles in 16 parts, the one of tiles 17 to 22 holds 18)
    ("one", 1, 1, 300, 1, 150),
    ("one", 1, 1, 300, 1, 200),
    ("one", 4, 1, 330, 60, 200),
    ("two", 16, 1, 1600, 1300, 150),
    ("two", 16, 1, 1600, 1300, 200),
    ("parts", 1, 1, 12000, 1, 18 * 128 + 20),
    ("parts", 16, 1, 12000, 5, 18 * 128 + 100),
]


@pytest.mark.parametrize("path,H,Hkv,n,new,at", JUMPS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("jump", [60, 100, 300])
def test_a_jump_clears_what_was_summed(bw, path, H, Hkv, n, new, at, D, jump):
    """Every score is 0 but one position's, which is `jump` (nats): the answer
    is that position's values.  From 87.4 on the factor of what was summed
    before is 0 in fp32, for every row of a warp at once.

    The others weigh n e^-60 < 2^-70 in all; the weight of the one is rounded
    from within a few 2^-24 of 1, and dividing and rounding to bf16 leaves
    2^-8 of the value."""
    c = Cache(131, [n], Hkv, D, 64)
    c.kp.zero_()
    page = int(c.table[0, at // 64])
    c.kp[page, :, at % 64, 0] = 8.0
    q = torch.zeros((new, H, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = jump / 8
    st = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    out = bw.bw_attn_paged_prefill(q, *c.args, st, scale=1.0)
    one = bw.bw_attn_paged_decode(q[-1:], *c.args, scale=1.0)
    assert bw.bw_device_error() == 0
    want = c.vp[page, :, at % 64].double().repeat_interleave(H // Hkv, 0)
    for got in (out, one):
        err = (got.double() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + 1e-18).all(), float(err.max())
