"""The same call twice, bit for bit, whatever ran in between (GB300).

Query tiles of 128 rows whose tokens do not fill them (a number of heads that does
not divide 128): what another call's CTA left in an SM's shared memory must have no
say in the result, not even in its last bits.
"""
import pytest

from test_gpu_paged import bw  # noqa: F401
from test_gpu_paged_shared import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def large_queries(D):
    """A call whose tiles are full, of queries that leave large numbers behind."""
    c = Batch(1, 3000, [0] * 64, 8, 2, D, 64, gain=3.0)
    c.q = c.q * 3e3
    start = torch.arange(0, 65 * 16, 16, dtype=torch.int32, device="cuda")
    q = (torch.randn((64 * 16, 8, D), device="cuda") * 3e3).bfloat16()
    table = torch.zeros((64, 2), dtype=torch.int32, device="cuda")
    table[:] = c.shared_table[:2]
    kv_len = torch.full((64,), 100, dtype=torch.int32, device="cuda")

    def run(bw):
        c.run(bw)
        bw.bw_attn_paged_prefill(q, c.kp, c.vp, table, kv_len, start)

    return run


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [3, 5, 7])
@pytest.mark.parametrize("n", [10, 100])
def test_shared_prefix(bw, D, G, n):  # noqa: F811
    c = Batch(7, 1099, [b * 37 % 200 for b in range(n)], 4 * G, 4, D, 128, gain=3.0)
    c.q = c.q * 2.0
    other = large_queries(D)
    want = c.run(bw)
    c.check(want)
    for i in range(40):
        if i % 3:
            other(bw)
        assert torch.equal(c.run(bw), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [3, 5, 7])
@pytest.mark.parametrize("tokens,length", [(500, 500), (2500, 2500), (60, 9000)])
def test_prompts(bw, D, G, tokens, length):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(G + tokens)

    def normal(*shape, gain=1.0):
        return (gain * torch.randn(shape, device="cuda", generator=gen)).bfloat16()

    pages = -(-length // 64)
    kp, vp = normal(pages, 4, 64, D, gain=3.0), normal(pages, 4, 64, D)
    table = torch.randperm(pages, device="cuda", generator=gen).int()[None].contiguous()
    kv_len = torch.tensor([length], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    q = normal(tokens, 4 * G, D, gain=2.0)
    other = large_queries(D)
    want = bw.bw_attn_paged_prefill(q, kp, vp, table, kv_len, start)
    for i in range(40):
        if i % 3:
            other(bw)
        assert torch.equal(bw.bw_attn_paged_prefill(q, kp, vp, table, kv_len, start),
                           want)
