"""What calls over a paged key-value cache (GB300) find in device memory that
the host cannot check: reported by bit 256 of the device error word, and
without harm for the calls after.  Every case stays within the buffers.
"""
import pytest

from test_gpu_paged import bw, take_bad  # noqa: F401
from test_gpu_paged_long import Long, check_means

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("words", [
    [1], [3], [200], [10 ** 6], [2 ** 31 - 1], [-1], [-40], [-304], [-500],
    [7, 1], [1, 1], [0x01010101] * 64, [-1] * 64])
@pytest.mark.parametrize("lens", [[240001], [777, 0, 50]])
def test_a_workspace_that_was_not_zeroed_is_reported(bw, words, lens):
    """Long calls (some units claimed) and short ones; the next call on the
    same workspace is right again."""
    H, Hkv, D = 32, 8, 128
    c = Long(171, lens, Hkv, D, 256)
    n = len(lens)
    q = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros((bw.bw_attn_paged_decode_workspace_bytes(n, H, Hkv, D),),
                     dtype=torch.uint8, device="cuda")
    ws.view(torch.int32)[:len(words)] = torch.tensor(words, dtype=torch.int32,
                                                     device="cuda")
    bw.bw_attn_paged_decode(q, *c.args, workspace=ws)
    torch.cuda.synchronize()
    take_bad(bw)
    for _ in range(2):
        out = bw.bw_attn_paged_decode(q, *c.args, workspace=ws)
        assert bw.bw_device_error() == 0
        check_means(c, out, H // Hkv, 0, 0)


@pytest.mark.parametrize("lens,tokens,window", [
    ([20000, 300, 40, 900], 30, 0),         # the key axis in parts
    ([20000, 300, 40, 900], 30, 64),        # items of one query tile
    ([3000, 3000, 3000, 3000], 2600, 0),    # items of two
])
@pytest.mark.parametrize("D", [64, 128])
def test_ranges_that_run_backwards(bw, lens, tokens, window, D):
    """q_start that decreases: ranges that overlap.  Reported, no row written,
    and the next call on the same workspace is right."""
    H, Hkv = 8, 8
    c = Long(181, lens, Hkv, D, 64)
    n = len(lens)
    q = torch.zeros((tokens, H, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros((bw.bw_attn_paged_prefill_workspace_bytes(
        tokens, n, H, Hkv, D),), dtype=torch.uint8, device="cuda")
    good = torch.tensor([0, tokens - 9, tokens - 6, tokens - 6, tokens],
                        dtype=torch.int32, device="cuda")
    want = bw.bw_attn_paged_prefill(q, *c.args, good, window=window)
    assert bw.bw_device_error() == 0
    for bad in ([0, tokens, 0, tokens, 0], [tokens, 0, 0, 0, 0],
                [0, 5, 3, 12, tokens], [0, 0, 0, tokens, tokens - 1]):
        st = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
        bw.bw_attn_paged_prefill(q, *c.args, st, window=window, out=out,
                                 workspace=ws)
        torch.cuda.synchronize()
        take_bad(bw)
        assert (out == 9.0).all()
        got = bw.bw_attn_paged_prefill(q, *c.args, good, window=window,
                                       workspace=ws)
        assert bw.bw_device_error() == 0
        assert torch.equal(got, want)
