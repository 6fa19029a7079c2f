"""Attention behind a shared prefix (GB300) where no sequence reaches the end of
the prefix: what lies beyond the longest one may hold anything.

Forms and tolerances are those of test_gpu_paged_shared.py.
"""
import pytest

from test_gpu_paged import bw  # noqa: F401
from test_gpu_paged_shared import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def short_batch(D, n, longest, page=16, shared=900):
    """Sequences of 0 to `longest` positions of a prefix of 900, NaN behind."""
    own = [None if b % 7 == 3 else longest - b * 5 % longest - shared for b in range(n)]
    assert max(shared + x for x in own if x is not None) == longest
    c = Batch(longest, shared, own, 8, 2, D, page)
    for i, p in enumerate(c.common):
        keep = min(max(longest - i * page, 0), page)
        for pool in (c.kp, c.vp):
            pool[int(p), :, keep:] = float("nan")
    return c


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("longest", [1, 100, 127, 128, 129, 384, 500, 899])
def test_rows_that_nobody_sees(bw, D, n, longest):  # noqa: F811
    c = short_batch(D, n, longest)
    out = c.run(bw)
    assert bw.bw_device_error() == 0
    assert out.isfinite().all()
    c.check(out)


@pytest.mark.parametrize("D", [64, 128])
def test_entries_that_nobody_uses(bw, D):  # noqa: F811
    """Pages of positions that no sequence reaches are not looked up."""
    c = short_batch(D, 9, 200)
    c.shared_table[-(-200 // 16):] = c.n_pages + 7
    c.check(c.run(bw))
    assert bw.bw_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("length", [-1, 2 ** 31 - 1])
def test_a_bad_length_reaches_nothing(bw, D, length):  # noqa: F811
    """Reported, zeros; the others are as without it."""
    c = short_batch(D, 9, 200)
    c.kv_len[1] = length
    out = c.run(bw)
    with pytest.raises(bw.BwError):
        bw.bw_device_error()
    assert (out[1] == 0).all()
    c.check(out, seqs=[0] + list(range(2, 9)))


@pytest.mark.parametrize("n", [6, 40])
def test_a_replayed_graph_follows_the_longest(bw, n):  # noqa: F811
    """Down to sequences that are all empty, and up again past the prefix."""
    c = Batch(3, 640, [30 + i for i in range(n)], 8, 2, 128, 32)
    ws = torch.zeros(bw.bw_attn_paged_shared_workspace_bytes(n, 8, 2, 128),
                     dtype=torch.uint8, device="cuda")
    out = torch.zeros((n, 8, 128), dtype=torch.bfloat16, device="cuda")
    c.run(bw, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(bw, out=out, workspace=ws)
    k, v, lens = c.k, c.v, c.lens
    for most in (2000, 640, 300, 1, 0, 641, 2000):
        c.lens = [min(m, max(0, most - b % 3)) for b, m in enumerate(lens)]
        c.kv_len.copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.k = [x[:m] for x, m in zip(k, c.lens)]
        c.v = [x[:m] for x, m in zip(v, c.lens)]
        graph.replay()
        c.check(out)
    assert bw.bw_device_error() == 0
