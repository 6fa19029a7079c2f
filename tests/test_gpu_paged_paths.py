"""bw_attn_paged_prefill (GB300) by the way a call is cut: items of one query
tile ("one"), items of two ("two"), and items of two whose key axis is cut into
parts that a second kernel joins ("parts").  The tolerances are those of
test_gpu_paged.py, whose caches these are.
"""
import numpy as np
import pytest

from test_gpu_paged import U, Cache, as_bf16, bw  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def exact(q, k, v, first, window, sinks, scale):
    """Tokens q [T][H][D] at positions first and on over k, v [n][Hkv][D]:
    (out, bound), [T][H][D] in 64 bits; the bound is that of attend() in
    test_gpu_paged.py for bf16 weights and a bf16 output."""
    T, H, D = q.shape
    q, k, v = q.double(), k.cuda().double(), v.cuda().double()
    G = H // k.shape[1]
    p = first + torch.arange(T, device="cuda")[:, None]
    j = torch.arange(len(k), device="cuda")[None, :]
    vis = j <= p
    if window:
        vis &= (j > p - window) | (j < sinks)
    out, bound = torch.empty_like(q), torch.empty_like(q)
    for h in range(H):
        kh, vh = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kh.T * scale).masked_fill(~vis, float("-inf"))
        mass = (q[:, h].abs() @ kh.abs().T * scale).masked_fill(~vis, 0.0)
        w = torch.softmax(s, 1)
        out[:, h] = w @ vh
        rel = (D + 4) * 2 * U * mass.amax(1) + (8 + vis.sum(1)) * U
        top = vh.abs().amax(1)[None, :].expand_as(vis).masked_fill(~vis, 0.0)
        tol = (2 * rel * top.amax(1))[:, None] + 2.0 ** -8 * (w @ vh.abs())
        bound[:, h] = tol + 2.0 ** -8 * (out[:, h].abs() + tol)
    return out, bound


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


# ---------------------------------------------------------------------------
# queries that are not finite
# ---------------------------------------------------------------------------

ODD = [
    # path, H, Hkv, positions, new tokens, window, sinks
    ("one", 4, 1, 330, 60, 0, 0),
    ("two", 16, 1, 1600, 1300, 0, 0),
    ("parts", 4, 2, 9000, 40, 0, 0),
    ("parts", 16, 1, 9000, 5, 5000, 4),
]


@pytest.mark.parametrize("path,H,Hkv,n,new,window,sinks", ODD)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), 3.0e38])
def test_a_query_that_is_not_finite_shows(bw, path, H, Hkv, n, new, window,
                                          sinks, D, odd):
    """A query with NaN or an infinity, or with scores past fp32's range: NaN
    in that token's head and nowhere else, as a softmax of such scores has it
    (whose sum is NaN), and as decode gives it.

    One position's first key value is 64, so that 3e38 times it is +infinity in
    fp32.  The other rows stay within the bound (not the same bit for bit: the
    rows of a warp decide together when a maximum follows, and the bf16 weights
    are relative to it)."""
    c = Cache(141, [n], Hkv, D, 64)
    at = n - new - 70
    c.k[0][at, :, 0] = 64.0
    c.kp[int(c.table[0, at // 64]), :, at % 64, 0] = 64.0
    rng = np.random.default_rng(142)
    q = as_bf16(rng.standard_normal((new, H, D))).cuda()
    st = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks)
    want, tol = exact(q, c.k[0], c.v[0], n - new, window, sinks, D ** -0.5)
    q[new - 1, 1, 0] = odd
    got = bw.bw_attn_paged_prefill(q, *c.args, st, **kw)
    one = bw.bw_attn_paged_decode(q[-1:], *c.args, **kw)
    assert bw.bw_device_error() == 0
    assert torch.isnan(got[new - 1, 1]).all()
    assert torch.isnan(one[0, 1]).all()
    keep = torch.ones((new, H), dtype=torch.bool, device="cuda")
    keep[new - 1, 1] = False
    err = (got.double() - want).abs()[keep]
    assert (err <= tol[keep]).all(), float((err - tol[keep]).max())
    assert torch.isfinite(one[0, keep[-1]]).all()


@pytest.mark.parametrize("path,H,Hkv,n,new,window,sinks", ODD)
@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_are_all_minus_infinity(bw, path, H, Hkv, n, new, window,
                                            sinks, D):
    """An infinite query against keys that are all below 0 there: the softmax of
    scores that are all -infinity is NaN, in that token's head alone."""
    c = Cache(143, [n], Hkv, D, 64)
    c.k[0][:, :, 0] = -1.0
    c.kp[..., 0] = -1.0
    rng = np.random.default_rng(144)
    q = as_bf16(rng.standard_normal((new, H, D))).cuda()
    st = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    kw = dict(window=window, sinks=sinks)
    want, tol = exact(q, c.k[0], c.v[0], n - new, window, sinks, D ** -0.5)
    q[new - 1, 1, 0] = float("inf")
    got = bw.bw_attn_paged_prefill(q, *c.args, st, **kw)
    one = bw.bw_attn_paged_decode(q[-1:], *c.args, **kw)
    assert bw.bw_device_error() == 0
    assert torch.isnan(got[new - 1, 1]).all()
    assert torch.isnan(one[0, 1]).all()
    keep = torch.ones((new, H), dtype=torch.bool, device="cuda")
    keep[new - 1, 1] = False
    err = (got.double() - want).abs()[keep]
    assert (err <= tol[keep]).all(), float((err - tol[keep]).max())


@pytest.mark.parametrize("lens", [[300], [5000, 70]])
@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 128), (12, 1, 64)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), float("-inf")])
def test_decode_of_a_value_that_is_not_finite(bw, lens, H, Hkv, D, bf16, odd):
    """Not finite in its dim, whatever its weight; the other dims as ever."""
    c = Cache(145, lens, Hkv, D, 64)
    at, dim = 130, 5
    c.vp[int(c.table[0, at // 64]), 0, at % 64, dim] = odd
    q = as_bf16(np.random.default_rng(146).standard_normal(
        (len(lens), H, D))).cuda()
    out = torch.full(q.shape, 9.0, device="cuda",
                     dtype=torch.bfloat16 if bf16 else torch.float32)
    bw.bw_attn_paged_decode(q, *c.args, out=out)
    assert bw.bw_device_error() == 0
    assert not torch.isfinite(out[0, :H // Hkv, dim]).any()
    for b, n in enumerate(lens):
        want, tol = exact(q[b:b + 1], c.k[b], c.v[b], n - 1, 0, 0, D ** -0.5)
        ok = (out[b].double() - want[0]).abs() <= tol[0]
        if b == 0:
            ok[:H // Hkv, dim] = True
        assert ok.all()


# ---------------------------------------------------------------------------
# random queries
# ---------------------------------------------------------------------------

LEAD = 3  # rows of no sequence, before and after

RANDOM = [
    # path, H, Hkv, page, lens, new, window, sinks
    ("one", 20, 5, 16, [509], [509], 0, 0),
    ("one", 4, 1, 64, [5000, 90], [60, 90], 300, 4),
    ("two", 16, 1, 64, [1600, 700], [1300, 300], 0, 0),
    ("two", 8, 8, 32, [2500, 300], [2400, 290], 0, 0),
    ("two", 20, 5, 16, [3000], [3000], 0, 0),
    ("two", 16, 8, 32, [1500, 130, 1400, 0, 1], [1400, 130, 1390, 0, 1], 700, 5),
    ("two", 6, 2, 64, [4000], [4000], 100, 200),
    ("two", 7, 1, 128, [3000, 41], [2990, 30], 1, 1),
    ("parts", 8, 2, 64, [9000, 5000, 70, 0], [40, 90, 70, 0], 0, 0),
    ("parts", 20, 5, 128, [32801], [200], 0, 0),
    ("parts", 8, 2, 64, [30000, 20000, 500], [40, 90, 2], 9000, 40),
    ("parts", 6, 2, 32, [12000], [300], 6000, 300),
    ("parts", 16, 1, 16, [9000, 4000], [5, 33], 5000, 4),
]


@pytest.mark.parametrize("path,H,Hkv,page,lens,new,window,sinks", RANDOM)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("peaked", [False, True])
def test_random_queries(bw, path, H, Hkv, page, lens, new, window, sinks, D,
                        peaked):
    """Every row against 64 bits, whatever way the call is cut, and the same
    twice.  peaked: few keys far above the others, the later the further, so
    that the maximum follows often and late.  Rows and pages that no token
    sees hold anything."""
    c = Cache(151, lens, Hkv, D, page)
    rng = np.random.default_rng(152)
    for b, (n, a) in enumerate(zip(lens, new)):
        if peaked and n:
            g = np.where(rng.random(n) < 0.02, 6.0 * (np.arange(n) + 50) / n, 0.2)
            c.k[b] = as_bf16(c.k[b].float().numpy() * g[:, None, None])
        p = torch.arange(n - a, n)[:, None]
        j = torch.arange(n)[None, :]
        vis = ((j <= p) & ((window == 0) | (j > p - window) | (j < sinks))).any(0)
        ids = torch.from_numpy(c.table[b].astype(np.int64))
        at, row = ids[torch.arange(n) // page], torch.arange(n) % page
        k = torch.where(vis[:, None, None], c.k[b], float("nan")).cuda()
        v = torch.where(vis[:, None, None], c.v[b], float("nan")).cuda()
        c.kp[at.cuda(), :, row.cuda()] = k
        c.vp[at.cuda(), :, row.cuda()] = v
        for i in range(-(-n // page)):
            if not vis[i * page:(i + 1) * page].any():
                c.table_d[b, i] = -1
    tokens = sum(new) + 2 * LEAD
    start = LEAD + np.concatenate([[0], np.cumsum(new)])
    q = as_bf16((3.0 if peaked else 1.5) *
                rng.standard_normal((tokens, H, D))).cuda()
    st = torch.from_numpy(start.astype(np.int32)).cuda()
    outs = []
    for _ in range(2):
        out = torch.full((tokens, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
        bw.bw_attn_paged_prefill(q, *c.args, st, window=window, sinks=sinks,
                                 out=out)
        assert bw.bw_device_error() == 0
        outs.append(out)
    assert torch.equal(*outs)
    assert (out[:LEAD] == 9.0).all() and (out[tokens - LEAD:] == 9.0).all()
    for b, (n, a) in enumerate(zip(lens, new)):
        if a == 0:
            continue
        rows = slice(int(start[b]), int(start[b + 1]))
        want, tol = exact(q[rows], c.k[b], c.v[b], n - a, window, sinks, D ** -0.5)
        err = (out[rows].double() - want).abs()
        assert (err <= tol).all(), (b, float((err - tol).max()))


# ---------------------------------------------------------------------------
# a captured call in parts
# ---------------------------------------------------------------------------

CAPTURED = [
    # H, Hkv, lens, tokens of the call, window, sinks
    (8, 2, [9000, 700], 60, 0, 0),
    (16, 1, [20000, 7000], 20, 8000, 30),
]


@pytest.mark.parametrize("H,Hkv,lens,tokens,window,sinks", CAPTURED)
@pytest.mark.parametrize("D", [64, 128])
def test_captured_in_parts(bw, H, Hkv, lens, tokens, window, sinks, D):
    """Captured once, replayed with other queries, lengths and ranges: as eager
    calls, bit for bit, and within the bound."""
    c = Cache(161, lens, Hkv, D, 64)
    q = torch.zeros((tokens, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.zeros((bw.bw_attn_paged_prefill_workspace_bytes(
        tokens, 2, H, Hkv, D),), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            bw.bw_attn_paged_prefill(q, *c.args, st, window=window, sinks=sinks,
                                     out=out, workspace=ws)
    for step, (n0, cut) in enumerate([(tokens - 4, 0), (tokens - 9, 5003),
                                      (0, 8990), (3, 300)]):
        q.copy_(torch.randn(q.shape, device="cuda"))
        st.copy_(torch.tensor([0, n0, tokens - step]))
        n = [lens[0] - cut, lens[1]]
        c.len_d.copy_(torch.tensor(n))
        out.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert bw.bw_device_error() == 0
        eager = torch.full_like(out, 9.0)
        bw.bw_attn_paged_prefill(q, *c.args, st, window=window, sinks=sinks,
                                 out=eager)
        assert torch.equal(out, eager)
        assert (out[tokens - step:] == 9.0).all()
        for b, (lo, hi) in enumerate([(0, n0), (n0, tokens - step)]):
            if lo == hi:
                continue
            want, tol = exact(q[lo:hi], c.k[b][:n[b]], c.v[b][:n[b]],
                              n[b] - (hi - lo), window, sinks, D ** -0.5)
            err = (out[lo:hi].double() - want).abs()
            assert (err <= tol).all(), (step, b, float((err - tol).max()))
