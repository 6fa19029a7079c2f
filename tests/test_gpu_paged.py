"""The calls over a paged key-value cache (GB300) against plain 64-bit forms.

The W2A8 kernel page keeps a preallocated KV cache (§六 item 2) for grouped
query heads (§一) whose RoPE turns adjacent pairs (§4.1); the cache here is cut
into pages.  Every row of the pools that no sequence's position owns holds
NaN, every page-table entry past a sequence's end is out of range, so a result
that is right shows that neither is used.

Tolerances (u = 2^-24 for fp32, a rounding to bf16 is off by at most 2^-8 of
the value):
  * rotated queries and keys: 2^-8 |z| for the rounding; the fast sine and
    cosine are off by at most 2^-20 on [-pi, pi], the reduced angle by less,
    and norm and products by a few u of the pair: 2^-19 (|y0| + |y1|) more.
  * attention: a score is a D-term fp32 sum, each step rounded or truncated:
    off by at most (D + 4) 2 u scale sum_d |q k| (the scaling and the change to
    base 2 included); a weight's relative error is that plus 8 u for the
    exponential and the rescaling; sums over n positions add n u.  An output
    is a weighted mean of v, so it is off by at most twice that (numerator and
    denominator) times the largest |v|.  bf16 weights (prefill) are off by
    2^-8 each: 2^-8 of the weighted mean of |v| more.  A bf16 output: 2^-8 of
    the value more.
"""
import numpy as np
import pytest

import synth  # noqa: F401  (the path set up by conftest)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

THETA = 500000.0
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_lib
    build_lib()
    import bit_gemv_bitlinear_gb300 as bw
    return bw


def as_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


class Cache:
    """Pools of NaN, shuffled pages, a table whose unused entries are out of
    range; lens: the positions of each sequence (written with normals)."""

    def __init__(self, seed, lens, Hkv, D, page, spare_pages=2, extra=0,
                 fill=True, max_pages=None):
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.Hkv, self.D, self.page = list(lens), Hkv, D, page
        need = [-(-n // page) for n in self.lens]
        self.max_pages = max_pages or max(max(need), 1) + 1
        self.n_pages = sum(need) + spare_pages
        ids = rng.permutation(self.n_pages)[:sum(need)]
        self.table = np.full((len(self.lens), self.max_pages), -7, np.int32)
        self.table[:, 1::2] = self.n_pages + 5
        k = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[k:k + n]
            k += n
        shape = (self.n_pages, Hkv, page, D)
        self.k = [as_bf16(rng.standard_normal((n, Hkv, D))) for n in self.lens]
        self.v = [as_bf16(rng.standard_normal((n, Hkv, D))) for n in self.lens]
        kp = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        vp = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        if fill:
            for b, n in enumerate(self.lens):
                for j in range(n):
                    p = self.table[b, j // page]
                    kp[p, :, j % page] = self.k[b][j]
                    vp[p, :, j % page] = self.v[b][j]
        # pages `extra` elements further apart than they need to be
        size = Hkv * page * D
        pool = torch.full((2, self.n_pages, size + extra), float("nan"),
                          dtype=torch.bfloat16, device="cuda")
        self.pool = pool
        self.kp = pool[0, :, :size].view(self.n_pages, Hkv, page, D)
        self.vp = pool[1, :, :size].view(self.n_pages, Hkv, page, D)
        self.kp.copy_(kp)
        self.vp.copy_(vp)
        self.table_d = torch.from_numpy(self.table).cuda()
        self.len_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    @property
    def args(self):
        return self.kp, self.vp, self.table_d, self.len_d

    def forget(self, b, j):
        """Position j of sequence b holds NaN from now on."""
        p = int(self.table[b, j // self.page])
        self.kp[p, :, j % self.page] = float("nan")
        self.vp[p, :, j % self.page] = float("nan")


def seen(p, window, sinks):
    j = np.arange(p + 1)
    if window == 0:
        return j
    return j[(j > p - window) | (j < sinks)]


def attend(q, k, v, scale, vis, p_bits=0.0):
    """One token: q [H][D], k, v [n][Hkv][D] in 64 bits, the positions vis:
    (out [H][D], bound [H][1])."""
    H, D = q.shape
    G = H // k.shape[1]
    out = np.zeros((H, D))
    tol = np.zeros((H, D))
    if len(vis) == 0:
        return out, tol
    kv, vv = k[vis], v[vis]
    for h in range(H):
        kk, vh = kv[:, h // G], vv[:, h // G]
        s = kk @ q[h] * scale
        mass = np.abs(kk) @ np.abs(q[h]) * scale
        w = np.exp(s - s.max())
        w /= w.sum()
        out[h] = w @ vh
        rel = (D + 4) * 2 * U * mass.max() + (8 + len(vis)) * U
        tol[h] = 2 * rel * np.abs(vh).max() + p_bits * (w @ np.abs(vh))
    return out, tol


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


# ---------------------------------------------------------------------------
# norm, rotation, append
# ---------------------------------------------------------------------------

def norm_rope(x, p, gamma, eps, theta):
    """x [..., D] in 64 bits at position p: (z, |y0| + |y1| of its pair)."""
    D = x.shape[-1]
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    a = p * theta ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(a), np.sin(a)
    z = np.empty_like(x)
    z[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    z[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    pair = np.abs(x[..., 0::2]) + np.abs(x[..., 1::2])
    return z, np.repeat(pair, 2, -1)


APPEND = [
    # H, Hkv, D, page, lens, new (None: one each), norm, extra
    (20, 5, 128, 64, [701], None, True, 0),
    (20, 5, 128, 16, [1, 16, 17, 0, 300], None, True, 0),
    (1, 1, 64, 16, [5], None, False, 0),
    (16, 1, 128, 256, [257, 255], None, True, 24),
    (64, 64, 128, 16, [33, 1], None, True, 0),
    (20, 5, 128, 32, [70, 33, 40, 1], [70, 1, 0, 1], True, 0),
    (32, 8, 64, 128, [129, 200, 77], [128, 3, 0], False, 8),
    (14, 2, 64, 16, [31] * 40, [2] * 40, True, 0),
    (6, 2, 128, 64, [3] * 1100, [1] * 1100, True, 0),
]


@pytest.mark.parametrize("H,Hkv,D,page,lens,new,norm,extra", APPEND)
@pytest.mark.parametrize("pad,in_place", [(0, False), (3, True)])
def test_append(bw, H, Hkv, D, page, lens, new, norm, extra, pad, in_place):
    c = Cache(11, lens, Hkv, D, page, extra=extra, fill=False)
    rng = np.random.default_rng(12)
    counts = new or [1] * len(lens)
    lead = pad if new else 0          # rows of no sequence, before and after
    tokens = sum(counts) + 2 * lead
    width = (H + 2 * Hkv) * D
    # rows of a wider buffer
    wide = as_bf16(rng.standard_normal((tokens, width + 8 * pad))).cuda()
    qkv = wide[:, :width]
    gq = gk = None
    if norm:
        gq = torch.from_numpy(rng.uniform(0.5, 1.5, D).astype(np.float32))
        gk = torch.from_numpy(rng.uniform(0.5, 1.5, D).astype(np.float32))
    start = lead + np.concatenate([[0], np.cumsum(counts)])
    x = f64(qkv).reshape(tokens, H + 2 * Hkv, D)
    before = c.pool.clone()
    raw_before = qkv.clone()
    q_out = qkv.unflatten(1, (H + 2 * Hkv, D))[:, :H] if in_place else \
        torch.full((tokens, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got = bw.bw_qk_norm_rope_append(
        qkv, *c.args, H,
        q_start=torch.from_numpy(start.astype(np.int32)).cuda() if new else None,
        q_gamma=gq.cuda() if norm else None,
        k_gamma=gk.cuda() if norm else None, eps=1e-6, theta=THETA,
        q_out=q_out)
    assert got is q_out
    assert bw.bw_device_error() == 0
    raw = raw_before.cpu().unflatten(1, (H + 2 * Hkv, D))
    want_pool = before.cpu()
    kp = want_pool[0, :, :Hkv * page * D].view(-1, Hkv, page, D)
    vp = want_pool[1, :, :Hkv * page * D].view(-1, Hkv, page, D)
    after = c.pool.cpu()
    ka = after[0, :, :Hkv * page * D].view(-1, Hkv, page, D)
    q_got = f64(q_out)
    owned = np.zeros(tokens, bool)
    for b, n in enumerate(counts):
        for i in range(n):
            t = start[b] + i
            p = lens[b] - n + i
            if p < 0:
                continue
            owned[t] = True
            z, pair = norm_rope(x[t, :H], p, gq.double().numpy() if norm else None,
                                1e-6, THETA)
            assert (np.abs(q_got[t] - z) <= 2.0 ** -8 * np.abs(z) +
                    2.0 ** -19 * pair + 1e-30).all(), (b, i)
            z, pair = norm_rope(x[t, H:H + Hkv], p,
                                gk.double().numpy() if norm else None, 1e-6, THETA)
            page_id = c.table[b, p // page]
            kg = f64(ka[page_id, :, p % page])
            assert (np.abs(kg - z) <= 2.0 ** -8 * np.abs(z) +
                    2.0 ** -19 * pair + 1e-30).all(), (b, i)
            kp[page_id, :, p % page] = ka[page_id, :, p % page]
            vp[page_id, :, p % page] = raw[t, H + Hkv:]
    # every other byte of the pools, and the rows of no sequence, untouched
    assert torch.equal(after.view(torch.int16), want_pool.view(torch.int16))
    fresh = raw[:, :H] if in_place else torch.full((tokens, H, D), 7.0,
                                                   dtype=torch.bfloat16)
    rest = torch.from_numpy(~owned)
    assert torch.equal(q_out.cpu()[rest], fresh[rest])
    if in_place:  # keys and values of the rows stay
        assert torch.equal(qkv.cpu()[:, H * D:], raw_before.cpu()[:, H * D:])


def test_append_far_position(bw):
    """The last position that the limits allow: angles of 2^24 radians."""
    page, D = 256, 128
    n = 1 << 24
    H = Hkv = 1
    kp = torch.zeros((2, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.full((1, n // page), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    x = as_bf16(np.random.default_rng(5).standard_normal((1, 3 * D))).cuda()
    q = bw.bw_qk_norm_rope_append(x, kp, vp, table, lens, H, theta=10000.0)
    assert bw.bw_device_error() == 0
    z, pair = norm_rope(f64(x)[0, :D], n - 1, None, 0.0, 10000.0)
    assert (np.abs(f64(q)[0, 0] - z) <= 2.0 ** -8 * np.abs(z) + 2.0 ** -19 * pair).all()
    assert torch.equal(vp[1, 0, page - 1], x[0, 2 * D:])
    assert int((vp != 0).sum()) <= D


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------

DECODE = [
    # H, Hkv, D, page, lens, window, sinks, extra
    (20, 5, 128, 16, [1], 0, 0, 0),
    (20, 5, 128, 64, [777], 0, 0, 0),
    (20, 5, 128, 64, [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1000], 0, 0, 0),
    (20, 5, 128, 16, [5000, 3], 0, 0, 0),
    (8, 8, 128, 256, [300, 257, 2], 0, 0, 40),
    (16, 1, 128, 32, [513, 77], 0, 0, 0),
    (9, 1, 64, 16, [200, 31], 0, 0, 0),
    (32, 4, 64, 32, [900, 1200, 40, 999, 1000, 1001, 1004, 1005], 1000, 4, 0),
    (14, 2, 64, 128, [400, 129, 1], 130, 0, 8),
    (20, 5, 128, 64, [200, 500, 64, 65, 70], 1, 0, 0),
    (20, 5, 128, 64, [200, 500, 64, 65, 70], 1, 1, 0),
    (6, 2, 128, 16, [2000, 333], 100, 300, 0),
    (6, 2, 128, 16, [700, 40], 33, 17, 0),
    (4, 4, 128, 16, [(7 * i) % 41 for i in range(300)], 0, 0, 0),
    (2, 1, 64, 16, [(5 * i) % 97 for i in range(1500)], 20, 2, 0),
]


def check_decode(bw, c, q, out, window, sinks, scale, bf16):
    got = f64(out)
    qf = f64(q)
    for b, n in enumerate(c.lens):
        ref, tol = attend(qf[b], f64(c.k[b]), f64(c.v[b]), scale,
                          seen(n - 1, window, sinks))
        if bf16:
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert (np.abs(got[b] - ref) <= tol).all(), \
            (b, n, np.abs(got[b] - ref).max(), tol.min())


@pytest.mark.parametrize("H,Hkv,D,page,lens,window,sinks,extra", DECODE)
@pytest.mark.parametrize("bf16", [False, True])
def test_decode(bw, H, Hkv, D, page, lens, window, sinks, extra, bf16):
    c = Cache(21, lens, Hkv, D, page, extra=extra)
    # rows and pages outside the window hold anything
    for b, n in enumerate(lens):
        vis = set(seen(n - 1, window, sinks).tolist())
        for j in range(n):
            if j not in vis:
                c.forget(b, j)
        for i in range(-(-n // page)):
            if not vis & set(range(i * page, min(n, (i + 1) * page))):
                c.table_d[b, i] = -1
    rng = np.random.default_rng(22)
    n = len(lens)
    wide = as_bf16(2.0 * rng.standard_normal((n, H + 1, D))).cuda()
    q = wide[:, :H]
    scale = 0.09
    ws = torch.zeros((bw.bw_attn_paged_decode_workspace_bytes(n, H, Hkv, D),),
                     dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):  # the workspace serves again
        wide_out = torch.full((n, H + 2, D), 3.0, device="cuda",
                              dtype=torch.bfloat16 if bf16 else torch.float32)
        bw.bw_attn_paged_decode(q, *c.args, window=window, sinks=sinks,
                                scale=scale, out=wide_out[:, :H], workspace=ws)
        assert bw.bw_device_error() == 0
        assert (wide_out[:, H:] == 3.0).all()
        outs.append(wide_out[:, :H].clone())
    assert torch.equal(outs[0], outs[1])
    check_decode(bw, c, q, outs[0], window, sinks, scale, bf16)


def test_decode_peaked_scores(bw):
    """Scores over a wide range, their largest anywhere: the running maximum
    moves often, and a tile's weights may all vanish."""
    lens = [1500, 640]
    c = Cache(31, lens, 2, 128, 32)
    for b, n in enumerate(lens):  # keys that grow, shrink, and jump
        g = np.linspace(0.1, 6.0, n) if b == 0 else np.linspace(6.0, 0.1, n)
        c.k[b] = as_bf16(f64(c.k[b]) * g[:, None, None])
        for j in range(n):
            c.kp[int(c.table[b, j // 32]), :, j % 32] = c.k[b][j].cuda()
    q = as_bf16(4.0 * np.random.default_rng(3).standard_normal((2, 8, 128))).cuda()
    out = bw.bw_attn_paged_decode(q, *c.args)
    assert bw.bw_device_error() == 0
    check_decode(bw, c, q, out, 0, 0, 128 ** -0.5, False)


# ---------------------------------------------------------------------------
# prefill
# ---------------------------------------------------------------------------

PREFILL = [
    # H, Hkv, D, page, lens, new, window, sinks, extra
    (20, 5, 128, 16, [1], [1], 0, 0, 0),
    (20, 5, 128, 64, [200], [200], 0, 0, 0),
    (20, 5, 128, 16, [509], [509], 0, 0, 0),
    (20, 5, 128, 64, [700, 33, 5, 129, 64], [100, 33, 0, 1, 64], 0, 0, 0),
    (4, 4, 128, 256, [300, 257], [300, 130], 0, 0, 40),
    (16, 1, 128, 32, [150, 40], [150, 17], 0, 0, 0),
    (9, 1, 64, 16, [90, 31], [60, 31], 0, 0, 0),
    (7, 1, 128, 16, [170], [101], 0, 0, 0),
    (16, 8, 64, 32, [600, 130, 1], [500, 130, 1], 70, 5, 0),
    (14, 2, 64, 128, [400, 300], [390, 20], 130, 0, 8),
    (8, 2, 128, 64, [333, 300], [300, 7], 1, 0, 0),
    (8, 2, 128, 64, [333, 300], [300, 7], 1, 1, 0),
    (6, 2, 128, 16, [600], [350], 33, 200, 0),
    (2, 2, 128, 128, [3100], [40], 0, 0, 0),
    (4, 1, 128, 16, [5000, 2], [3, 2], 900, 4, 0),
    (2, 1, 64, 16, [(5 * i) % 47 + 1 for i in range(200)],
     [(3 * i) % 5 % ((5 * i) % 47 + 1) for i in range(200)], 20, 2, 0),
]


def check_prefill(c, q, out, start, new, window, sinks, scale):
    got, qf = f64(out), f64(q)
    for b, n in enumerate(new):
        kk, vv = f64(c.k[b]), f64(c.v[b])
        for i in range(n):
            p = c.lens[b] - n + i
            ref, tol = attend(qf[start[b] + i], kk, vv, scale,
                              seen(p, window, sinks), 2.0 ** -8)
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            err = np.abs(got[start[b] + i] - ref)
            assert (err <= tol).all(), (b, i, p, err.max(), tol[err > tol][:3])


@pytest.mark.parametrize("H,Hkv,D,page,lens,new,window,sinks,extra", PREFILL)
def test_prefill(bw, H, Hkv, D, page, lens, new, window, sinks, extra):
    c = Cache(41, lens, Hkv, D, page, extra=extra)
    for b, (n, a) in enumerate(zip(lens, new)):
        vis = set()
        for p in range(n - a, n):
            vis |= set(seen(p, window, sinks).tolist())
        for j in range(n):
            if j not in vis:
                c.forget(b, j)
        for i in range(-(-n // page)):
            if not vis & set(range(i * page, min(n, (i + 1) * page))):
                c.table_d[b, i] = -1
    lead = 3
    tokens = sum(new) + 2 * lead
    start = lead + np.concatenate([[0], np.cumsum(new)])
    rng = np.random.default_rng(42)
    wide = as_bf16(2.0 * rng.standard_normal((tokens, H + 1, D))).cuda()
    q = wide[:, :H]
    scale = 0.09
    ws = torch.zeros((bw.bw_attn_paged_prefill_workspace_bytes(
        tokens, len(lens), H, Hkv, D),), dtype=torch.uint8, device="cuda")
    st = torch.from_numpy(start.astype(np.int32)).cuda()
    outs = []
    for _ in range(2):
        wide_out = torch.full((tokens, H + 2, D), 3.0, dtype=torch.bfloat16,
                              device="cuda")
        bw.bw_attn_paged_prefill(q, *c.args, st, window=window, sinks=sinks,
                                 scale=scale, out=wide_out[:, :H],
                                 workspace=ws)
        assert bw.bw_device_error() == 0
        assert (wide_out[:, H:] == 3.0).all()
        assert (wide_out[:lead] == 3.0).all()
        assert (wide_out[tokens - lead:] == 3.0).all()
        outs.append(wide_out[:, :H].clone())
    assert torch.equal(outs[0], outs[1])
    check_prefill(c, q, outs[0], start, new, window, sinks, scale)


def test_prefill_peaked_scores(bw):
    lens, new = [700, 300], [256, 300]
    c = Cache(51, lens, 2, 128, 32)
    for b, n in enumerate(lens):
        g = np.linspace(0.1, 6.0, n) if b == 0 else np.linspace(6.0, 0.1, n)
        c.k[b] = as_bf16(f64(c.k[b]) * g[:, None, None])
        for j in range(n):
            c.kp[int(c.table[b, j // 32]), :, j % 32] = c.k[b][j].cuda()
    start = np.concatenate([[0], np.cumsum(new)])
    q = as_bf16(4.0 * np.random.default_rng(3).standard_normal(
        (int(start[-1]), 8, 128))).cuda()
    out = bw.bw_attn_paged_prefill(q, *c.args,
                                   torch.from_numpy(start.astype(np.int32)).cuda())
    assert bw.bw_device_error() == 0
    check_prefill(c, q, out, start, new, 0, 0, 128 ** -0.5)


# ---------------------------------------------------------------------------
# what the host cannot check
# ---------------------------------------------------------------------------

BAD = 256


def take_bad(bw):
    with pytest.raises(bw.BwError) as e:
        bw.bw_device_error()
    assert e.value.status == 1
    assert bw.bw_device_error() == 0


@pytest.mark.parametrize("what", ["negative length", "long length", "bad page"])
def test_bad_contents_of_the_cache(bw, what):
    """One bad sequence among three: reported, the others right, nothing of
    the others' pages written."""
    H, Hkv, D, page = 8, 2, 128, 16
    lens = [40, 50, 60]
    c = Cache(61, lens, Hkv, D, page)
    if what == "negative length":
        c.len_d[1] = -3
    elif what == "long length":
        c.len_d[1] = c.max_pages * page + 1
    else:
        c.table_d[1, 3] = c.n_pages  # holds the last positions
    q = as_bf16(np.random.default_rng(3).standard_normal((3, H, D))).cuda()
    out = bw.bw_attn_paged_decode(q, *c.args, scale=0.1)
    torch.cuda.synchronize()
    take_bad(bw)
    good = out.clone()
    if what == "bad page":  # reads as zeros: positions 48 and 49 weigh in
        k, v = c.k[1].clone(), c.v[1].clone()
        k[48:], v[48:] = 0, 0
        ref, tol = attend(f64(q)[1], f64(k), f64(v), 0.1, np.arange(50))
        assert (np.abs(f64(out)[1] - ref) <= tol).all()
    else:
        assert (out[1] == 0).all()
    for b in (0, 2):
        ref, tol = attend(f64(q)[b], f64(c.k[b]), f64(c.v[b]), 0.1,
                          np.arange(lens[b]))
        assert (np.abs(f64(good)[b] - ref) <= tol).all()
    start = torch.tensor([0, 4, 9, 12], dtype=torch.int32, device="cuda")
    qp = as_bf16(np.random.default_rng(4).standard_normal((12, H, D))).cuda()
    po = bw.bw_attn_paged_prefill(qp, *c.args, start, scale=0.1)
    torch.cuda.synchronize()
    take_bad(bw)
    if what != "bad page":
        assert (po[4:9] == 0).all()
    assert torch.isfinite(po.float()).all()
    qkv = as_bf16(np.random.default_rng(5).standard_normal(
        (12, (H + 2 * Hkv) * D))).cuda()
    before = c.pool.clone()
    q_out = torch.full((12, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    bw.bw_qk_norm_rope_append(qkv, *c.args, H, q_start=start, q_out=q_out)
    torch.cuda.synchronize()
    take_bad(bw)
    changed = (c.pool.view(torch.int16) != before.view(torch.int16)) \
        .flatten(2).any(-1).any(0).cpu().numpy()
    mine = set()
    for b, n in ((0, 4), (2, 3)):
        mine |= {int(c.table[b, p // page]) for p in range(lens[b] - n, lens[b])}
    if what == "bad page":
        mine |= {int(c.table[1, p // page]) for p in range(45, 48)}
        assert (q_out[4:9] != 7.0).any()
    else:
        assert (q_out[4:9] == 7.0).all()
    assert set(np.nonzero(changed)[0].tolist()) <= mine


@pytest.mark.parametrize("start", [[0, 5, 3, 12], [-1, 2, 4, 12], [0, 2, 4, 13],
                                   [0, 2, 60, 60], [2 ** 31 - 1] * 4])
def test_bad_token_ranges(bw, start):
    H, Hkv, D, page = 8, 2, 128, 16
    c = Cache(62, [40, 50, 60], Hkv, D, page)
    st = torch.tensor(start, dtype=torch.int64).to(torch.int32).cuda()
    q = as_bf16(np.random.default_rng(4).standard_normal((12, H, D))).cuda()
    out = bw.bw_attn_paged_prefill(q, *c.args, st)
    torch.cuda.synchronize()
    take_bad(bw)
    assert torch.isfinite(out.float()).all()
    qkv = as_bf16(np.random.default_rng(5).standard_normal(
        (12, (H + 2 * Hkv) * D))).cuda()
    bw.bw_qk_norm_rope_append(qkv, *c.args, H, q_start=st)
    torch.cuda.synchronize()
    take_bad(bw)


def test_more_tokens_than_positions(bw):
    H, Hkv, D, page = 8, 2, 128, 16
    c = Cache(63, [3, 20], Hkv, D, page)
    st = torch.tensor([0, 5, 9], dtype=torch.int32, device="cuda")
    q = as_bf16(np.random.default_rng(4).standard_normal((9, H, D))).cuda()
    out = bw.bw_attn_paged_prefill(q, *c.args, st, scale=0.1)
    torch.cuda.synchronize()
    take_bad(bw)
    assert (out[:5] == 0).all()
    for i in range(4):
        ref, tol = attend(f64(q)[5 + i], f64(c.k[1]), f64(c.v[1]), 0.1,
                          np.arange(17 + i), 2.0 ** -8)
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert (np.abs(f64(out)[5 + i] - ref) <= tol).all()


# ---------------------------------------------------------------------------
# streams, graphs, the operators together
# ---------------------------------------------------------------------------

def test_serving_steps(bw):
    """Prompts in, then tokens one by one through captured graphs on a side
    stream: the same results as one 64-bit model of the three operators, and
    as eager calls, bit for bit."""
    H, Hkv, D, page = 20, 5, 128, 32
    rng = np.random.default_rng(71)
    prompts, steps, window, sinks = [75, 1, 130], 6, 50, 3
    n = len(prompts)
    width = (H + 2 * Hkv) * D
    gq = rng.uniform(0.5, 2.0, D).astype(np.float32)
    gk = rng.uniform(0.5, 2.0, D).astype(np.float32)
    rows = as_bf16(rng.standard_normal((sum(prompts), width)))
    news = as_bf16(rng.standard_normal((steps, n, width)))

    def serve(graph):
        c = Cache(72, [p + steps for p in prompts], Hkv, D, page, fill=False)
        c.len_d.copy_(torch.tensor(prompts))
        start = torch.tensor(np.concatenate([[0], np.cumsum(prompts)]),
                             dtype=torch.int32, device="cuda")
        g1, g2 = torch.from_numpy(gq).cuda(), torch.from_numpy(gk).cuda()
        q = bw.bw_qk_norm_rope_append(rows.cuda(), *c.args, H, q_start=start,
                                      q_gamma=g1, k_gamma=g2)
        first = bw.bw_attn_paged_prefill(q, *c.args, start, window=window,
                                         sinks=sinks)
        x = torch.zeros((n, width), dtype=torch.bfloat16, device="cuda")
        out = torch.zeros((n, H, D), device="cuda")
        qs = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros((bw.bw_attn_paged_decode_workspace_bytes(n, H, Hkv, D),),
                         dtype=torch.uint8, device="cuda")

        def step():
            c.len_d.add_(1)
            bw.bw_qk_norm_rope_append(x, *c.args, H, q_gamma=g1, k_gamma=g2,
                                      q_out=qs)
            bw.bw_attn_paged_decode(qs, *c.args, window=window, sinks=sinks,
                                    out=out, workspace=ws)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = []
        with torch.cuda.stream(side):
            if graph:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    step()
            for s in range(steps):
                x.copy_(news[s])
                g.replay() if graph else step()
                outs.append(out.clone())
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert bw.bw_device_error() == 0
        return c, first, torch.stack(outs)

    c, first, outs = serve(True)
    _, first2, outs2 = serve(False)
    assert torch.equal(first, first2) and torch.equal(outs, outs2)

    # what the cache holds is checked against 64 bits, then the attention
    # against what the cache holds
    start = np.concatenate([[0], np.cumsum(prompts)])
    for b, n0 in enumerate(prompts):
        raw = torch.cat([rows[start[b]:start[b + 1]], news[:, b]])
        x = f64(raw).reshape(-1, H + 2 * Hkv, D)
        total = n0 + steps
        ids = torch.from_numpy(c.table[b, :-(-total // page)].astype(np.int64))
        kc = f64(c.kp.cpu()[ids].transpose(1, 2).reshape(-1, Hkv, D)[:total])
        vc = f64(c.vp.cpu()[ids].transpose(1, 2).reshape(-1, Hkv, D)[:total])
        assert (vc == x[:, H + Hkv:]).all()
        q64 = np.empty((total, H, D))
        for p in range(total):
            zk, pair = norm_rope(x[p, H:H + Hkv], p, gk.astype(np.float64),
                                 1e-5, THETA)
            assert (np.abs(kc[p] - zk) <= 2.0 ** -8 * np.abs(zk) +
                    2.0 ** -19 * pair).all()
            q64[p], _ = norm_rope(x[p, :H], p, gq.astype(np.float64), 1e-5, THETA)
        # q was rounded to bf16: a score moves by 2^-8 of its terms' mass, so
        # a weight by that much, an output by twice that of the largest |v|
        for p in list(range(0, n0, 13)) + list(range(n0 - 1, total)):
            vis = seen(p, window, sinks)
            ref, tol = attend(q64[p], kc, vc, D ** -0.5, vis, 2.0 ** -8)
            mass = max((np.abs(kc[vis][:, h // (H // Hkv)]) @ np.abs(q64[p, h])).max()
                       for h in range(H)) * D ** -0.5
            tol = tol + 2 * 1.01 * 2.0 ** -8 * mass * np.abs(vc[vis]).max()
            got = f64(first)[start[b] + p] if p < n0 else f64(outs)[p - n0, b]
            assert (np.abs(got - ref) <= tol + 2.0 ** -8 * np.abs(ref)).all(), (b, p)


def test_prefill_equals_decode_token_by_token(bw):
    """A chunk's last row and the single-token call see the same positions."""
    H, Hkv, D, page = 8, 2, 128, 64
    lens, new = [500, 90], [37, 90]
    c = Cache(81, lens, Hkv, D, page)
    start = np.concatenate([[0], np.cumsum(new)])
    q = as_bf16(np.random.default_rng(1).standard_normal((int(start[-1]), H, D))).cuda()
    out = bw.bw_attn_paged_prefill(q, *c.args,
                                   torch.from_numpy(start.astype(np.int32)).cuda())
    one = bw.bw_attn_paged_decode(q[start[1:] - 1], *c.args)
    assert bw.bw_device_error() == 0
    v = max(float(x.abs().max()) for x in c.v)
    # the prefill's weights and output are bf16: 2^-8 of the mean of |v|, twice
    diff = (out[start[1:] - 1].float() - one).abs().max()
    assert float(diff) <= 2 * 1.01 * 2.0 ** -8 * v


def test_two_calls_at_once_on_two_streams(bw):
    H, Hkv, D, page = 20, 5, 128, 32
    c = Cache(91, [800, 33, 1200], Hkv, D, page)
    q = as_bf16(np.random.default_rng(1).standard_normal((3, H, D))).cuda()
    want = bw.bw_attn_paged_decode(q, *c.args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        outs.append(bw.bw_attn_paged_decode(q, *c.args, stream=streams[i % 2]))
    torch.cuda.synchronize()
    assert bw.bw_device_error() == 0
    for o in outs:
        assert torch.equal(o, want)


def test_refusals(bw):
    H, Hkv, D, page = 8, 2, 128, 16
    c = Cache(95, [40, 50], Hkv, D, page)
    kp, vp, table, lens = c.args
    q = torch.zeros((2, H, D), dtype=torch.bfloat16, device="cuda")
    ok = dict(q=q, k_pages=kp, v_pages=vp, page_table=table, kv_len=lens)

    def refused(exc, **kw):
        with pytest.raises(exc):
            bw.bw_attn_paged_decode(**{**ok, **kw})

    refused(TypeError, q=q.float())
    refused(ValueError, q=q.cpu())
    refused(ValueError, q=q[:1])
    refused(ValueError, q=q[:, :, :64])
    refused(ValueError, q=q.transpose(1, 2))
    refused(ValueError, k_pages=kp[:-1])
    refused(ValueError, k_pages=kp.transpose(1, 2))
    refused(TypeError, kv_len=lens.long())
    refused(ValueError, kv_len=lens[:1])
    refused(ValueError, page_table=table[:, ::2])
    refused(bw.BwError, scale=0.0)
    refused(bw.BwError, scale=float("nan"))
    refused(bw.BwError, window=-1)
    refused(bw.BwError, sinks=-1)
    refused(bw.BwError, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    refused(TypeError, out=torch.zeros((2, H, D), dtype=torch.float16, device="cuda"))
    refused(ValueError, out=torch.zeros((2, H, D)))
    refused(bw.BwError, q=torch.zeros((2, 7, D), dtype=torch.bfloat16, device="cuda"))
    refused(bw.BwError, q=torch.zeros((2, 34, D), dtype=torch.bfloat16, device="cuda"))
    odd = torch.zeros((2, H * D + 4), dtype=torch.bfloat16, device="cuda")
    refused(bw.BwError, q=odd[:, :H * D].unflatten(1, (H, D)))
    st = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    with pytest.raises(bw.BwError):  # in place
        bw.bw_attn_paged_prefill(q, *c.args, st, out=q)
    with pytest.raises(ValueError):
        bw.bw_attn_paged_prefill(q, *c.args, st[:2])
    qkv = torch.zeros((2, (H + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        bw.bw_qk_norm_rope_append(qkv[:, :-8], *c.args, H)
    with pytest.raises(bw.BwError):
        bw.bw_qk_norm_rope_append(qkv[:1], *c.args, H)
    with pytest.raises(bw.BwError):
        bw.bw_qk_norm_rope_append(qkv, *c.args, H, theta=0.5)
    with pytest.raises(ValueError):
        bw.bw_qk_norm_rope_append(qkv, *c.args, H,
                                  q_gamma=torch.ones(64, device="cuda"))
    assert bw.bw_device_error() == 0
