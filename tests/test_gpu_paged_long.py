"""The calls over a paged key-value cache (GB300) where they are large: long
caches and batches whose work is claimed while a call runs, many query tiles,
offsets past 2^31 elements, and one workspace under calls of many shapes.

A query of zeros gives every visible position the weight one, and values that
are small integers have sums that fp32 and the tensor cores hold exactly (all
partial sums are below 2^24), so the answer is the mean of the visible values
but for the last division: a position left out, taken twice or taken from
another page shows.  Tolerances (u = 2^-24): decode's parts are multiplied by
1 / l before or after the last additions, 8 u of the mean of |v| in all; a
bf16 output is off by 2^-8 of the value more.  Where queries are not zero the
bounds are those of test_gpu_paged.py.
"""
import numpy as np
import pytest

from test_gpu_paged import U, Cache, as_bf16, attend, bw, f64, seen  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


class Long:
    """A cache made on the device: integers from -8 to 8 as values, normals as
    keys, NaN in every row that no position owns."""

    def __init__(self, seed, lens, Hkv, D, page, max_pages=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.Hkv, self.D, self.page = list(lens), Hkv, D, page
        need = [-(-n // page) for n in lens]
        total = sum(need) + 2
        self.kp = torch.randn((total, Hkv, page, D), generator=g, device="cuda",
                              dtype=torch.bfloat16)
        self.vp = torch.randint(-8, 9, (total, Hkv, page, D), generator=g,
                                device="cuda", dtype=torch.int8).bfloat16()
        ids = torch.randperm(total, generator=g, device="cuda").int()
        width = max_pages or max(need) + 1
        self.table = torch.full((len(lens), width), total + 9, device="cuda",
                                dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
            if lens[b] % page:
                for pool in (self.kp, self.vp):
                    pool[self.table[b, n - 1].long(), :, lens[b] % page:] = \
                        float("nan")
        for i in ids[at:].tolist():
            self.kp[i] = self.vp[i] = float("nan")
        self.len_d = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    @property
    def args(self):
        return self.kp, self.vp, self.table, self.len_d

    def rows(self, pool, b, n=None):
        """[n][Hkv][D] in 64 bits."""
        n = self.lens[b] if n is None else n
        ids = self.table[b, :-(-n // self.page)].long()
        return pool[ids].transpose(1, 2).reshape(-1, self.Hkv, self.D)[:n].double()


def check_means(c, out, G, window, sinks, lens=None):
    bits = 2.0 ** -8 if out.dtype is torch.bfloat16 else 0.0
    for b, n in enumerate(lens or c.lens):
        if n == 0:
            assert (out[b] == 0).all()
            continue
        v = c.rows(c.vp, b, n)
        if window:
            v = v[torch.from_numpy(seen(n - 1, window, sinks)).cuda()]
        ref = v.mean(0).repeat_interleave(G, 0)
        tol = 8 * U * v.abs().mean(0).repeat_interleave(G, 0)
        tol = tol + bits * (ref.abs() + tol)
        err = (out[b].double() - ref).abs()
        assert (err <= tol).all(), (b, n, float((err - tol).max()))


CLAIMED = [
    # H, Hkv, D, page, lens, window, sinks: tiles for which some are claimed,
    # then more than 64 tiles a CTA that are all dealt
    (16, 2, 128, 64, [600003, 0, 1] + [18000 + 37 * i for i in range(20)], 0, 0),
    (4, 4, 64, 16, [24000 + 11 * i for i in range(31)] + [5], 0, 0),
    (32, 8, 128, 256, [240001], 0, 0),
    (5, 1, 64, 128, [2900007], 0, 0),
    (16, 2, 128, 64, [130000] * 8, 120000, 130),
    (16, 2, 128, 64, [400003, 0, 1] + [12000 + 37 * i for i in range(20)], 0, 0),
    (4, 4, 64, 16, [16000 + 11 * i for i in range(31)] + [5], 0, 0),
    (32, 8, 128, 256, [160001], 0, 0),
    (10, 1, 64, 128, [1300007], 0, 0),
    (16, 1, 128, 32, [1260001, 63, 64, 65], 0, 0),
    (32, 2, 128, 64, [100000] * 8, 90000, 130),
]


@pytest.mark.parametrize("H,Hkv,D,page,lens,window,sinks", CLAIMED)
@pytest.mark.parametrize("bf16", [False, True])
def test_decode_counts_every_position_once(bw, H, Hkv, D, page, lens, window,
                                           sinks, bf16):
    c = Long(1, lens, Hkv, D, page)
    n = len(lens)
    q = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
    dtype = torch.bfloat16 if bf16 else torch.float32
    ws = torch.zeros((bw.bw_attn_paged_decode_workspace_bytes(n, H, Hkv, D),),
                     dtype=torch.uint8, device="cuda")
    for _ in range(3):
        out = torch.full((n, H, D), 9.0, dtype=dtype, device="cuda")
        bw.bw_attn_paged_decode(q, *c.args, window=window, sinks=sinks, out=out,
                                workspace=ws)
        assert bw.bw_device_error() == 0
        check_means(c, out, H // Hkv, window, sinks)


def test_decode_replays_with_other_lengths(bw):
    """One captured call serves lengths of every kind: all claimed, all dealt,
    none; a second graph shares the workspace."""
    H, Hkv, D, page = 16, 2, 128, 64
    full = [500000] + [24000 + i for i in range(24)]
    c = Long(2, full, Hkv, D, page)
    n = len(full)
    q = torch.zeros((n, H, D), dtype=torch.bfloat16, device="cuda")
    outs = [torch.zeros((n, H, D), device="cuda") for _ in range(2)]
    ws = torch.zeros((bw.bw_attn_paged_decode_workspace_bytes(n, H, Hkv, D),),
                     dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for o in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                bw.bw_attn_paged_decode(q, *c.args, out=o, workspace=ws)
            graphs.append(g)
        for lens in (full, [0] * n, [1] * n, [480017] + [23011 + i for i in range(24)],
                     [777] * n, full):
            # pages past a shorter length are used no more: no NaN needed there
            c.len_d.copy_(torch.tensor(lens))
            for g, o in zip(graphs, outs):
                o.fill_(9.0)
                g.replay()
            torch.cuda.synchronize()
            assert bw.bw_device_error() == 0
            for o in outs:
                check_means(c, o, H // Hkv, 0, 0, lens)


def test_decode_long_random(bw):
    """Scores that differ, over claimed units: against 64 bits."""
    H, Hkv, D, page = 8, 2, 128, 64
    lens = [960001, 20, 4000]
    c = Long(3, lens, Hkv, D, page)
    q = torch.randn((3, H, D), device="cuda").bfloat16()
    out = bw.bw_attn_paged_decode(q, *c.args, scale=0.2)
    assert bw.bw_device_error() == 0
    for b, n in enumerate(lens):
        k, v = c.rows(c.kp, b), c.rows(c.vp, b)
        for h in range(H):
            s = k[:, h // 4] @ q[b, h].double() * 0.2
            mass = (k[:, h // 4].abs() @ q[b, h].double().abs()).max() * 0.2
            w = torch.softmax(s, 0)
            ref = w @ v[:, h // 4]
            # a score: (D + 4) 2 u of its terms' mass; exponential and
            # rescaling: a rescaling at most for every doubling of the
            # maximum's bits and join, 64 u; sums: a warp adds 16 positions of
            # every tile in turn, at most n / 64 tiles, then the parts
            rel = (D + 4) * 2 * U * float(mass) + (64 + n / 64 + 16) * U
            tol = 2 * rel * 8
            assert float((out[b, h].double() - ref).abs().max()) <= tol, (b, h)


PREFILL = [
    # H, Hkv, D, page, lens, new, window, sinks: many items a CTA
    (8, 8, 128, 64, [20003], [20003], 0, 0),
    (8, 8, 64, 32, [9000, 13001], [9000, 12000], 0, 0),
    (24, 8, 128, 128, [9001, 5, 3000], [9001, 5, 2999], 700, 9),
    (16, 1, 64, 16, [4097, 1, 6000], [4097, 1, 5000], 0, 0),
    (4, 1, 128, 256, [60000], [70], 0, 0),
]


@pytest.mark.parametrize("H,Hkv,D,page,lens,new,window,sinks", PREFILL)
def test_prefill_counts_every_position_once(bw, H, Hkv, D, page, lens, new,
                                            window, sinks):
    c = Long(4, lens, Hkv, D, page)
    start = np.concatenate([[0], np.cumsum(new)])
    st = torch.from_numpy(start.astype(np.int32)).cuda()
    q = torch.zeros((int(start[-1]), H, D), dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
        bw.bw_attn_paged_prefill(q, *c.args, st, window=window, sinks=sinks,
                                 out=out)
        assert bw.bw_device_error() == 0
        for b, n in enumerate(lens):
            v = c.rows(c.vp, b)
            p = torch.arange(n - new[b], n, device="cuda")
            lo = (p - window + 1).clamp(min=0) if window else torch.zeros_like(p)
            s1 = lo.clamp(max=sinks)

            def sums(x):
                acc = torch.cat([torch.zeros_like(x[:1]), x.cumsum(0)])
                return (acc[p + 1] - acc[lo] + acc[s1]) / \
                    (p + 1 - lo + s1)[:, None, None]

            ref = sums(v).repeat_interleave(H // Hkv, 1)
            tol = 8 * U * sums(v.abs()).repeat_interleave(H // Hkv, 1)
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
            err = (out[int(start[b]):int(start[b + 1])].double() - ref).abs()
            assert (err <= tol).all(), (b, float((err - tol).max()))


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_scores_that_jump(bw, D):
    """The largest scores come in a tile's second half, in single positions
    and in later tiles, far above what came before."""
    lens, new, H, Hkv, page = [900, 390], [300, 390], 6, 2, 32
    c = Cache(52, lens, Hkv, D, page)
    rng = np.random.default_rng(9)
    for b, n in enumerate(lens):
        j = np.arange(n)
        g = np.where((j // 64) % 2 == 1, 6.0, 0.05) if b == 0 else \
            np.where(rng.random(n) < 0.02, 8.0 * (j + 50) / n, 0.2)
        c.k[b] = as_bf16(f64(c.k[b]) * g[:, None, None])
        for i in range(n):
            c.kp[int(c.table[b, i // page]), :, i % page] = c.k[b][i].cuda()
    start = np.concatenate([[0], np.cumsum(new)])
    q = as_bf16(4.0 * rng.standard_normal((int(start[-1]), H, D))).cuda()
    out = bw.bw_attn_paged_prefill(q, *c.args,
                                   torch.from_numpy(start.astype(np.int32)).cuda())
    assert bw.bw_device_error() == 0
    qf, got = f64(q), f64(out)
    for b, n in enumerate(new):
        kk, vv = f64(c.k[b]), f64(c.v[b])
        for i in range(n):
            p = lens[b] - n + i
            ref, tol = attend(qf[start[b] + i], kk, vv, D ** -0.5,
                              np.arange(p + 1), 2.0 ** -8)
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            assert (np.abs(got[start[b] + i] - ref) <= tol).all(), (b, p)


def test_offsets_past_31_bits(bw):
    """Pages 2^27 elements apart and token rows 1.2e9 elements apart."""
    H, Hkv, D, page, lens = 4, 2, 128, 16, [100, 171]
    stride, size = 1 << 27, Hkv * page * D
    n_pages = 34  # the last begin past 2^32 elements, 2^33 bytes
    pool = torch.empty((n_pages - 1) * stride + 2 * size, dtype=torch.bfloat16,
                       device="cuda")
    kp = pool.as_strided((n_pages, Hkv, page, D), (stride, page * D, D, 1))
    vp = pool.as_strided((n_pages, Hkv, page, D), (stride, page * D, D, 1), size)
    kp.fill_(float("nan"))
    vp.fill_(float("nan"))
    table = torch.full((2, 11), -1, dtype=torch.int32)
    table[0, :7] = torch.arange(33, 26, -1)
    table[1, :11] = torch.arange(16, 27)
    table = table.cuda()
    ld = 1_200_000_000
    big = torch.empty(2 * ld + 2 * (H + 2 * Hkv) * D, dtype=torch.bfloat16,
                      device="cuda")
    width = (H + 2 * Hkv) * D
    rng = np.random.default_rng(5)
    x = [as_bf16(rng.standard_normal((n, width))) for n in lens]
    c = Cache.__new__(Cache)
    c.k = [t.view(-1, H + 2 * Hkv, D)[:, H:H + Hkv] for t in x]
    c.v = [t.view(-1, H + 2 * Hkv, D)[:, H + Hkv:] for t in x]
    for b, n in enumerate(lens):
        for j in range(n):
            kp[int(table[b, j // page]), :, j % page] = c.k[b][j].cuda()
            vp[int(table[b, j // page]), :, j % page] = c.v[b][j].cuda()
    len_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    # one sequence's last three tokens, rows ld apart
    qkv = big.as_strided((3, width), (ld, 1))
    qkv.copy_(x[1][-3:])
    q_out = big.as_strided((3, H, D), (ld, D, 1), width)
    st = torch.tensor([0, 0, 3], dtype=torch.int32, device="cuda")
    bw.bw_qk_norm_rope_append(qkv, kp, vp, table, len_d, H, q_start=st,
                              q_out=q_out)
    assert bw.bw_device_error() == 0
    # the same call over small buffers
    kp2 = torch.zeros((n_pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp2 = torch.zeros_like(kp2)
    q2 = bw.bw_qk_norm_rope_append(qkv.contiguous(), kp2, vp2, table, len_d, H,
                                   q_start=st)
    assert torch.equal(q2, q_out)
    for j in range(lens[1] - 3, lens[1]):
        p = int(table[1, j // page])
        assert torch.equal(kp[p, :, j % page], kp2[p, :, j % page])
        assert torch.equal(vp[p, :, j % page], c.v[1][j].cuda())
        c.k[1][j] = kp[p, :, j % page].cpu()
    # attention: from and to rows ld apart
    out = big.as_strided((3, H, D), (ld, D, 1), width + H * D)
    bw.bw_attn_paged_prefill(q_out, kp, vp, table, len_d, st, out=out)
    one = big.as_strided((2, H, D), (ld, D, 1))
    bw.bw_attn_paged_decode(q_out[1:], kp, vp, table, len_d, out=one)
    assert bw.bw_device_error() == 0
    qf = f64(q_out)
    for i in range(3):
        p = lens[1] - 3 + i
        ref, tol = attend(qf[i], f64(c.k[1]), f64(c.v[1]), D ** -0.5,
                          np.arange(p + 1), 2.0 ** -8)
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert (np.abs(f64(out)[i] - ref) <= tol).all()
    for b in range(2):
        ref, tol = attend(qf[1 + b], f64(c.k[b]), f64(c.v[b]), D ** -0.5,
                          np.arange(lens[b]))
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert (np.abs(f64(one)[b] - ref) <= tol).all()


def test_one_workspace_under_calls_of_many_shapes(bw):
    """Decode of several shapes and split prefill, one after the other on one
    workspace that was zeroed once."""
    shapes = [(16, 2, 128, [960000]), (4, 4, 64, [720001]), (5, 1, 64, [77, 3]),
              (16, 1, 128, [1300000])]
    caches = [Long(6 + i, lens, Hkv, D, 64) for i, (_, Hkv, D, lens)
              in enumerate(shapes)]
    need = 0
    for H, Hkv, D, lens in shapes:
        need = max(need, bw.bw_attn_paged_decode_workspace_bytes(
            len(lens), H, Hkv, D), bw.bw_attn_paged_prefill_workspace_bytes(
                40, len(lens), H, Hkv, D))
    ws = torch.zeros((need,), dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 0, 2, 1, 3):
        (H, Hkv, D, lens), c = shapes[i], caches[i]
        q = torch.zeros((len(lens), H, D), dtype=torch.bfloat16, device="cuda")
        out = bw.bw_attn_paged_decode(q, *c.args, workspace=ws)
        check_means(c, out, H // Hkv, 0, 0)
        st = torch.tensor([0, 40] + [40] * (len(lens) - 1), dtype=torch.int32,
                          device="cuda")
        rows = torch.randn((40, H, D), device="cuda").bfloat16()
        got = bw.bw_attn_paged_prefill(rows, *c.args, st, workspace=ws)
        assert torch.equal(got, bw.bw_attn_paged_prefill(rows, *c.args, st))
        assert bw.bw_device_error() == 0


@pytest.mark.parametrize("H,Hkv,D,lens,new", [
    (8, 2, 128, [5000, 100], [60, 100]),     # split
    (8, 8, 64, [3000, 2500], [3000, 2500]),  # not split
])
def test_captured_prefill_and_append(bw, H, Hkv, D, lens, new):
    """Captured once, replayed with other tokens, lengths, ranges and pages:
    the same as eager calls, bit for bit."""
    c = Long(8, lens, Hkv, D, 64)
    tokens = sum(new)
    width = (H + 2 * Hkv) * D
    qkv = torch.zeros((tokens, width), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((tokens, H, D), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    st = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.zeros((bw.bw_attn_paged_prefill_workspace_bytes(
        tokens, 2, H, Hkv, D),), dtype=torch.uint8, device="cuda")

    def call():
        bw.bw_qk_norm_rope_append(qkv, *c.args, H, q_start=st, q_out=q)
        bw.bw_attn_paged_prefill(q, *c.args, st, window=600, sinks=3, out=out,
                                 workspace=ws)

    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            call()
    keep = c.kp.clone(), c.vp.clone()
    for step in range(3):
        n0 = [new[0], new[0] - 7, 0][step]
        n1 = [new[1], 5, new[1]][step]
        x = torch.randn((tokens, width), device="cuda").bfloat16()
        results = []
        for run in (g.replay, call):
            c.kp.copy_(keep[0])
            c.vp.copy_(keep[1])
            qkv.copy_(x)
            st.copy_(torch.tensor([0, n0, n0 + n1]))
            c.len_d.copy_(torch.tensor([lens[0] - 3 * step, lens[1]]))
            out.fill_(5.0)
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert bw.bw_device_error() == 0
            results.append([t.view(torch.int16).clone() for t in (q, out, c.kp, c.vp)])
        for a, b in zip(*results):
            assert torch.equal(a, b)
        assert (out[n0 + n1:] == 5.0).all()


@pytest.mark.parametrize("H,Hkv,D", [(20, 5, 128), (8, 8, 128), (6, 1, 64)])
def test_short_prompts_again_and_again(bw, H, Hkv, D):
    """Few tiles, copies that land late or early: the same every time."""
    lens = [200, 130, 517, 64]
    c = Long(14, lens, Hkv, D, 32)
    q = torch.randn((sum(lens), H, D), device="cuda").bfloat16()
    st = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32,
                      device="cuda")
    sweep = torch.empty(64 << 20, device="cuda")  # more than L2 holds
    want = bw.bw_attn_paged_prefill(q, *c.args, st)
    for i in range(200):
        if i % 4 == 0:
            sweep.fill_(i)
        assert torch.equal(want, bw.bw_attn_paged_prefill(q, *c.args, st))
    assert bw.bw_device_error() == 0


def test_calls_at_once_on_two_streams(bw):
    """Prefill, split and not, and decode beside each other, a workspace each."""
    H, Hkv, D, page = 16, 4, 128, 64
    c = Long(9, [30000, 4000, 700], Hkv, D, page)
    st = torch.tensor([0, 0, 3000, 3600], dtype=torch.int32, device="cuda")
    q = torch.randn((3600, H, D), device="cuda").bfloat16()
    few = torch.tensor([0, 40, 40, 45], dtype=torch.int32, device="cuda")
    calls = [lambda s: bw.bw_attn_paged_prefill(q, *c.args, st, stream=s),
             lambda s: bw.bw_attn_paged_decode(q[:3], *c.args, stream=s),
             lambda s: bw.bw_attn_paged_prefill(q[:45], *c.args, few, stream=s)]
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(12):
        got.append((i % 3, calls[i % 3](streams[(i // 2) % 2])))
    torch.cuda.synchronize()
    assert bw.bw_device_error() == 0
    for k, o in got:
        assert torch.equal(o, want[k])


def test_sequences_that_share_pages(bw):
    """The same pages in two sequences' tables, one of them longer."""
    H, Hkv, D, page = 8, 2, 128, 16
    c = Cache(10, [100, 70], Hkv, D, page)
    c.table_d[1, :4] = c.table_d[0, :4]
    c.k[1][:64], c.v[1][:64] = c.k[0][:64], c.v[0][:64]
    q = as_bf16(np.random.default_rng(2).standard_normal((2, H, D))).cuda()
    one = bw.bw_attn_paged_decode(q, *c.args, scale=0.1)
    st = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    two = bw.bw_attn_paged_prefill(q, *c.args, st, scale=0.1)
    assert bw.bw_device_error() == 0
    for b, n in enumerate(c.lens):
        ref, tol = attend(f64(q)[b], f64(c.k[b]), f64(c.v[b]), 0.1, np.arange(n))
        assert (np.abs(f64(one)[b] - ref) <= tol).all()
        ref, tol = attend(f64(q)[b], f64(c.k[b]), f64(c.v[b]), 0.1,
                          np.arange(n), 2.0 ** -8)
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert (np.abs(f64(two)[b] - ref) <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_nothing_to_see(bw, D):
    """Only empty sequences; only rows of no sequence."""
    H, Hkv, page = 6, 2, 16
    for n in (1, 300):
        c = Cache(11, [0] * n, Hkv, D, page)
        q = as_bf16(np.random.default_rng(2).standard_normal((n, H, D))).cuda()
        for dtype in (torch.float32, torch.bfloat16):
            out = torch.full((n, H, D), 9.0, dtype=dtype, device="cuda")
            bw.bw_attn_paged_decode(q, *c.args, out=out)
            assert (out == 0).all()
        st = torch.full((n + 1,), min(n, 3), dtype=torch.int32, device="cuda")
        out = torch.full((n, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
        bw.bw_attn_paged_prefill(q, *c.args, st, out=out)
        assert (out == 9.0).all()
        qkv = torch.ones((n, (H + 2 * Hkv) * D), dtype=torch.bfloat16, device="cuda")
        for starts in (st, None):
            out.fill_(9.0)
            bw.bw_qk_norm_rope_append(qkv, *c.args, H, q_start=starts, q_out=out)
            assert (out == 9.0).all()
        assert torch.isnan(c.pool).all()
        assert bw.bw_device_error() == 0


def test_largest_window_and_sinks(bw):
    H, Hkv, D, page, most = 4, 2, 128, 16, 2 ** 31 - 1
    c = Cache(12, [300, 41], Hkv, D, page)
    q = as_bf16(np.random.default_rng(2).standard_normal((2, H, D))).cuda()
    want = bw.bw_attn_paged_decode(q, *c.args)
    st = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    wide = bw.bw_attn_paged_prefill(q, *c.args, st)
    for window, sinks in ((most, 0), (most, most), (300, 0)):
        assert torch.equal(want, bw.bw_attn_paged_decode(
            q, *c.args, window=window, sinks=sinks))
        assert torch.equal(wide, bw.bw_attn_paged_prefill(
            q, *c.args, st, window=window, sinks=sinks))
    assert bw.bw_device_error() == 0
    for bad in (dict(window=2 ** 31), dict(window=2 ** 32), dict(sinks=2 ** 32),
                dict(window=-2 ** 32)):
        with pytest.raises(ValueError):
            bw.bw_attn_paged_decode(q, *c.args, **bad)
        with pytest.raises(ValueError):
            bw.bw_attn_paged_prefill(q, *c.args, st, **bad)


def test_decode_in_place_is_refused(bw):
    c = Cache(13, [30], 2, 128, 16)
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bw.BwError):
        bw.bw_attn_paged_decode(q, *c.args, out=q)
