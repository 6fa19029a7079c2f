"""Attention of a batch that shares a prefix (GB300) against a plain 64-bit
form.

Every row of the pools that no position owns holds NaN, and every table entry
that a call should not use is out of range, so a result that is right shows
that neither is used.  Tolerances: those of test_gpu_paged.py for weights of
bf16 (a score is off by at most (D + 4) 2 u of its sum of magnitudes, a weight
by that, 8 u and n u of the sums, and 2^-8 for its rounding; an output by twice
the former of the largest |v|, and the mean of |v| times 2^-8; its own rounding
2^-8 of it).
"""
import numpy as np
import pytest

from test_gpu_paged import U, as_bf16, bw, f64  # noqa: F401

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


class Batch:
    """own: positions of each sequence behind the prefix; -k: k positions fewer
    than the prefix has, None: an empty sequence."""

    def __init__(self, seed, shared, own, H, Hkv, D, page, extra=0, gain=1.0,
                 spare=1):
        self.rng = rng = np.random.default_rng(seed)
        self.shared, self.H, self.Hkv, self.D, self.page = shared, H, Hkv, D, page
        self.lens = [0 if x is None else shared + x for x in own]
        first = shared // page
        common = -(-shared // page)
        mine = [max(0, -(-n // page) - first) if n > shared else 0 for n in self.lens]
        self.n_pages = common + sum(mine) + 2
        ids = rng.permutation(self.n_pages)
        self.max_pages = max([first + m for m in mine] + [1]) + spare
        table = np.full((len(own), self.max_pages), self.n_pages + 3, np.int32)
        table[:, ::2] = -5
        shape = (self.n_pages, Hkv, page, D)
        pools = [torch.full(shape, float("nan"), dtype=torch.bfloat16) for _ in "kv"]
        kd = [as_bf16(gain * rng.standard_normal((shared, Hkv, D))),
              as_bf16(rng.standard_normal((shared, Hkv, D)))]
        self.common = ids[:common].astype(np.int32)

        def put(rows, pages, start):
            for which in range(2):
                for i, p in enumerate(pages):
                    lo, hi = max(i * page, start), min((i + 1) * page, start + len(rows[which]))
                    if lo < hi:
                        pools[which][p, :, lo - i * page:hi - i * page] = \
                            rows[which][lo - start:hi - start].transpose(0, 1)

        put(kd, self.common, 0)
        self.k, self.v = [], []
        at = common
        for b, n in enumerate(self.lens):
            rows = [as_bf16(rng.standard_normal((max(0, n - shared), Hkv, D)))
                    for _ in "kv"]
            pages = ids[at:at + mine[b]]
            at += mine[b]
            table[b, first:first + mine[b]] = pages
            put(rows, [0] * first + list(pages), shared)
            self.k.append(torch.cat((kd[0][:n], rows[0])).double())
            self.v.append(torch.cat((kd[1][:n], rows[1])).double())
        size = Hkv * page * D
        pool = torch.full((2, self.n_pages, size + extra), float("nan"),
                          dtype=torch.bfloat16, device="cuda")
        self.kp = pool[0, :, :size].view(shape)
        self.vp = pool[1, :, :size].view(shape)
        self.kp.copy_(pools[0])
        self.vp.copy_(pools[1])
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        # entries past the prefix are not used either
        self.shared_table = torch.tensor(list(self.common) + [-9],
                                         dtype=torch.int32, device="cuda")
        self.shared_len = torch.tensor([shared], dtype=torch.int32, device="cuda")
        self.q = as_bf16(rng.standard_normal((len(own), H, D))).cuda()

    @property
    def args(self):
        return (self.kp, self.vp, self.table, self.kv_len, self.shared_table,
                self.shared_len)

    def run(self, bw, **kw):
        return bw.bw_attn_paged_shared(self.q, *self.args, **kw)

    def check(self, got, scale=None, seqs=None):
        H, Hkv, D = self.H, self.Hkv, self.D
        scale = 1.0 / D ** 0.5 if scale is None else scale
        for b in range(len(self.lens)) if seqs is None else seqs:
            n = self.lens[b]
            g = got[b].double().cpu()
            if n == 0:
                assert (g == 0).all()
                continue
            q = self.q[b].double().cpu().view(Hkv, H // Hkv, D)
            k, v = self.k[b].transpose(0, 1), self.v[b].transpose(0, 1)
            s = (q @ k.transpose(1, 2)) * scale
            mass = (q.abs() @ k.abs().transpose(1, 2)).amax(2, keepdim=True) * scale
            w = torch.softmax(s, 2)
            want = w @ v
            rel = (D + 4) * 2 * U * mass + (8 + n) * U
            tol = 2 * rel * v.abs().amax(1, keepdim=True) + 2.0 ** -8 * (w @ v.abs())
            tol = tol + 2.0 ** -8 * want.abs()
            off = (g.view_as(want) - want).abs()
            assert (off <= tol).all(), (b, n, float((off / tol).max()))


CASES = [
    # H, Hkv, D, page, shared, own, extra
    (20, 5, 128, 16, 1027, [1, 30, 180, 7], 0),
    (20, 5, 128, 64, 1, [1], 0),
    (20, 5, 128, 64, 0, [1, 700, None], 0),          # nothing is shared
    (20, 5, 128, 64, 700, [0, 0, -1, -699, None], 0),  # nothing of one's own
    (20, 5, 128, 128, 256, [1, 5, -128, -129, -255, 64, None, 3], 24),
    (20, 5, 128, 32, 2500, [i * 7 % 90 for i in range(33)], 0),   # 2 query tiles
    (20, 5, 128, 64, 900, [i * 11 % 150 - 20 for i in range(70)], 0),
    (8, 8, 128, 16, 333, [3] * 129, 0),
    (16, 1, 64, 256, 5000, [100, None, 40, -4000, 1, 900, 17, 2, 3], 0),
    (16, 1, 128, 16, 129, [5] * 17, 0),
    (7, 1, 64, 32, 127, [1, 2, 3], 8),
    (32, 4, 64, 32, 640, [i % 40 for i in range(100)], 0),
    (12, 4, 64, 64, 1999, [65, 130], 0),
    (64, 64, 128, 16, 200, [1, 20], 0),
    (5, 1, 128, 128, 6001, [1, 2], 0),
    (28, 4, 128, 16, 4100, [3], 0),
]


@pytest.mark.parametrize("H,Hkv,D,page,shared,own,extra", CASES)
def test_shared(bw, H, Hkv, D, page, shared, own, extra):  # noqa: F811
    c = Batch(31, shared, own, H, Hkv, D, page, extra)
    out = torch.full((len(own), H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    assert c.run(bw, out=out) is out
    assert bw.bw_device_error() == 0
    c.check(out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("shared", [126, 127, 128, 129, 255, 256, 257, 383, 385])
def test_ends_of_tiles(bw, D, n, shared):  # noqa: F811
    c = Batch(shared, shared, [(i * 13) % 70 - 1 for i in range(n)], 8, 2, D, 32)
    c.check(c.run(bw))
    assert bw.bw_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [2, 40])
def test_scores_that_rise(bw, D, n):  # noqa: F811
    """The maximum moves by hundreds from tile to tile, and in either part."""
    c = Batch(5, 1500, [30 + i for i in range(n)], 8, 2, D, 16, gain=0.0)
    rise = torch.linspace(0, 40, 1500)
    k = torch.zeros(1500, 2, D)
    k[:, :, 0] = rise[:, None]
    k = k.bfloat16()
    for i, p in enumerate(c.common):
        part = k[i * 16:(i + 1) * 16]
        c.kp[int(p), :, :len(part)] = part.transpose(0, 1).cuda()
    c.q[:, :, 0] = 30.0
    c.q[n - 1, :, 0] = -30.0
    for b in range(n):
        c.k[b][:1500] = k.double()
    c.check(c.run(bw))
    c.check(c.run(bw, scale=0.5), scale=0.5)


@pytest.mark.parametrize("D", [64, 128])
def test_what_is_not_finite(bw, D):  # noqa: F811
    """NaN in a query stays in its head, scores of +infinity give NaN there,
    as do scores that are all -infinity."""
    c = Batch(6, 300, [20] * 9, 8, 2, D, 16)
    c.q[2, 3, 5] = float("nan")
    c.q[4, 1] = 3e38
    c.q[7, 6, 2] = float("-inf")
    out = c.run(bw)
    assert out[2, 3].isnan().all() and out[4, 1].isnan().all()
    assert out[7, 6].isnan().all()
    out[2, 3] = out[4, 1] = out[7, 6] = 0.0
    assert out.isfinite().all()
    c.check(out, seqs=[0, 1, 3, 5, 6, 8])
    # all scores -infinity: every key positive, a query of -infinity
    c = Batch(7, 300, [20] * 3, 2, 2, D, 16)
    c.kp.copy_(c.kp.abs() + 0.25)
    c.q[1, 0] = float("-inf")
    out = c.run(bw)
    assert out[1, 0].isnan().all()
    assert out[0].isfinite().all() and out[1, 1].isfinite().all()


def test_as_the_decode_call(bw):  # noqa: F811
    """The same sequences with the shared pages in their own tables."""
    c = Batch(8, 1024, [i * 3 + 1 for i in range(50)], 20, 5, 128, 64)
    table = c.table.clone()
    table[:, :1024 // 64] = c.shared_table[:-1]
    want = bw.bw_attn_paged_decode(c.q, c.kp, c.vp, table, c.kv_len)
    got = c.run(bw)
    c.check(got)
    assert float((got.float() - want).abs().max()) < 0.03 * float(want.abs().max())
    # and what the table holds there makes no difference
    assert torch.equal(got, bw.bw_attn_paged_shared(
        c.q, c.kp, c.vp, table, c.kv_len, c.shared_table, c.shared_len))


def test_strided_rows(bw):  # noqa: F811
    c = Batch(9, 400, [3, 9, None, -7, 40], 6, 2, 64, 16)
    wide = torch.zeros(5, 8, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, :6] = c.q
    c.q = wide[:, :6]
    out = torch.full((5, 10, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    c.run(bw, out=out[:, :6])
    c.check(out[:, :6])
    assert (out[:, 6:] == 4.0).all()


def bad(bw):  # noqa: F811
    with pytest.raises(bw.BwError) as e:
        bw.bw_device_error()
    assert e.value.status == 1


@pytest.mark.parametrize("D,n", [(64, 5), (128, 5), (128, 50)])
def test_bad_numbers_on_the_device(bw, D, n):  # noqa: F811
    """Reported; nothing outside the buffers is used, and the call after it is
    as ever."""
    c = Batch(10, 500, [i % 9 + 1 for i in range(n)], 8, 2, D, 16)
    want = c.run(bw)
    assert bw.bw_device_error() == 0
    good_len, good_table = c.kv_len.clone(), c.shared_table.clone()
    for n_bad in (-1, 16 * len(good_table) + 1, 2 ** 31 - 1, -2 ** 31):
        c.shared_len.fill_(n_bad)
        c.run(bw)
        bad(bw)
    c.shared_len.fill_(500)
    for page in (-1, c.n_pages, 2 ** 31 - 1):
        c.shared_table[3] = page
        out = c.run(bw)
        bad(bw)
        assert out.isfinite().all()  # zeros are read
        c.shared_table.copy_(good_table)
    for length in (-1, 2 ** 31 - 1, -2 ** 31, 16 * c.max_pages + 1):
        c.kv_len[1] = length
        out = c.run(bw)
        bad(bw)
        assert (out[1] == 0).all()
        c.kv_len.copy_(good_len)
        c.check(out, seqs=[0] + list(range(2, n)))
    entry = c.table[2, 500 // 16].clone()
    c.table[2, 500 // 16] = c.n_pages
    out = c.run(bw)
    bad(bw)
    c.check(out, seqs=[0, 1] + list(range(3, n)))
    c.table[2, 500 // 16] = entry
    assert torch.equal(c.run(bw), want)
    assert bw.bw_device_error() == 0


@pytest.mark.parametrize("n", [6, 40])
def test_captured(bw, n):  # noqa: F811
    """A replayed graph follows the lengths on the device, the prefix's too."""
    c = Batch(11, 640, [30 + i for i in range(n)], 8, 2, 128, 32)
    ws = torch.zeros(bw.bw_attn_paged_shared_workspace_bytes(n, 8, 2, 128),
                     dtype=torch.uint8, device="cuda")
    out = torch.zeros((n, 8, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(bw, out=out, workspace=ws, stream=side)
    side.synchronize()
    c.check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(bw, out=out, workspace=ws)
        c.run(bw, out=out, workspace=ws)
    k, v = c.k, c.v
    for less in (0, 5, 33):
        c.lens = [max(0, 640 + 30 + b - less * b) for b in range(n)]
        c.kv_len.copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.k = [x[:m] for x, m in zip(k, c.lens)]
        c.v = [x[:m] for x, m in zip(v, c.lens)]
        graph.replay()
        c.check(out)
    # a shorter prefix: the rest of it is looked up by sequence
    c.shared_len.fill_(96)
    c.table[:, :20] = c.shared_table[:20]
    graph.replay()
    c.check(out)
    assert bw.bw_device_error() == 0


def test_one_workspace_for_all_paged_calls(bw):  # noqa: F811
    c = Batch(12, 700, [3 + i for i in range(40)], 20, 5, 128, 64)
    d = Batch(13, 300, [2, 900, None], 32, 4, 64, 16)
    size = max(bw.bw_attn_paged_shared_workspace_bytes(40, 20, 5, 128),
               bw.bw_attn_paged_shared_workspace_bytes(3, 32, 4, 64), 20 << 20)
    ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    table = c.table.clone()
    table[:, :700 // 64] = c.shared_table[:700 // 64]
    for b in range(40):  # the page that the prefix ends in, whole
        p = int(table[b, 10])
        c.kp[p, :, :60] = c.kp[int(c.shared_table[10]), :, :60]
        c.vp[p, :, :60] = c.vp[int(c.shared_table[10]), :, :60]
    for _ in range(2):
        c.check(c.run(bw, workspace=ws))
        d.check(d.run(bw, workspace=ws))
        dec = bw.bw_attn_paged_decode(c.q, c.kp, c.vp, table, c.kv_len, workspace=ws)
        c.check(dec)
        d.check(d.run(bw, workspace=ws))
        start = torch.arange(41, dtype=torch.int32, device="cuda")
        c.check(bw.bw_attn_paged_prefill(c.q, c.kp, c.vp, table, c.kv_len, start,
                                         workspace=ws))
    assert bw.bw_device_error() == 0
    ws[0] = 1  # a workspace that was not zeroed is reported
    c.run(bw, workspace=ws)
    bad(bw)


def test_two_calls_at_once(bw):  # noqa: F811
    """On two streams, each with a workspace of its own, beside other work."""
    a = Batch(31, 900, [5 + i for i in range(40)], 20, 5, 128, 64)
    b = Batch(32, 700, [i for i in range(33)], 16, 2, 64, 16)
    outs = [torch.zeros_like(c.q) for c in (a, b)]
    ws = [torch.zeros(bw.bw_attn_paged_shared_workspace_bytes(
        len(c.lens), c.H, c.Hkv, c.D), dtype=torch.uint8, device="cuda") for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    x = torch.zeros(1 << 24, device="cuda")
    torch.cuda.synchronize()
    for _ in range(30):
        for c, o, w, st in zip((a, b), outs, ws, streams):
            with torch.cuda.stream(st):
                c.run(bw, out=o, workspace=w)
        x.add_(1.0)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])
    assert bw.bw_device_error() == 0


def test_long_prefix(bw):  # noqa: F811
    """100001 positions, against 64 bits on the GPU; many tiles a CTA."""
    shared, n, H, Hkv, D, page = 100001, 5, 8, 2, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    pages = -(-shared // page)

    def normal(*s):
        return torch.randn(s, device="cuda", generator=gen).bfloat16()

    kp, vp = normal(pages + n, Hkv, page, D), normal(pages + n, Hkv, page, D)
    order = torch.randperm(pages + n, device="cuda", generator=gen).int()
    table = torch.full((n, pages + 1), -1, dtype=torch.int32, device="cuda")
    table[:, pages - 1] = order[pages:]
    lens = [shared + 3 * b for b in range(n)]
    q = normal(n, H, D)
    got = bw.bw_attn_paged_shared(
        q, kp, vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
        order[:pages].contiguous(),
        torch.tensor([shared], dtype=torch.int32, device="cuda"))
    assert bw.bw_device_error() == 0
    off = shared - (pages - 1) * page
    for b in range(n):
        def rows(pool):
            x = pool[order[:pages].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :shared]
            return torch.cat((x, pool[int(table[b, pages - 1])][:, off:off + 3 * b]), 1).double()

        k, v = rows(kp), rows(vp)
        s = q[b].double().view(Hkv, H // Hkv, D) @ k.transpose(1, 2) / D ** 0.5
        w = torch.softmax(s, 2)
        want = (w @ v).view(H, D)
        # the weights' roundings are independent: n of them, of at most 2^-8
        # each, give the mean of |v| times 2^-8 at most
        tol = 2.0 ** -8 * (w @ v.abs()).view(H, D) + 2.0 ** -8 * want.abs()
        tol = tol + 2 * ((D + 4) * 2 * U * 40 + lens[b] * U) * v.abs().max()
        assert ((got[b].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("n,shared,own,H,Hkv,D", [
    (64, 200, 9000, 20, 5, 128),     # units claimed while the call runs
    (200, 5000, 2500, 32, 4, 64),
    (1500, 300, 120, 32, 8, 64),     # more items than SMs: all tiles in one order
    (4096, 150, 70, 8, 8, 128),
    (600, 4000, 3, 64, 64, 64),
    (3, 60000, 30000, 16, 1, 128),
])
def test_against_the_decode_call(bw, n, shared, own, H, Hkv, D):  # noqa: F811
    """Large batches: the decode call over tables that hold the shared pages too
    (fp32 output, which has tests of its own against 64 bits).  The prefix's
    weights are rounded to bf16, 2^-8 of the mean of |v| at most; their
    roundings are independent, and normal values' mean of |v| is below 1."""
    page = 64
    gen = torch.Generator(device="cuda").manual_seed(n)
    lens = [0 if b % 97 == 5 else shared + (own * (b * 0.618 % 1.0)).__int__()
            for b in range(n)]
    first, common = shared // page, -(-shared // page)
    mine = [max(0, -(-x // page) - first) for x in lens]
    total = common + sum(mine)
    kp = torch.randn((total, Hkv, page, D), device="cuda", generator=gen).bfloat16()
    vp = torch.randn((total, Hkv, page, D), device="cuda", generator=gen).bfloat16()
    order = torch.randperm(total, device="cuda", generator=gen).int()
    table = torch.full((n, first + max(mine)), -1, dtype=torch.int32)
    at = common
    for b in range(n):
        table[b, first:first + mine[b]] = order[at:at + mine[b]].cpu()
        at += mine[b]
    table = table.cuda()
    whole = table.clone()
    whole[:, :first] = order[:first]
    part = shared - first * page  # the page that the prefix ends in, copied
    if part:
        for b in range(n):
            if lens[b] > first * page:
                for pool in (kp, vp):
                    pool[int(whole[b, first]), :, :part] = pool[int(order[first]), :, :part]
    q = (0.7 * torch.randn((n, H, D), device="cuda", generator=gen)).bfloat16()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.zeros(bw.bw_attn_paged_shared_workspace_bytes(n, H, Hkv, D),
                     dtype=torch.uint8, device="cuda")
    want = bw.bw_attn_paged_decode(q, kp, vp, whole, kv_len)
    for _ in range(2):
        got = bw.bw_attn_paged_shared(
            q, kp, vp, table, kv_len, order[:common].contiguous(),
            torch.tensor([shared], dtype=torch.int32, device="cuda"), workspace=ws)
        off = (got.float() - want).abs()
        assert float((off - 2.0 ** -8 * want.abs()).max()) <= 2.0 ** -8
    assert bw.bw_device_error() == 0


def test_refusals(bw):  # noqa: F811
    c = Batch(14, 64, [3, 4], 8, 2, 64, 16)

    def refused(error, **kw):
        a = dict(q=c.q, k_pages=c.kp, v_pages=c.vp, page_table=c.table,
                 kv_len=c.kv_len, shared_table=c.shared_table,
                 shared_len=c.shared_len)
        a.update(kw)
        with pytest.raises(error):
            bw.bw_attn_paged_shared(**a)

    refused(TypeError, shared_len=64)
    refused(TypeError, shared_len=c.shared_len.long())
    refused(ValueError, shared_len=c.shared_len.cpu())
    refused(ValueError, shared_table=c.shared_table[:0])
    refused(TypeError, shared_table=None)
    refused(ValueError, q=c.q[0])
    refused(ValueError, out=c.q[:1])
    refused(TypeError, out=c.q.float())
    refused(bw.BwError, scale=0.0)
    refused(bw.BwError, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert bw.bw_device_error() == 0
