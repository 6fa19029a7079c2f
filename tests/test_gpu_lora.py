"""Low-rank adapters beside a shared projection on a GB300, against plain
64-bit forms.

Tolerances (u = 2^-24): A x multiplies exactly and sums K terms, each step
rounded or truncated: K 2 u of the sum of magnitudes; its scaling 3 u and the
two bf16 values that keep it 2^-17 of it.  B u multiplies exactly and sums 2 R
terms: (2 R) 2 u of the sum of magnitudes, the addition to y 2 u of both.  The
output's own rounding: 2^-8 of the value.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24


@pytest.fixture(scope="module")
def bw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_lib
    build_lib()
    import bit_gemv_bitlinear_gb300 as bw
    return bw


def f64(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, seed, M, N, K, R, n, ids=None, scaled=True):
        rng = np.random.default_rng(seed)
        self.M, self.N, self.K, self.R, self.n = M, N, K, R, n

        def normal(*shape, gain=1.0):
            return torch.from_numpy(
                (gain * rng.standard_normal(shape)).astype(np.float32)).cuda()

        self.x = torch.from_numpy(
            rng.integers(-128, 128, (M, K)).astype(np.int8)).cuda()
        self.s = torch.from_numpy(
            rng.uniform(10, 60, M).astype(np.float32)).cuda()
        self.A = normal(n, R, K, gain=K ** -0.5).bfloat16()
        self.B = normal(n, N, R, gain=R ** -0.5).bfloat16()
        self.scale = torch.from_numpy(
            rng.uniform(-2, 2, n).astype(np.float32)).cuda() if scaled else None
        if ids is None:
            ids = rng.integers(-1, n, M)
        self.ids = np.asarray(ids, np.int32)
        self.adapter = torch.from_numpy(self.ids).cuda()
        self.y = normal(M, N).bfloat16()

    def run(self, bw, y=None, **kw):
        return bw.bw_lora_add(self.y if y is None else y, self.x, self.s, self.A,
                              self.B, self.adapter, scale=self.scale, **kw)

    def check(self, got, y=None, skip=()):
        y = f64(self.y if y is None else y)
        want, tol = y.copy(), np.zeros_like(y)
        x, s = f64(self.x), f64(self.s)
        for a in range(self.n):
            rows = [m for m in range(self.M) if self.ids[m] == a and m not in skip]
            if not rows:
                continue
            c = 1.0 if self.scale is None else float(self.scale[a])
            A, B = f64(self.A[a]), f64(self.B[a])
            xs = x[rows] * (c / s[rows])[:, None]
            u, mass = xs @ A.T, np.abs(xs) @ np.abs(A).T
            off = self.K * 2 * U * mass + (3 * U + 2.0 ** -17) * np.abs(u)
            d = u @ B.T
            size = np.abs(u) @ np.abs(B).T
            tol[rows] += off @ np.abs(B).T + 2 * self.R * 2 * U * size
            tol[rows] += 2 * U * (np.abs(d) + np.abs(y[rows]))
            want[rows] += d
        tol[tol > 0] += 2.0 ** -8 * np.abs(want)[tol > 0]
        bad = np.abs(f64(got) - want) > tol
        bad[list(skip)] = False
        assert not bad.any(), np.argwhere(bad)[:5]


CASES = [
    # M, N, K, R, n
    (1, 40, 24, 8, 1),
    (1, 1, 4, 8, 2),
    (1, 2560, 2560, 16, 8),
    (2, 31, 36, 24, 3),
    (15, 32, 64, 32, 1),
    (16, 33, 100, 40, 3),
    (17, 64, 256, 128, 5),
    (61, 130, 516, 16, 48),
    (255, 96, 260, 8, 70),
    (256, 40, 128, 64, 300),
    (257, 264, 520, 64, 4),
    (300, 1021, 68, 40, 20),
    (333, 513, 1028, 128, 3),
    (1000, 256, 512, 16, 2),
    (12, 13824, 72, 16, 5),          # several clusters a tile
    (40, 9000, 64, 128, 7),
    (130, 4100, 40, 32, 3),
    (512, 72, 48, 24, 200),
    (512, 72, 48, 24, 1),
    (513, 8, 64, 8, 3),
    (640, 136, 260, 24, 40),
    (700, 200, 132, 128, 9),
    (1025, 2568, 512, 64, 3),
]


@pytest.mark.parametrize("M,N,K,R,n", CASES)
@pytest.mark.parametrize("scaled", [True, False])
def test_mixed_rows(bw, M, N, K, R, n, scaled):
    c = Case(M + N, M, N, K, R, n, scaled=scaled)
    out = torch.full_like(c.y, float("nan"))
    assert c.run(bw, out=out) is out
    c.check(out)
    assert bw.bw_device_error() == 0


@pytest.mark.parametrize("M", [64, 512, 600, 4096])
def test_rows_by_request(bw, M):
    """Requests one after the other, as prompts lie in a batch."""
    c = Case(M, M, 200, 128, 32, 6, ids=np.arange(M) * 6 // M)
    c.check(c.run(bw, out=torch.empty_like(c.y)))


@pytest.mark.parametrize("M", [40, 400, 530])
@pytest.mark.parametrize("off,pad", [(0, 24), (8, 0), (3, 2)])
def test_columns_of_a_fused_projection(bw, M, off, pad):
    """In place and into columns of a wider buffer; the others stay."""
    c = Case(M, M, 72, 64, 16, 4)
    wide = torch.full((M, off + 72 + pad), 3.0, dtype=torch.bfloat16, device="cuda")
    view = wide[:, off:off + 72]
    view.copy_(c.y)
    assert c.run(bw, y=view) is view
    c.check(view)
    assert (wide[:, :off] == 3.0).all() and (wide[:, off + 72:] == 3.0).all()
    out = torch.full((M, 80), 5.0, dtype=torch.bfloat16, device="cuda")
    c.run(bw, out=out[:, :72])
    c.check(out[:, :72])
    assert (out[:, 72:] == 5.0).all()


@pytest.mark.parametrize("M", [20, 300, 520])
def test_rows_without_an_adapter(bw, M):
    c = Case(M, M, 64, 64, 16, 4, ids=np.full(M, -1))
    out = torch.zeros_like(c.y)
    c.run(bw, out=out)
    assert torch.equal(out, c.y)
    kept = c.y.clone()
    c.run(bw)
    assert torch.equal(c.y, kept)


@pytest.mark.parametrize("M", [20, 300, 520])
def test_bad_adapter_numbers(bw, M):
    """Reported, and those rows are as without one."""
    c = Case(M, M, 64, 64, 16, 4)
    for m, bad in ((0, 4), (3, -2), (M - 1, 2 ** 31 - 1), (7, -2 ** 31)):
        c.ids[m] = bad
    c.adapter.copy_(torch.from_numpy(c.ids))
    out = c.run(bw, out=torch.empty_like(c.y))
    with pytest.raises(bw.BwError) as e:
        bw.bw_device_error()
    assert e.value.status == 1  # the caller's mistake, not a time-out
    assert bw.bw_device_error() == 0
    c.check(out)
    assert torch.equal(out[[0, 3, M - 1, 7]], c.y[[0, 3, M - 1, 7]])


@pytest.mark.parametrize("M", [20, 300, 520])
def test_what_is_not_finite_stays_in_its_rows(bw, M):
    c = Case(M, M, 64, 64, 16, 4, ids=np.arange(M) % 4)
    c.A[1, 3, 5] = float("nan")
    c.B[2, 7, 1] = float("inf")
    c.s[4] = float("nan")  # a row of adapter 0, as a bad norm leaves it
    out = c.run(bw, out=torch.empty_like(c.y))
    skip = [m for m in range(M) if m % 4 in (1, 2) or m == 4]
    c.check(out, skip=skip)
    assert out[1::4].isnan().all() and out[4].isnan().all()
    assert not out[2::4, 7].isfinite().any()
    assert out[2::4, 8:].isfinite().all()


def test_inputs_at_odd_places(bw):
    """x on 4 bytes, where 8 codes are no vector."""
    c = Case(3, 50, 64, 64, 16, 4)
    buf = torch.zeros(50 * 64 + 4, dtype=torch.int8, device="cuda")
    x = buf[4:].view(50, 64)
    x.copy_(c.x)
    c.x = x
    c.check(c.run(bw, out=torch.empty_like(c.y)))


@pytest.mark.parametrize("M", [18, 520])
def test_far_adapters(bw, M):
    """Offsets beyond 32 bits: 40000 adapters of 128 x 516."""
    n, R, K, N = 40000, 128, 516, 8
    torch.cuda.empty_cache()
    c = Case(5, M, N, K, R, 1, ids=np.zeros(M))
    A = torch.empty((n, R, K), dtype=torch.bfloat16, device="cuda")
    B = torch.empty((n, N, R), dtype=torch.bfloat16, device="cuda")
    A[n - 1], B[n - 1] = c.A[0], c.B[0]
    scale = torch.zeros(n, device="cuda")
    scale[n - 1] = c.scale[0]
    ids = torch.full((M,), n - 1, dtype=torch.int32, device="cuda")
    out = bw.bw_lora_add(c.y, c.x, c.s, A, B, ids, scale=scale,
                         out=torch.empty_like(c.y))
    c.check(out)


@pytest.mark.parametrize("M", [30, 300, 600])
def test_captured_and_on_another_stream(bw, M):
    """A replayed graph follows the adapter numbers on the device."""
    c = Case(M, M, 96, 128, 16, 9)
    ws = torch.empty(bw.bw_lora_workspace_bytes(M, 16), dtype=torch.uint8,
                     device="cuda")
    out = torch.zeros_like(c.y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run(bw, out=out, workspace=ws, stream=side)
    side.synchronize()
    c.check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(bw, out=out, workspace=ws)
    for seed in (1, 2):
        c.ids = np.random.default_rng(seed).integers(-1, 9, M).astype(np.int32)
        c.adapter.copy_(torch.from_numpy(c.ids))
        graph.replay()
        c.check(out)


@pytest.mark.parametrize("M", [1, 60, 600])
def test_two_calls_at_once(bw, M):
    """On two streams, each with a workspace of its own."""
    a, b = Case(21, M, 512, 640, 16, 9), Case(22, M, 512, 640, 16, 9)
    outs = [torch.zeros_like(c.y) for c in (a, b)]
    size = bw.bw_lora_workspace_bytes(M, 16)
    ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, o, w, st in zip((a, b), outs, ws, streams):
            c.run(bw, out=o, workspace=w, stream=st)
    torch.cuda.synchronize()
    a.check(outs[0])
    b.check(outs[1])


def test_same_result_twice(bw):
    c = Case(9, 200, 640, 640, 64, 20)
    first = c.run(bw, out=torch.empty_like(c.y))
    assert torch.equal(first, c.run(bw, out=torch.empty_like(c.y)))


def test_refusals(bw):
    c = Case(1, 4, 64, 64, 16, 4)

    def refused(error, **kw):
        a = dict(y=c.y, x=c.x, s=c.s, A=c.A, B=c.B, adapter=c.adapter,
                 scale=c.scale)
        a.update(kw)
        with pytest.raises(error):
            bw.bw_lora_add(**a)

    refused(ValueError, x=c.x[:3])
    refused(TypeError, x=c.x.int())
    refused(ValueError, s=c.s[:3])
    refused(ValueError, B=c.B[:3])
    refused(ValueError, B=c.B.transpose(1, 2))
    refused(TypeError, adapter=c.adapter.long())
    refused(ValueError, scale=c.scale[:2])
    refused(ValueError, y=c.y.t())
    refused(ValueError, out=c.y[:, :60])
    refused(ValueError, A=c.A[0])
    refused(bw.BwError, A=c.A[:, :12].contiguous(), B=c.B[:, :, :12].contiguous())
    refused(bw.BwError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert bw.bw_device_error() == 0
