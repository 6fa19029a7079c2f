"""A decoder layer's step for a batch of requests, made of the public calls
(GB300): norms with 8-bit codes, W2A8 projections, adapters, the append to the
paged cache, the attention behind a shared prefix, and the gated feed-forward
([W2A8] §一, §4.1, §六 of the kernel page).

Every stage is checked against a plain 64-bit form of the same inputs, so
tolerances do not add up: those of the calls' own tests, and 2^-8 of the value
for a projection's bf16 output (its int32 sums are exact).  Then the same steps
replayed from a graph, bit for bit.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
THETA = 10000.0


@pytest.fixture(scope="module")
def bw():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conftest import build_lib
    build_lib()
    import bit_gemv_bitlinear_gb300 as bw
    return bw


class Linear:
    """Ternary weights [N][K] in the device layout, and as numbers."""

    def __init__(self, bw, gen, N, K, bounds):
        W = torch.randn((N, K), device="cuda", generator=gen) * 0.05
        canon, self.ws = bw.bw_quant_weight(W, bounds)
        self.packed = bw.bw_repack(canon, N, K)
        self.bounds, self.N, self.K = bounds, N, K
        shifts = torch.arange(0, 8, 2, device="cuda")
        w = (canon[..., None].int() >> shifts & 3) - 1
        scale = torch.cat([self.ws[i].double().expand(b - a) for i, (a, b) in
                           enumerate(zip(bounds, bounds[1:]))])
        self.w = w.reshape(N, K).double() * scale[:, None]

    def run(self, bw, q, s, y):
        return bw.bw_gemv_w2a8(q, self.packed, s, self.ws, self.bounds, self.N,
                               self.K, y=y)

    def check(self, q, s, y):
        want = q.double() @ self.w.T / s.double()[:, None]
        assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 4 * U * want.abs().max()).all()


class Layer:
    H, Hkv, D, FFN, PAGE, RANK = 8, 2, 64, 640, 16, 16
    DIM = H * D

    def __init__(self, bw, n, shared, seed=1):
        self.gen = gen = torch.Generator(device="cuda").manual_seed(seed)
        H, Hkv, D, dim, ffn = self.H, self.Hkv, self.D, self.DIM, self.FFN

        def normal(*shape, gain=1.0):
            return torch.randn(shape, device="cuda", generator=gen) * gain

        q, kv = H * D, Hkv * D
        self.qkv_n = q + 2 * kv
        self.wqkv = Linear(bw, gen, self.qkv_n, dim, [0, q, q + kv, self.qkv_n])
        self.wo = Linear(bw, gen, dim, dim, [0, dim])
        self.w13 = Linear(bw, gen, 2 * ffn, dim, [0, ffn, 2 * ffn])
        self.w2 = Linear(bw, gen, dim, ffn, [0, dim])
        self.g = [1.0 + 0.2 * normal(k) for k in (dim, dim, dim, ffn, D, D)]
        # adapters of q | k | v, two requests without one
        self.A = normal(5, self.RANK, dim, gain=dim ** -0.5).bfloat16()
        self.B = normal(5, self.qkv_n, self.RANK, gain=0.3).bfloat16()
        self.c = 0.5 + torch.rand(5, device="cuda", generator=gen)
        ids = [(3 * b) % 5 for b in range(n)]
        ids[1] = ids[-1] = -1
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        # pages: the prefix's, then each sequence's own
        P = self.PAGE
        common, own = -(-shared // P), 6
        first = shared // P
        pages = common + n * own
        self.kp = normal(pages, Hkv, P, D).bfloat16()
        self.vp = normal(pages, Hkv, P, D).bfloat16()
        order = torch.randperm(pages, device="cuda", generator=gen).int()
        self.shared_table = order[:common].contiguous()
        self.table = torch.full((n, first + own), -1, dtype=torch.int32, device="cuda")
        self.table[:, first:] = order[common:].view(n, own)
        self.shared = torch.tensor([shared], dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([shared + 3 * b % 11 for b in range(n)],
                                   dtype=torch.int32, device="cuda")
        self.n = n

        def zeros(*shape, kind=torch.bfloat16):
            return torch.zeros(shape, dtype=kind, device="cuda")

        self.h = normal(n, dim)
        self.down = normal(n, dim).bfloat16()
        self.codes = [(zeros(n, k, kind=torch.int8), zeros(n, kind=torch.float32))
                      for k in (dim, dim, dim, ffn)]
        self.qkv, self.o = zeros(n, self.qkv_n), zeros(n, dim)
        self.gu, self.attn = zeros(n, 2 * ffn), zeros(n, H, D)
        size = bw.bw_attn_paged_shared_workspace_bytes(n, H, Hkv, D)
        self.ws = zeros(size, kind=torch.uint8)
        self.lora_ws = zeros(bw.bw_lora_workspace_bytes(n, self.RANK), kind=torch.uint8)

    def step(self, bw, look=lambda name: None):
        """One token of every sequence; look(name) after each call."""
        n, H, Hkv, D = self.n, self.H, self.Hkv, self.D
        g_attn, g_sub, g_ffn, g_down, g_q, g_k = self.g
        self.kv_len.add_(1)
        c = self.codes
        bw.bw_add_rms_norm_quant(self.down, g_attn, h=self.h, q=c[0][0], s=c[0][1])
        look("attn_norm")
        self.wqkv.run(bw, *c[0], self.qkv)
        look("qkv")
        bw.bw_lora_add(self.qkv, *c[0], self.A, self.B, self.ids, scale=self.c,
                       workspace=self.lora_ws)
        look("lora")
        heads = self.qkv.view(n, H + 2 * Hkv, D)
        bw.bw_qk_norm_rope_append(self.qkv, self.kp, self.vp, self.table,
                                  self.kv_len, H, q_gamma=g_q, k_gamma=g_k,
                                  theta=THETA, q_out=heads[:, :H])
        look("append")
        bw.bw_attn_paged_shared(heads[:, :H], self.kp, self.vp, self.table,
                                self.kv_len, self.shared_table, self.shared,
                                out=self.attn, workspace=self.ws)
        look("attn")
        bw.bw_add_rms_norm_quant(self.attn.view(n, -1), g_sub, q=c[1][0], s=c[1][1])
        look("sub_norm")
        self.wo.run(bw, *c[1], self.o)
        look("o")
        bw.bw_add_rms_norm_quant(self.o, g_ffn, h=self.h, q=c[2][0], s=c[2][1])
        look("ffn_norm")
        self.w13.run(bw, *c[2], self.gu)
        look("gu")
        bw.bw_relu2_rms_norm_quant(self.gu, g_down, q=c[3][0], s=c[3][1])
        look("down_norm")
        self.w2.run(bw, *c[3], self.down)
        look("down")

    def state(self):
        return [t.clone() for t in (self.h, self.down, self.kp, self.vp,
                                    self.qkv, self.attn, self.kv_len)]


def check_codes(q, s, v, gamma):
    t = v / (v * v).mean(1, keepdim=True).add(1e-5).sqrt() * gamma.double()
    scale = 127.0 / t.abs().amax(1, keepdim=True).clamp(min=1e-5)
    assert ((s.double()[:, None] - scale).abs() <= 60 * U * scale).all()
    assert ((q.double() - t * scale).abs() <= 0.5 + 127 * 130 * U).all()


@pytest.mark.parametrize("n,shared", [(3, 40), (6, 333), (37, 128), (150, 700)])
def test_every_stage(bw, n, shared):
    m = Layer(bw, n, shared)
    H, Hkv, D, P = m.H, m.Hkv, m.D, m.PAGE
    before = {}

    def look(name):
        if name == "attn_norm":
            v = before["h"] + before["down"].float()
            assert torch.equal(m.h, v)
            check_codes(*m.codes[0], v.double(), m.g[0])
        elif name == "qkv":
            m.wqkv.check(*m.codes[0], m.qkv)
            before["qkv"] = m.qkv.double()
        elif name == "lora":
            x = m.codes[0][0].double() / m.codes[0][1].double()[:, None]
            d = torch.zeros_like(before["qkv"])
            tol = torch.zeros_like(d)
            for b, a in enumerate(m.ids.tolist()):
                if a >= 0:
                    A, B, c = m.A[a].double(), m.B[a].double(), float(m.c[a])
                    u = c * (A @ x[b])
                    mass = abs(c) * (A.abs() @ x[b].abs())
                    d[b] = B @ u
                    tol[b] = B.abs() @ (m.DIM * 2 * U * mass + 2.0 ** -16 * u.abs()) + \
                        2.0 ** -8 * (before["qkv"][b] + d[b]).abs() + \
                        64 * U * (B.abs() @ u.abs() + before["qkv"][b].abs())
            assert ((m.qkv.double() - before["qkv"] - d).abs() <= tol).all()
            before["qkv"] = m.qkv.double().view(n, H + 2 * Hkv, D)
        elif name == "append":
            x = before["qkv"][:, :H + Hkv]
            gam = torch.cat((m.g[4].expand(H, D), m.g[5].expand(Hkv, D))).double()
            y = x / (x * x).mean(2, keepdim=True).add(1e-5).sqrt() * gam
            f = THETA ** (-2.0 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
            ang = (m.kv_len.double()[:, None] - 1) * f
            co, si = ang.cos()[:, None], ang.sin()[:, None]
            e, o = y[..., 0::2], y[..., 1::2]
            z = torch.stack((e * co - o * si, e * si + o * co), -1).flatten(2)
            pair = (e.abs() + o.abs()).repeat_interleave(2, -1)
            tol = 2.0 ** -8 * z.abs() + 2.0 ** -19 * pair
            got = m.qkv.view(n, H + 2 * Hkv, D)[:, :H].double()
            assert ((got - z[:, :H]).abs() <= tol[:, :H]).all()
            for b, p in enumerate((m.kv_len - 1).tolist()):
                page = int(m.table[b, p // P])
                k, v = m.kp[page, :, p % P], m.vp[page, :, p % P]
                assert ((k.double() - z[b, H:]).abs() <= tol[b, H:]).all()
                assert torch.equal(v.double(), before["qkv"][b, H + Hkv:])
        elif name == "attn":
            q = m.qkv.view(n, H + 2 * Hkv, D)[:, :H].double()
            j = torch.arange(int(m.kv_len.max()), device="cuda")
            for b, length in enumerate(m.kv_len.tolist()):
                pages = torch.where(j[:length] < shared,
                                    m.shared_table[(j[:length] // P).clamp(max=len(m.shared_table) - 1)],
                                    m.table[b, j[:length] // P]).long()
                k = m.kp[pages, :, j[:length] % P].transpose(0, 1).double()
                v = m.vp[pages, :, j[:length] % P].transpose(0, 1).double()
                s = q[b].view(Hkv, H // Hkv, D) @ k.transpose(1, 2) / D ** 0.5
                mass = (q[b].abs().view(Hkv, H // Hkv, D) @ k.abs().transpose(1, 2)).amax(2, keepdim=True) / D ** 0.5
                w = torch.softmax(s, 2)
                want = w @ v
                tol = 2 * ((D + 4) * 2 * U * mass + (8 + length) * U) * v.abs().amax(1, keepdim=True) + \
                    2.0 ** -8 * (w @ v.abs()) + 2.0 ** -8 * want.abs()
                assert ((m.attn[b].double().view_as(want) - want).abs() <= tol).all()
        elif name == "sub_norm":
            check_codes(*m.codes[1], m.attn.view(n, -1).double(), m.g[1])
            before["h"] = m.h.clone()
        elif name == "o":
            m.wo.check(*m.codes[1], m.o)
        elif name == "ffn_norm":
            assert torch.equal(m.h, before["h"] + m.o.float())
            check_codes(*m.codes[2], m.h.double(), m.g[2])
        elif name == "gu":
            m.w13.check(*m.codes[2], m.gu)
        elif name == "down_norm":
            g, u = m.gu.double().chunk(2, 1)
            check_codes(*m.codes[3], g.clamp(min=0) ** 2 * u, m.g[3])
        elif name == "down":
            m.w2.check(*m.codes[3], m.down)

    for _ in range(2):
        before["h"], before["down"] = m.h.clone(), m.down.clone()
        m.step(bw, look)
    assert bw.bw_device_error() == 0


@pytest.mark.parametrize("n,shared", [(6, 333), (150, 700)])
def test_steps_from_a_graph(bw, n, shared):
    """Replayed steps give the eager ones' results, bit for bit, with nothing
    waited for in between."""
    eager, graphed = Layer(bw, n, shared), Layer(bw, n, shared)
    for a, b in zip(eager.state(), graphed.state()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(bw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            graphed.step(bw)
        for _ in range(5):
            graph.replay()
    side.synchronize()
    for _ in range(6):
        eager.step(bw)
    torch.cuda.synchronize()
    for a, b in zip(eager.state(), graphed.state()):
        assert torch.equal(a, b)
    assert bool(graphed.h.isfinite().all())
    assert bw.bw_device_error() == 0
