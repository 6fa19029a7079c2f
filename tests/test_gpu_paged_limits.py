"""The calls over a paged key-value cache (GB300) at the limits that bw.h names:
the longest sequences, the most tokens, heads and sequences, and calls from
two host threads at once.  Tolerances as in test_gpu_paged.py and, for queries
of zeros over values that are small integers, test_gpu_paged_long.py.
"""
import threading

import numpy as np
import pytest

from test_gpu_paged import (U, Cache, as_bf16, attend, bw, f64,  # noqa: F401
                            norm_rope, seen)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LONGEST = 1 << 24


def integers(*shape):
    g = torch.Generator(device="cuda").manual_seed(201)
    return torch.randint(-8, 9, shape, generator=g, device="cuda",
                         dtype=torch.int8).bfloat16()


@pytest.mark.parametrize("H,Hkv,D,page,lens,new", [
    (4, 1, 128, 256, [LONGEST, LONGEST - 77], [5, 3]),          # in parts
    (64, 64, 64, 256, [LONGEST - 5, LONGEST, 9], [1, 2, 3]),    # items of one
    (16, 1, 64, 16, [LONGEST], [2]),
])
def test_longest_sequences(bw, H, Hkv, D, page, lens, new):
    """Sequences of 2^24 positions whose table names the same few pages again
    and again.  A query of zeros sees the mean of the values; their partial
    sums are integers below 2^24 (8 * 2^24 only in magnitude of all parts,
    whose signs are random: 5 sigma of the sum are below 2^17)."""
    pages = 16
    vp = integers(pages, Hkv, page, D)
    kp = torch.randn((pages, Hkv, page, D), device="cuda").bfloat16()
    width = LONGEST // page
    table = (torch.arange(width, device="cuda", dtype=torch.int32) % pages)
    table = torch.stack([table.roll(b) for b in range(len(lens))]).contiguous()
    len_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    T = sum(new)
    st = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32,
                      device="cuda")
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    out = bw.bw_attn_paged_prefill(q, kp, vp, table, len_d, st)
    one = bw.bw_attn_paged_decode(q[:len(lens)], kp, vp, table, len_d)
    assert bw.bw_device_error() == 0

    def mean(x, b, p):  # of positions 0 .. p of sequence b
        total = torch.zeros((Hkv, D), dtype=torch.float64, device="cuda")
        full, rest = divmod(p + 1, page)
        for i in range(pages):
            count = full // pages + (i < full % pages)
            total += count * x[int(table[b, i])].double().sum(1)
        if rest:
            total += x[int(table[b, full])][:, :rest].double().sum(1)
        return (total / (p + 1)).repeat_interleave(H // Hkv, 0)

    t = 0
    for b, (n, a) in enumerate(zip(lens, new)):
        for i in range(a):
            ref, size = mean(vp, b, n - a + i), mean(vp.abs(), b, n - a + i)
            tol = 8 * U * size
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
            err = (out[t].double() - ref).abs()
            assert (err <= tol).all(), (b, i, float((err - tol).max()))
            t += 1
        err = (one[b].double() - ref).abs()
        assert (err <= 8 * U * size).all(), (b, float(err.max()))


def test_most_tokens(bw):
    """2^20 tokens of one sequence: appended, then seen."""
    T, H, Hkv, D, page = 1 << 20, 1, 1, 64, 256
    v = integers(T, D)
    qkv = torch.zeros((T, 3 * D), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(202)
    qkv[:, D:2 * D] = torch.randn((T, D), generator=g, device="cuda").bfloat16()
    qkv[:, 2 * D:] = v
    kp = torch.zeros((T // page, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.randperm(T // page, generator=g, device="cuda").int()[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    st = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    q = bw.bw_qk_norm_rope_append(qkv, kp, vp, table, lens, H, q_start=st)
    assert bw.bw_device_error() == 0
    ids = table[0].long()
    assert torch.equal(vp[ids].view(T, D), v)
    k = kp[ids].view(T, D)
    for t in (0, 1, 255, 256, 77777, T - 1):
        z, pair = norm_rope(f64(qkv[t, D:2 * D]), t, None, 0.0, 500000.0)
        assert (np.abs(f64(k[t]) - z) <= 2.0 ** -8 * np.abs(z) +
                2.0 ** -19 * pair).all(), t
    out = bw.bw_attn_paged_prefill(q, kp, vp, table, lens, st)
    assert bw.bw_device_error() == 0
    n = torch.arange(1, T + 1, device="cuda")[:, None]
    ref = v.double().cumsum(0) / n
    tol = 8 * U * v.double().abs().cumsum(0) / n
    tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (out[:, 0].double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("D", [64, 128])
def test_most_heads(bw, D):
    """16 query heads to each of 64 key heads."""
    H, Hkv, page = 1024, 64, 16
    lens, new = [150, 33, 0], [20, 33, 0]
    c = Cache(203, lens, Hkv, D, page)
    rng = np.random.default_rng(204)
    start = np.concatenate([[0], np.cumsum(new)])
    q = as_bf16(rng.standard_normal((int(start[-1]), H, D))).cuda()
    out = bw.bw_attn_paged_prefill(q, *c.args,
                                   torch.from_numpy(start.astype(np.int32)).cuda())
    one = bw.bw_attn_paged_decode(q[:3], *c.args)
    assert bw.bw_device_error() == 0
    for b in range(2):
        k, v = f64(c.k[b]), f64(c.v[b])
        for i in (0, new[b] - 1):
            p = lens[b] - new[b] + i
            ref, tol = attend(f64(q[start[b] + i]), k, v, D ** -0.5,
                              np.arange(p + 1), 2.0 ** -8)
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            assert (np.abs(f64(out[start[b] + i]) - ref) <= tol).all()
        ref, tol = attend(f64(q[b]), k, v, D ** -0.5, np.arange(lens[b]))
        assert (np.abs(f64(one[b]) - ref) <= tol).all()
    assert (one[2] == 0).all()


@pytest.mark.parametrize("H,Hkv,D", [(4, 2, 64), (2, 2, 128)])
def test_most_sequences(bw, H, Hkv, D):
    """4096 sequences, many of them empty: append, prefill, decode."""
    n, page, window, sinks = 4096, 16, 20, 2
    new = [(5 * i) % 7 % 4 for i in range(n)]
    lens = [a + (3 * i) % 29 if a or i % 3 else 0 for i, a in enumerate(new)]
    c = Cache(205, lens, Hkv, D, page)
    rng = np.random.default_rng(206)
    start = np.concatenate([[0], np.cumsum(new)])
    T = int(start[-1])
    st = torch.from_numpy(start.astype(np.int32)).cuda()
    qkv = as_bf16(rng.standard_normal((T, (H + 2 * Hkv) * D))).cuda()
    q = bw.bw_qk_norm_rope_append(qkv, *c.args, H, q_start=st)
    out = bw.bw_attn_paged_prefill(q, *c.args, st, window=window, sinks=sinks)
    q1 = as_bf16(rng.standard_normal((n, H, D))).cuda()
    one = bw.bw_attn_paged_decode(q1, *c.args, window=window, sinks=sinks)
    assert bw.bw_device_error() == 0
    qf, x = f64(q), f64(qkv).reshape(T, H + 2 * Hkv, D)
    kp, vp = f64(c.kp), f64(c.vp)
    outf, onef, q1f = f64(out), f64(one), f64(q1)
    for b in range(0, n, 5):
        ids = c.table[b, :-(-lens[b] // page)]
        k = kp[ids].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:lens[b]]
        v = vp[ids].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:lens[b]]
        for i in range(new[b]):
            t, p = int(start[b]) + i, lens[b] - new[b] + i
            for got, raw in ((qf[t], x[t, :H]), (k[p], x[t, H:H + Hkv])):
                z, pair = norm_rope(raw, p, None, 0.0, 500000.0)
                assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) +
                        2.0 ** -19 * pair).all(), (b, i)
            assert (v[p] == x[t, H + Hkv:]).all()
            ref, tol = attend(qf[t], k, v, D ** -0.5, seen(p, window, sinks),
                              2.0 ** -8)
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            assert (np.abs(outf[t] - ref) <= tol).all(), (b, i)
        ref, tol = attend(q1f[b], k, v, D ** -0.5, seen(lens[b] - 1, window, sinks))
        assert (np.abs(onef[b] - ref) <= tol).all(), b


@pytest.mark.parametrize("theta", [1.0, 10000.0, 2.9e38])
@pytest.mark.parametrize("which", ["q", "k", "both", "none"])
def test_gains_of_one_kind_and_any_theta(bw, which, theta):
    H, Hkv, D, page, n = 6, 3, 128, 32, 40
    c = Cache(207, [n], Hkv, D, page, fill=False)
    rng = np.random.default_rng(208)
    qkv = as_bf16(rng.standard_normal((n, (H + 2 * Hkv) * D))).cuda()
    gamma = rng.uniform(-1.5, 1.5, (2, D)).astype(np.float32)
    gains = [torch.from_numpy(g).cuda() if which in (w, "both") else None
             for g, w in zip(gamma, "qk")]
    st = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    q = bw.bw_qk_norm_rope_append(qkv, *c.args, H, q_start=st, q_gamma=gains[0],
                                  k_gamma=gains[1], theta=theta)
    assert bw.bw_device_error() == 0
    x = f64(qkv).reshape(n, H + 2 * Hkv, D)
    t32 = float(np.float32(theta))
    for p in range(n):
        k = f64(c.kp[int(c.table[0, p // page]), :, p % page])
        for got, raw, g, on in ((f64(q[p]), x[p, :H], gamma[0], gains[0]),
                                (k, x[p, H:H + Hkv], gamma[1], gains[1])):
            z, pair = norm_rope(raw, p, None if on is None else g.astype(float),
                                1e-5, t32)
            assert (np.abs(got - z) <= 2.0 ** -8 * np.abs(z) +
                    2.0 ** -19 * pair + 1e-30).all(), p


def test_calls_from_two_host_threads(bw):
    """Unlike thetas, shapes and streams, a workspace each: as one by one."""
    jobs = []
    for i, (H, Hkv, D) in enumerate([(8, 2, 128), (9, 3, 64)]):
        lens, new = [900 + i, 70], [300, 60]
        c = Cache(209 + i, lens, Hkv, D, 32)
        qkv = as_bf16(np.random.default_rng(i).standard_normal(
            (360, (H + 2 * Hkv) * D))).cuda()
        st = torch.tensor([0, 300, 360], dtype=torch.int32, device="cuda")
        jobs.append((c, qkv, st, H, [1e4, 5e5][i]))

    def serve(job, stream):
        c, qkv, st, H, theta = job
        q = bw.bw_qk_norm_rope_append(qkv, *c.args, H, q_start=st, theta=theta,
                                      stream=stream)
        return (q, bw.bw_attn_paged_prefill(q, *c.args, st, stream=stream),
                bw.bw_attn_paged_decode(q[:2], *c.args, stream=stream))

    want = [serve(job, None) for job in jobs]
    torch.cuda.synchronize()
    results, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(40):
                results[i].append(serve(jobs[i], stream))
            stream.synchronize()
        except Exception as e:  # shown below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert bw.bw_device_error() == 0
    for i in range(2):
        for r in results[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)
