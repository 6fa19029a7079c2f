"""Cases, plain forms and exact values of the operators over a paged key-value
cache: the per-head norm and rotation of queries and keys with the append to
the pages, the attention of one new token per sequence, and the causal
attention of prompts, with an optional sliding window and first tokens that
stay visible.

A case is a dict of plain values; `prepare` makes its inputs from a seed,
`run` makes one pass (the framework's call where `own` is true, elementary
torch operations otherwise), `exact` gives the same outputs in 64 bits.

The cache of all sequences is two pools of pages, bf16 [n_pages][Hkv][page][D];
position j of sequence b lies in row j % page of page page_table[b][j // page].
kv_len[b] counts the positions of sequence b, the new tokens included.
"""
import math

import torch

own = False

THETA = 500000.0
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    """20 query heads over 5 key-value heads of 128 dims are this repository's
    own decoder; the others are generic."""
    return [
        # A single sequence's next token: latency alone.
        _append("append one token", seqs=1, new=1, past=700, heads=20, kv_heads=5, dim=128, page=64, norm=True),
        # The next tokens of a full serving batch, each at its own position.
        _append("append a decode batch", seqs=96, new=1, past=400, heads=20, kv_heads=5, dim=128, page=16, norm=True),
        # The prompts of a ragged batch behind a short past; no norm, as in a decoder without one.
        _append("append prompts", seqs=7, new=1170, past=37, heads=32, kv_heads=8, dim=64, page=32, norm=False),
        # A long prompt in one go.
        _append("append a long prompt", seqs=1, new=16381, past=0, heads=20, kv_heads=5, dim=128, page=128, norm=True),
        # One user, a short chat: latency alone.
        _decode("decode one short", seqs=1, longest=777, heads=20, kv_heads=5, dim=128, page=16, window=0, sinks=0, out="fp32"),
        # One user, a long document: one row of work over a long axis.
        _decode("decode one long", seqs=1, longest=131071, heads=20, kv_heads=5, dim=128, page=64, window=0, sinks=0, out="fp32"),
        # A serving batch of unlike contexts, from a few tokens to 8191.
        _decode("decode a ragged batch", seqs=64, longest=8191, heads=20, kv_heads=5, dim=128, page=64, window=0, sinks=0, out="fp32"),
        # The same with a window and four first tokens, eight query heads to a key head.
        _decode("decode a windowed batch", seqs=120, longest=6000, heads=32, kv_heads=4, dim=64, page=32, window=1000, sinks=4, out="bf16"),
        # A short prompt of odd length: few tiles.
        _prefill("prefill one short", seqs=1, new=509, past=0, heads=20, kv_heads=5, dim=128, page=16, window=0, sinks=0),
        # A long prompt: the tensor cores' case.
        _prefill("prefill one long", seqs=1, new=8192, past=0, heads=20, kv_heads=5, dim=128, page=64, window=0, sinks=0),
        # A small chunk behind a long past: few rows over a long axis.
        _prefill("prefill a chunk", seqs=1, new=200, past=32601, heads=20, kv_heads=5, dim=128, page=128, window=0, sinks=0),
        # Ragged prompts with a window and first tokens, no sharing of key heads beyond two.
        _prefill("prefill a windowed batch", seqs=6, new=2900, past=130, heads=16, kv_heads=8, dim=64, page=32, window=700, sinks=5),
    ]


def _append(name, **kw):
    return {"name": name, "op": "append", **kw}


def _decode(name, **kw):
    return {"name": name, "op": "decode", **kw}


def _prefill(name, **kw):
    return {"name": name, "op": "prefill", **kw}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Heads, pages and masks of the same kinds; lengths and batches over their
    logarithms, no more work than the largest listed case of the operator."""
    heads, kv_heads, dim = rng.choice([(20, 5, 128), (8, 8, 128), (28, 4, 128), (32, 4, 64), (16, 8, 64), (14, 2, 64), (40, 8, 128)])
    page = rng.choice([16, 32, 64, 128])
    shape = {"heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page}
    width = (heads + 2 * kv_heads) * dim
    op = rng.choice(["append", "decode", "prefill"])
    if op == "append":
        if rng.random() < 0.4:
            seqs, new = _log(rng, 1, 200), 1
        else:
            seqs = rng.randint(1, 9)
            new = _log(rng, 2, max(3, 60_000_000 // (width * seqs)))
        new = min(new, 9000)
        return {"op": op, "seqs": seqs, "new": new, "past": rng.randint(0, 500), "norm": rng.random() < 0.7, **shape}
    window = rng.choice([0, 0, rng.randint(1, 300), rng.randint(300, 2000)])
    sinks = rng.choice([0, 1, 4, 7, 40]) if window else 0
    if op == "decode":
        seqs = _log(rng, 1, 128)
        most = 300_000_000 // (kv_heads * dim * seqs)
        longest = _log(rng, 3, max(4, min(100_000, most)))
        return {"op": op, "seqs": seqs, "longest": longest, "window": window, "sinks": sinks, "out": rng.choice(["fp32", "bf16"]), **shape}
    seqs = rng.randint(1, 6)
    most = math.sqrt(500_000_000 / (heads * seqs))
    new = _log(rng, 3, int(min(5000, most)))
    past = rng.choice([0, rng.randint(1, 300), _log(rng, 300, max(301, min(12000, int(300_000_000 / (heads * seqs * new)))))])
    return {"op": op, "seqs": seqs, "new": new, "past": past, "window": window, "sinks": sinks, **shape}


def _lengths(case):
    """(new, kv_len) of each sequence: host integers that go by the case alone,
    so that every seed has the same work.  The first sequence has the most; a
    batch has short ones and one of a single token among them."""
    n = case["seqs"]
    share = [1.0] + [0.6180339887 * i % 1.0 for i in range(1, n)]
    if case["op"] == "decode":
        kv = [max(1, int(case["longest"] * s)) for s in share]
        return [1] * n, kv
    if case["new"] == 1:
        new = [1] * n
    else:
        new = [max(1, int(case["new"] * (0.4 + 0.6 * s))) for s in share]
        new[0] = case["new"]
        if n > 2:
            new[2] = 1
    past = [int(case["past"] * s) for s in share]
    return new, [a + b for a, b in zip(new, past)]


def _visible(case, p):
    """How many positions a token at position p sees."""
    if not case["window"] or p < case["window"]:
        return p + 1
    return case["window"] + min(case["sinks"], p + 1 - case["window"])


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    """Pools of pages in a shuffled order, lengths, a page table, and the new
    tokens: a q|k|v projection's rows for the append, rotated queries for the
    attention (scaled so that the softmax weights are uneven, as in a trained
    model).  Outputs and workspaces that a program keeps are made here too."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    n, heads, kv_heads, dim, page = case["seqs"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    new, kv = _lengths(case)
    pages = [-(-k // page) for k in kv]
    most, total = max(pages), sum(pages)
    n_pages = total + 3
    order = torch.randperm(n_pages, device=dev, generator=gen)[:total].to(torch.int32)
    first = torch.tensor([sum(pages[:b]) for b in range(n)], device=dev)
    count = torch.tensor(pages, device=dev)
    at = torch.arange(most, device=dev)[None, :]
    table = torch.where(at < count[:, None], order[(first[:, None] + at).clamp_max(total - 1)], torch.full((), -1, dtype=torch.int32, device=dev))
    tokens = sum(new)
    start = torch.tensor([sum(new[:b]) for b in range(n + 1)], dtype=torch.int32, device=dev)

    def normal(*shape, gain=1.0):
        return (torch.randn(shape, device=dev, generator=gen) * gain).to(torch.bfloat16)

    state = {
        "case": dict(case), "tokens": tokens,
        "k_pages": normal(n_pages, kv_heads, page, dim), "v_pages": normal(n_pages, kv_heads, page, dim),
        "page_table": table.contiguous(), "kv_len": torch.tensor(kv, dtype=torch.int32, device=dev),
        "q_start": start, "most_new": max(new), "window": case.get("window", 0), "sinks": case.get("sinks", 0),
    }
    if case["op"] == "append":
        state["qkv"] = normal(tokens, (heads + 2 * kv_heads) * dim, gain=1.5)
        state["q_gamma"] = 1.0 + 0.2 * torch.randn(dim, device=dev, generator=gen) if case["norm"] else None
        state["k_gamma"] = 1.0 + 0.2 * torch.randn(dim, device=dev, generator=gen) if case["norm"] else None
        state["q_out"] = torch.zeros((tokens, heads, dim), dtype=torch.bfloat16, device=dev)
    else:
        state["q"] = normal(tokens, heads, dim, gain=2.0)
        kind = torch.float32 if case.get("out") == "fp32" else torch.bfloat16
        state["out"] = torch.zeros((tokens, heads, dim), dtype=kind, device=dev)
        # the most that either attention asks of a caller for these sizes
        state["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=dev)
    return state


#: Bytes of scratch that a program which serves these cases keeps, zeroed once.
WORKSPACE = 64 << 20


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "prefill": _own_prefill}[op](state)
    return {"append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[op](state)


def _own_append(s):
    import bit_gemv_bitlinear_gb300 as bw
    bw.bw_qk_norm_rope_append(s["qkv"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], s["case"]["heads"],
                              q_start=None if s["case"]["new"] == 1 else s["q_start"], q_gamma=s["q_gamma"], k_gamma=s["k_gamma"],
                              eps=EPS, theta=THETA, q_out=s["q_out"])
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _own_decode(s):
    import bit_gemv_bitlinear_gb300 as bw
    return bw.bw_attn_paged_decode(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"],
                                   window=s["window"], sinks=s["sinks"], out=s["out"], workspace=s["workspace"])


def _own_prefill(s):
    import bit_gemv_bitlinear_gb300 as bw
    return bw.bw_attn_paged_prefill(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], s["q_start"],
                                    window=s["window"], sinks=s["sinks"], out=s["out"], workspace=s["workspace"])


def _token_places(s):
    """Sequence and position of every token."""
    t = torch.arange(s["tokens"], device=s["q_start"].device)
    start = s["q_start"].long()
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    pos = s["kv_len"].long()[b] - start[b + 1] + t
    return b, pos


def _plain_append(s):
    heads, kv_heads, dim, page = (s["case"][k] for k in ("heads", "kv_heads", "dim", "page"))
    b, pos = _token_places(s)
    x = s["qkv"].float().view(s["tokens"], heads + 2 * kv_heads, dim)
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], s["qkv"].view(s["tokens"], heads + 2 * kv_heads, dim)[:, heads + kv_heads:]
    if s["q_gamma"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_gamma"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_gamma"]
    # the angles of far positions in 64 bits
    f = THETA ** (-2.0 * torch.arange(dim // 2, device=x.device, dtype=torch.float64) / dim)
    angle = pos.double()[:, None] * f
    c, n = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turn(y):
        e, o = y[..., 0::2], y[..., 1::2]
        return torch.stack((e * c - o * n, e * n + o * c), -1).flatten(-2).to(torch.bfloat16)

    s["q_out"].copy_(turn(q))
    where = s["page_table"].long()[b, pos // page]
    s["k_pages"][where, :, pos % page] = turn(k)
    s["v_pages"][where, :, pos % page] = v
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _rows(pool, table):
    """The keys or values of every sequence, in the order of their positions:
    [B][Hkv][positions][D] in 32 bits (rows past a sequence's end hold others')."""
    x = pool[table.long().clamp_min(0)]  # [B][pages][Hkv][page][D]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3).float()


def _plain_attention(s, q, pos, valid):
    """q [B][T][H][D] at positions pos [B][T]: [B][T][H][D] in 32 bits."""
    n, t, heads, dim = q.shape
    k, v = _rows(s["k_pages"], s["page_table"]), _rows(s["v_pages"], s["page_table"])
    kv_heads, length = k.shape[1], k.shape[2]
    j = torch.arange(length, device=q.device)
    seen = (j <= pos[..., None]) & valid[..., None]
    if s["window"]:
        seen &= (j > pos[..., None] - s["window"]) | (j < s["sinks"])
    v = v * (j < s["kv_len"][:, None])[:, None, :, None]
    g = heads // kv_heads
    q = q.float().view(n, t, kv_heads, g, dim).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B][Hkv][G T][D]
    w = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(dim))
    del k, q
    w = w.view(n, kv_heads, g, t, length).masked_fill_(~seen[:, None, None], float("-inf"))
    m = w.amax(-1, keepdim=True)
    w = w.sub_(m.masked_fill(m == float("-inf"), 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    out = (w.flatten(2, 3) @ v).view(n, kv_heads, g, t, dim) / total.clamp_min(1e-30)
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3)


def _plain_decode(s):
    pos = s["kv_len"].long()[:, None] - 1
    out = _plain_attention(s, s["q"][:, None], pos, pos >= 0)
    s["out"].copy_(out[:, 0])
    return s["out"]


def _plain_prefill(s):
    n, most = s["case"]["seqs"], s["most_new"]
    start = s["q_start"].long()
    i = torch.arange(most, device=start.device)[None, :]
    count = (start[1:] - start[:-1])[:, None]
    rows = (start[:-1, None] + i).clamp_max(s["tokens"] - 1)
    out = _plain_attention(s, s["q"][rows], s["kv_len"].long()[:, None] - count + i, i < count)
    b, _ = _token_places(s)
    t = torch.arange(s["tokens"], device=start.device)
    s["out"].copy_(out[b, t - start[b]])
    return s["out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    new, kv = _lengths(case)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    tokens = sum(new)
    table = 4 * sum(-(-k // case["page"]) for k in kv) + 8 * len(kv)
    if case["op"] == "append":
        values = tokens * (heads + 2 * kv_heads) * dim
        flops = tokens * (heads + kv_heads) * dim * (10 if case["norm"] else 6)
        return {"bytes": 4 * values + 8 * dim + 8 * len(kv), "flops": flops}
    pairs, rows = 0, 0
    for a, k in zip(new, kv):
        w = case["window"]
        low = k - a  # the first new token's position
        if w:
            pairs += sum(_visible(case, p) for p in range(low, k))
            first = max(0, low + 1 - w)
            rows += k - first + min(case["sinks"], first)
        else:
            pairs += a * (low + 1) + a * (a - 1) // 2
            rows += k
    out = 4 if case.get("out") == "fp32" else 2
    return {"bytes": 4 * rows * kv_heads * dim + tokens * heads * dim * (2 + out) + table, "flops": 4 * pairs * heads * dim}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """Sequence by sequence from the operators' definition; the same inputs as
    `run`, none of its code."""
    s = prepare(case, seed)
    new, kv = _lengths(case)
    heads, kv_heads, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    g = heads // kv_heads
    table = s["page_table"].cpu().tolist()
    if case["op"] == "append":
        k_pool, v_pool = s["k_pages"].double(), s["v_pages"].double()
        q_all, t = [], 0
        i = torch.arange(dim // 2, dtype=torch.float64, device=k_pool.device)
        turn_of = torch.exp(i * (-2.0 / dim * math.log(THETA)))
        for b, (a, length) in enumerate(zip(new, kv)):
            x = s["qkv"][t:t + a].double()
            t += a
            q = x[:, :heads * dim].reshape(a, heads, dim)
            k = x[:, heads * dim:(heads + kv_heads) * dim].reshape(a, kv_heads, dim)
            v = x[:, (heads + kv_heads) * dim:].reshape(a, kv_heads, dim)
            if case["norm"]:
                q = q / ((q * q).sum(2, keepdim=True) / dim + EPS).sqrt() * s["q_gamma"].double()
                k = k / ((k * k).sum(2, keepdim=True) / dim + EPS).sqrt() * s["k_gamma"].double()
            p = torch.arange(length - a, length, device=x.device)
            z = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), p.double()[:, None, None] * turn_of)
            q = torch.view_as_real(torch.view_as_complex(q.reshape(a, heads, dim // 2, 2).contiguous()) * z).reshape(a, heads, dim)
            k = torch.view_as_real(torch.view_as_complex(k.reshape(a, kv_heads, dim // 2, 2).contiguous()) * z).reshape(a, kv_heads, dim)
            q_all.append(q)
            for first in range((length - a) // page, -(-length // page)):  # page by page
                lo, hi = max(first * page, length - a), min((first + 1) * page, length)
                to = slice(lo - first * page, hi - first * page)
                k_pool[table[b][first], :, to] = k[lo - (length - a):hi - (length - a)].transpose(0, 1)
                v_pool[table[b][first], :, to] = v[lo - (length - a):hi - (length - a)].transpose(0, 1)
        return {"q": torch.cat(q_all), "k_pages": k_pool, "v_pages": v_pool}
    out = torch.zeros(s["tokens"], heads, dim, dtype=torch.float64, device=s["q"].device)
    t = 0
    for b, (a, length) in enumerate(zip(new, kv)):
        ids = torch.tensor(table[b][:-(-length // page)], device=out.device)
        k_rows = s["k_pages"][ids].transpose(1, 2).reshape(-1, kv_heads, dim)[:length]
        v_rows = s["v_pages"][ids].transpose(1, 2).reshape(-1, kv_heads, dim)[:length]
        for first in range(0, a, 1024):  # 1024 tokens at a time
            last = min(a, first + 1024)
            p = torch.arange(length - a + first, length - a + last, device=out.device)
            end = length - a + last
            j = torch.arange(end, device=out.device)
            hidden = j[None, :] > p[:, None]
            if case["window"]:
                hidden |= (p[:, None] - j[None, :] >= case["window"]) & (j[None, :] >= case["sinks"])
            for h in range(heads):
                score = s["q"][t + first:t + last, h].double() @ k_rows[:end, h // g].double().T / math.sqrt(dim)
                weight = torch.softmax(score.masked_fill(hidden, float("-inf")), 1)
                out[t + first:t + last, h] = weight @ v_rows[:end, h // g].double()
        t += a
    return out
