"""Cases, plain forms and exact values of the operators that stand between the
projections of a served decoder layer: the residual's addition with the
root-mean-square norm and its 8-bit output, the gated form of it that feeds the
down projection, the low-rank adapters of many requests beside a shared
projection, and the attention of a batch whose sequences share a long prefix.

A case is a dict of plain values; `prepare` makes its inputs from a seed,
`run` makes one pass (the framework's call where `own` is true, elementary
torch operations otherwise), `exact` gives the same outputs in 64 bits.

What an operator holds in 8 bits is returned as the values it stands for,
codes / scale, in bf16.
"""
import math

import torch

own = False

EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    """Widths of 2560, 6912, 3840 and 13824 and 20 query heads over 5 key-value
    heads of 128 dims are this repository's own decoder; the others are
    generic."""
    return [
        # One user's next token, in front of the fused q|k|v projection: latency alone.
        _norm("norm one token", rows=1, width=2560, kind="bf16", residual=True),
        # The attention's output of a serving batch in front of its projection: no residual there.
        _norm("norm a decode batch", rows=96, width=2560, kind="fp32", residual=False),
        # A prompt's tokens, the most rows that one projection takes.
        _norm("norm a prompt", rows=4096, width=2560, kind="bf16", residual=True),
        # The gated products of a serving batch in front of the down projection.
        _gate("gate a decode batch", rows=64, width=6912),
        # The same for a prompt of odd length.
        _gate("gate a prompt", rows=2039, width=6912),
        # One user's token through its own adapter: latency alone.
        _lora("adapt one token", rows=1, n=2560, k=2560, rank=16, adapters=8),
        # A serving batch, nearly every request with another adapter, some without one.
        _lora("adapt a decode batch", rows=61, n=3840, k=2560, rank=16, adapters=48),
        # Prompts of a few requests over the widest projection, at a high rank.
        _lora("adapt prompts", rows=2011, n=13824, k=2560, rank=64, adapters=5),
        # A few chats behind a short system prompt: latency alone.
        _shared("share a short prefix", seqs=8, shared=1027, new=180, heads=20, kv_heads=5, dim=128, page=16, padded=False),
        # A serving batch behind a long system prompt, which ends inside a page.
        _shared("share a prompt", seqs=64, shared=8209, new=500, heads=20, kv_heads=5, dim=128, page=64, padded=False),
        # Many questions about one long document.
        _shared("share a document", seqs=48, shared=100001, new=300, heads=20, kv_heads=5, dim=128, page=128, padded=False),
        # A large batch of short answers, eight query heads to a key head, in a batch with empty places.
        _shared("share by heads of 64", seqs=230, shared=2600, new=90, heads=32, kv_heads=4, dim=64, page=32, padded=True),
    ]


def _norm(name, **kw):
    return {"name": name, "op": "norm", **kw}


def _gate(name, **kw):
    return {"name": name, "op": "gate", **kw}


def _lora(name, **kw):
    return {"name": name, "op": "lora", **kw}


def _shared(name, **kw):
    return {"name": name, "op": "shared", **kw}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """The same kinds; rows, widths, batches and lengths over their logarithms,
    no more work than the largest listed case of the operator."""
    op = rng.choice(["norm", "gate", "lora", "shared", "shared"])
    if op in ("norm", "gate"):
        width = rng.choice([64, 1021, 2048, 2560, 2564, 4096, 5120, 6912, 8192, 13824, _log(rng, 33, 16000)])
        rows = _log(rng, 1, min(4096, 10_000_000 // width))
        if op == "gate":
            return {"op": op, "rows": rows, "width": width}
        return {"op": op, "rows": rows, "width": width, "kind": rng.choice(["bf16", "fp32"]), "residual": rng.random() < 0.6}
    if op == "lora":
        n, k = rng.choice([(2560, 2560), (3840, 2560), (13824, 2560), (2560, 6912), (640, 1024), (1021, 516), (4096, 4096)])
        rank, adapters = rng.choice([8, 16, 24, 32, 64, 128]), _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, min(2011, 27_000_000 // n, 1_500_000_000 // (k * rank))))
        return {"op": op, "rows": rows, "n": n, "k": k, "rank": rank, "adapters": adapters}
    heads, kv_heads, dim = rng.choice([(20, 5, 128), (8, 8, 128), (28, 4, 128), (32, 4, 64), (16, 8, 64), (14, 2, 64), (40, 8, 128), (16, 1, 64)])
    seqs = _log(rng, 1, 256)
    shared = _log(rng, 1, max(2, min(100_000, 96_000_000 // (heads * seqs))))
    new = _log(rng, 1, max(2, min(2000, 150_000_000 // (kv_heads * dim * seqs))))
    return {"op": op, "seqs": seqs, "shared": shared, "new": new, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": rng.choice([16, 32, 64, 128]), "padded": seqs > 3 and rng.random() < 0.4}


def _lengths(case):
    """The length of each sequence, by the case alone, so that every seed has
    the same work.  In a padded batch some places are empty and one sequence
    has not reached the end of the prefix."""
    n = case["seqs"]
    kv = [case["shared"] + max(1, int(case["new"] * (1.0 if b == 0 else 0.6180339887 * b % 1.0))) for b in range(n)]
    if case["padded"]:
        kv[0] = kv[n // 2] = 0
        kv[2] = (case["shared"] + 1) // 2
    return kv


def _adapters_of(case):
    """The adapter of each row: decode batches mix them row by row and leave
    every eighth row without one, prompts lie one after the other."""
    m, n = case["rows"], case["adapters"]
    if m == 1:
        return [n // 2]
    if m <= 256:
        return [-1 if i % 8 == 7 else (i * 7) % n for i in range(m)]
    return [i * n // m for i in range(m)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    """Inputs in the layouts that the neighbouring calls write, with the
    outputs and the workspace that a program keeps."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, gain=1.0, kind=torch.float32):
        return (torch.randn(shape, device=dev, generator=gen) * gain).to(kind)

    state = {"case": dict(case)}
    op = case["op"]
    if op in ("norm", "gate"):
        m, k = case["rows"], case["width"]
        # channels of unlike size, as a residual stream has them
        gains = torch.exp(0.7 * normal(k))
        if op == "norm":
            kind = torch.bfloat16 if case["kind"] == "bf16" else torch.float32
            state["x"] = (normal(m, k) * gains).to(kind)
            state["h"] = normal(m, k, gain=3.0) * gains if case["residual"] else None
            state["h_out"] = torch.zeros((m, k), device=dev) if case["residual"] else None
        else:
            state["gu"] = torch.cat((normal(m, k), normal(m, k) * gains), 1).to(torch.bfloat16)
        state["gamma"] = 1.0 + 0.2 * normal(k)
        state["q"] = torch.zeros((m, k), dtype=torch.int8, device=dev)
        state["s"] = torch.zeros((m,), device=dev)
        state["values"] = torch.zeros((m, k), dtype=torch.bfloat16, device=dev)
    elif op == "lora":
        m, n, k, rank, count = (case[x] for x in ("rows", "n", "k", "rank", "adapters"))
        x = normal(m, k)
        state["s"] = 127.0 / x.abs().amax(1)
        state["x"] = torch.round(x * state["s"][:, None]).to(torch.int8)
        state["y"] = normal(m, n, kind=torch.bfloat16)
        state["out"] = torch.zeros((m, n), dtype=torch.bfloat16, device=dev)
        state["A"] = normal(count, rank, k, gain=k ** -0.5, kind=torch.bfloat16)
        state["B"] = normal(count, n, rank, gain=rank ** -0.5, kind=torch.bfloat16)
        state["scale"] = 0.5 + 0.3 * torch.rand(count, device=dev, generator=gen)
        state["adapter"] = torch.tensor(_adapters_of(case), dtype=torch.int32, device=dev)
        state["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=dev)
    else:
        n, page, shared = case["seqs"], case["page"], case["shared"]
        heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
        kv = _lengths(case)
        first = shared // page  # a page that the prefix fills in part is each sequence's own
        mine = [max(0, -(-x // page) - first) for x in kv]
        common = -(-shared // page)
        n_pages = common + sum(mine) + 3
        order = torch.randperm(n_pages, device=dev, generator=gen).to(torch.int32)
        begin = torch.tensor([common + sum(mine[:b]) for b in range(n)], device=dev)
        count = torch.tensor(mine, device=dev)
        width = first + max(mine)
        at = torch.arange(width, device=dev)[None, :] - first
        table = torch.where(at < 0, order[torch.arange(width, device=dev).clamp_max(common - 1)][None, :],
                            order[(begin[:, None] + at.clamp_min(0)).clamp_max(n_pages - 1)])
        state["page_table"] = torch.where(at < count[:, None], table, torch.full_like(table, -1)).contiguous()
        state["shared_table"] = order[:common].contiguous()
        state["shared_len"] = torch.tensor([shared], dtype=torch.int32, device=dev)
        state["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=dev)
        state["k_pages"] = normal(n_pages, kv_heads, page, dim, kind=torch.bfloat16)
        state["v_pages"] = normal(n_pages, kv_heads, page, dim, kind=torch.bfloat16)
        # uneven softmax weights, as in a trained model
        state["q"] = normal(n, heads, dim, gain=2.0, kind=torch.bfloat16)
        state["out"] = torch.zeros((n, heads, dim), dtype=torch.bfloat16, device=dev)
        state["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=dev)
    return state


#: Bytes of scratch that a program which serves these cases keeps, zeroed once.
WORKSPACE = 96 << 20


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "gate": _own_gate, "lora": _own_lora, "shared": _own_shared}[op](state)
    return {"norm": _plain_norm, "gate": _plain_gate, "lora": _plain_lora, "shared": _plain_shared}[op](state)


def _own_norm(s):
    import bit_gemv_bitlinear_gb300 as bw
    bw.bw_add_rms_norm_quant(s["x"], s["gamma"], h=s["h"], eps=EPS, h_out=s["h_out"], q=s["q"], s=s["s"])
    return {"h": s["h_out"], "s": s["s"], "values": torch.div(s["q"], s["s"][:, None], out=s["values"])}


def _own_gate(s):
    import bit_gemv_bitlinear_gb300 as bw
    bw.bw_relu2_rms_norm_quant(s["gu"], s["gamma"], eps=EPS, q=s["q"], s=s["s"])
    return {"s": s["s"], "values": torch.div(s["q"], s["s"][:, None], out=s["values"])}


def _own_lora(s):
    import bit_gemv_bitlinear_gb300 as bw
    return bw.bw_lora_add(s["y"], s["x"], s["s"], s["A"], s["B"], s["adapter"], scale=s["scale"], out=s["out"], workspace=s["workspace"])


def _own_shared(s):
    import bit_gemv_bitlinear_gb300 as bw
    return bw.bw_attn_paged_shared(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], s["shared_table"], s["shared_len"],
                                   out=s["out"], workspace=s["workspace"])


def _plain_quant(s, t):
    """Codes of 8 bits with a scale for each row of t, and what they stand for."""
    t = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["gamma"]
    torch.div(127.0, t.abs().amax(1).clamp_min(1e-5), out=s["s"])
    s["q"].copy_(torch.round(t * s["s"][:, None]))
    return {"s": s["s"], "values": torch.div(s["q"], s["s"][:, None], out=s["values"])}


def _plain_norm(s):
    if s["h"] is None:
        return {"h": None, **_plain_quant(s, s["x"].float())}
    return {"h": s["h_out"], **_plain_quant(s, torch.add(s["h"], s["x"], out=s["h_out"]))}


def _plain_gate(s):
    g, u = s["gu"].float().chunk(2, 1)
    return _plain_quant(s, torch.relu(g).square() * u)


def _plain_lora(s):
    """Every row through every adapter at once, with zeros in the place of the
    adapters that are not the row's: two products over all of them."""
    count, rank, k = s["A"].shape
    u = (s["x"].float() / s["s"][:, None]) @ s["A"].float().view(count * rank, k).T
    mine = s["adapter"][:, None] == torch.arange(count, device=u.device)
    u = u.view(-1, count, rank) * (mine * s["scale"])[:, :, None]
    delta = u.flatten(1) @ s["B"].float().permute(0, 2, 1).flatten(0, 1)
    return torch.add(s["y"], delta, out=s["out"])


def _plain_shared(s):
    """The prefix's keys and values are taken once for the whole batch, the own
    ones by sequence; one softmax over both."""
    n, heads, dim = s["q"].shape
    kv_heads, page = s["k_pages"].shape[1:3]
    g, shared, first = heads // kv_heads, s["case"]["shared"], s["case"]["shared"] // page
    q = s["q"].float().view(n, kv_heads, g, dim) * (1.0 / math.sqrt(dim))

    def prefix(pool):
        return pool[s["shared_table"].long()].transpose(0, 1).flatten(1, 2)[:, :shared].float()  # [Hkv][shared][D]

    def rest(pool):
        return pool[s["page_table"][:, first:].long().clamp_min(0)].transpose(1, 2).flatten(2, 3).float()  # [n][Hkv][own][D]

    a = (q.transpose(0, 1).flatten(1, 2) @ prefix(s["k_pages"]).transpose(1, 2)).view(kv_heads, n, g, shared)
    hidden = torch.arange(shared, device=q.device) >= s["kv_len"][:, None]
    a = a.masked_fill_(hidden[None, :, None], float("-inf"))
    k = rest(s["k_pages"])
    j = first * page + torch.arange(k.shape[2], device=q.device)
    seen = (j >= shared) & (j < s["kv_len"][:, None])
    b = (q @ k.transpose(2, 3)).masked_fill_(~seen[:, None, None], float("-inf")).transpose(0, 1)  # [Hkv][n][g][own]
    m = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True) if b.shape[-1] else a.new_tensor(float("-inf")))
    m = m.masked_fill(m == float("-inf"), 0.0)
    a, b = a.sub_(m).exp_(), (b - m).exp_()
    total = a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True)
    out = (a.flatten(1, 2) @ prefix(s["v_pages"])).view(kv_heads, n, g, dim)
    out = out + (b.transpose(0, 1) @ (rest(s["v_pages"]) * seen[:, None, :, None])).transpose(0, 1)
    s["out"].copy_((out / total.clamp_min(1e-30)).transpose(0, 1).reshape(n, heads, dim))
    return s["out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "gate"):
        m, k = case["rows"], case["width"]
        if op == "gate":
            return {"bytes": m * (5 * k + 4) + 4 * k, "flops": 9 * m * k}
        x = 2 if case["kind"] == "bf16" else 4
        return {"bytes": m * (k * (x + (8 if case["residual"] else 0) + 1) + 4) + 4 * k, "flops": 7 * m * k}
    if op == "lora":
        m, n, k, rank = (case[x] for x in ("rows", "n", "k", "rank"))
        used = [a for a in _adapters_of(case) if a >= 0]
        return {"bytes": m * (k + 4 * n + 8) + 2 * len(set(used)) * rank * (n + k), "flops": 2 * len(used) * rank * (n + k) + m * n}
    kv = _lengths(case)
    heads, kv_heads, dim, shared = case["heads"], case["kv_heads"], case["dim"], case["shared"]
    rows = min(shared, max(kv)) + sum(max(0, x - shared) for x in kv)
    table = 4 * sum(-(-max(0, x - shared) // case["page"]) for x in kv) + 4 * -(-shared // case["page"]) + 4 * len(kv)
    return {"bytes": 4 * rows * kv_heads * dim + 4 * len(kv) * heads * dim + table, "flops": 4 * sum(kv) * heads * dim}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """Row by row, adapter by adapter and sequence by sequence from the
    operators' definitions; the same inputs as `run`, none of its code."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "gate"):
        k = case["width"]
        if op == "norm":
            t = s["x"].double()
            if case["residual"]:
                t = t + s["h"].double()
            h = t if case["residual"] else None
        else:
            t = s["gu"][:, :k].double().clamp(min=0) ** 2 * s["gu"][:, k:].double()
        t = t * s["gamma"].double() / torch.sqrt((t * t).sum(1, keepdim=True) / k + EPS)
        scale = 127.0 / t.abs().max(1, keepdim=True).values.clamp(min=1e-5)
        got = {"s": scale[:, 0], "values": torch.clamp(torch.round(t * scale), -128, 127) / scale}
        return {"h": h, **got} if op == "norm" else got
    if op == "lora":
        out = s["y"].double()
        for a in range(case["adapters"]):
            rows = torch.nonzero(s["adapter"] == a)[:, 0]
            if len(rows):
                u = (s["x"][rows].double() / s["s"][rows].double()[:, None]) @ s["A"][a].double().T
                out[rows] += s["scale"][a].double() * (u @ s["B"][a].double().T)
        return out
    heads, kv_heads, dim, page, shared = (case[x] for x in ("heads", "kv_heads", "dim", "page", "shared"))
    g = heads // kv_heads
    common, table = s["shared_table"].cpu().tolist(), s["page_table"].cpu().tolist()
    out = torch.zeros(case["seqs"], heads, dim, dtype=torch.float64, device=s["q"].device)

    def gather(pool, ids):
        ids = torch.tensor(ids, dtype=torch.int64, device=out.device)
        return pool[ids].transpose(0, 1).reshape(kv_heads, -1, dim).double()

    k_all, v_all = gather(s["k_pages"], common), gather(s["v_pages"], common)
    for b, length in enumerate(_lengths(case)):
        if not length:
            continue
        end, first = min(length, shared), shared // page
        k, v = k_all[:, :end], v_all[:, :end]
        if length > shared:
            ids = table[b][first:-(-length // page)]
            tail = slice(shared - first * page, length - first * page)
            k = torch.cat((k, gather(s["k_pages"], ids)[:, tail]), 1)
            v = torch.cat((v, gather(s["v_pages"], ids)[:, tail]), 1)
        score = torch.einsum("gqd,gjd->gqj", s["q"][b].double().view(kv_heads, g, dim), k) / math.sqrt(dim)
        out[b] = torch.einsum("gqj,gjd->gqd", torch.softmax(score, 2), v).reshape(heads, dim)
    return out
