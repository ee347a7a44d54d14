"""The paged key-value cache operators as measured cases: append with rotation, attention of the newest
tokens, block selection by key bounds, and attention over the selected blocks.

``run`` computes them in plain torch operations (fp32, angles and block scores in fp64) or, with ``own``
set, calls this package's entry points.  ``exact`` evaluates the definitions in fp64.
"""

import math

import torch

own = False

DEV = "cuda"
LOWEST = float("-inf")
E4M3_MAX = 448.0


# ----------------------------------------------------------------------------- cases


def listed():
    base = dict(H=32, Hkv=8, d=128, page=64, kv="bf16", idle=0)
    app = dict(base, op="append", rope=128, inter=False, chunks=0, chunk=0)
    att = dict(base, op="decode", out="bf16")
    sel = dict(base, op="select", n_select=64, first=1, last=2)
    spa = dict(base, op="sparse", n_select=64, out="bf16")
    return [
        # one sequence decoding: the append is launch latency
        dict(app, name="append_b1", B=1, T=1, lo=1021, hi=1021),
        # speculative window of 4 drafted tokens for 64 sequences into an 8-bit cache, two slots idle
        dict(app, name="append_b64_t4_e4m3", B=64, T=4, lo=100, hi=8000, kv="e4m3", idle=2),
        # mixed batch: 60 decoding sequences and 4 prefill chunks of 512 tokens
        dict(app, name="append_mixed", B=64, T=1, lo=0, hi=4000, chunks=4, chunk=512),
        # prompts of 8 sequences, half of each head rotated, interleaved pairs, ragged lengths
        dict(app, name="append_prefill", B=8, T=1, lo=0, hi=70, chunks=8, chunk=4093, rope=64, inter=True),
        # one sequence decoding at 1 thousand tokens: latency of the split and the join
        dict(att, name="decode_b1_1k", B=1, T=1, lo=1021, hi=1021),
        # speculative window over a 64-wide head cache, small pages, fp32 output (the verify step's own type)
        dict(att, name="decode_b16_t4_d64_f32", B=16, T=4, H=24, d=64, page=16, lo=200, hi=6000, out="f32"),
        # a decode batch of 64 at ordinary lengths, ragged
        dict(att, name="decode_b64_8k", B=64, T=1, lo=500, hi=15500),
        # long contexts, 8-bit cache: more than 2^31 cached values
        dict(att, name="decode_b64_48k_e4m3", B=64, T=1, lo=30000, hi=65000, kv="e4m3"),
        # block choice of one sequence at 128 thousand tokens, and of a window batch at 64 thousand
        dict(sel, name="select_b1_128k", B=1, T=1, lo=131001, hi=131001),
        dict(sel, name="select_b32_t2_64k", B=32, T=2, lo=20000, hi=90000),
        # attention over the chosen blocks: one sequence, and a window batch with an 8-bit cache
        dict(spa, name="sparse_b1_128k", B=1, T=1, lo=131001, hi=131001),
        dict(spa, name="sparse_b32_t2_e4m3", B=32, T=2, lo=20000, hi=60000, kv="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "select", "sparse"])
    H, Hkv = rng.choice([(32, 8), (32, 4), (32, 2), (32, 32), (16, 1), (24, 8), (10, 2), (6, 3)])
    c = dict(op=op, H=H, Hkv=Hkv, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             kv=rng.choice(["bf16", "bf16", "e4m3"]), B=_log(rng, 1, 64), T=rng.choice([1, 1, 1, 2, 3, 4, 5, 8]))
    c["idle"] = 0 if c["B"] < 3 or rng.random() < 0.6 else rng.randint(1, max(1, c["B"] // 8))
    # cached tokens x kv heads over the batch stay below 8 million, so that no draw passes the largest listed case
    top = max(2, min(130000 if op in ("select", "sparse") else 60000, 8000000 // (c["B"] * c["Hkv"])))
    c["hi"] = _log(rng, min(top, 32 * c["page"]) if op == "select" else 1, top)
    c["lo"] = rng.randint(c["hi"] // 2 if op == "select" else 0, c["hi"])
    if op == "append":
        c["rope"] = rng.choice([0, 32, c["d"] // 2, c["d"]])
        c["inter"] = rng.random() < 0.5
        c["chunks"] = rng.randint(0, min(4, c["B"]))
        c["chunk"] = _log(rng, 2, 3000) if c["chunks"] else 0
    else:
        if op != "select":
            c["out"] = rng.choice(["bf16", "f32"])
        if op == "sparse":
            c["n_select"] = _log(rng, 4, 128)
        if op == "select":  # fewer than a sequence has, so that there is something to choose
            c["n_select"] = _log(rng, 4, max(4, min(128, c["hi"] // (4 * c["page"]))))
            c["first"], c["last"] = rng.randint(0, 1), rng.randint(0, 2)
    return c


def _lengths(c):
    """Tokens cached before the call, per sequence: spread over [lo, hi] (-1 marks an idle slot), from the case alone."""
    n = [c["lo"] + int((c["hi"] - c["lo"]) * ((i * 0.6180339887) % 1.0) + 0.5) for i in range(c["B"])]
    for i in range(c["idle"]):
        n[(i * 7 + 1) % c["B"]] = -1
    return n


def _news(c):
    """New tokens per sequence: T each; an append's last `chunks` sequences bring a prefill chunk instead."""
    n = [c["T"]] * c["B"]
    for i in range(c.get("chunks", 0)):
        n[c["B"] - 1 - i] = max(1, c["chunk"] - 3 * i)
    return n


def _blocks(c, new=None):
    new = new or [c["T"]] * c["B"]
    return [-(-(p + n) // c["page"]) if p >= 0 else 0 for p, n in zip(_lengths(c), new)]


def work(c):
    size = 1 if c["kv"] == "e4m3" else 2
    past, d, H, Hkv, T, P = _lengths(c), c["d"], c["H"], c["Hkv"], c["T"], c["page"]
    live = [p for p in past if p >= 0]
    if c["op"] == "append":
        new = [n for p, n in zip(past, _news(c)) if p >= 0]
        N = sum(new)
        touched = sum((p + n - 1) // P - p // P + 1 for p, n in zip(live, new))
        moved = N * d * (2 * 2 * H + 2 * Hkv * (2 + size)) + touched * Hkv * d * 4
        return {"bytes": moved, "flops": 6 * N * (H + Hkv) * c["rope"] // 2}
    rows = len(live) * T * H * d
    if c["op"] == "select":
        blocks = sum(-(-(p + T) // P) for p in live)
        pairs = sum((p + t) // P + 1 for p in live for t in range(T))
        return {"bytes": blocks * Hkv * d * 4 + rows * 2 + len(past) * T * Hkv * c["n_select"] * 4, "flops": 4 * d * H * pairs}
    io = rows * (2 + (2 if c["out"] == "bf16" else 4))
    if c["op"] == "decode":
        keys = sum(p + T for p in live)
        pairs = sum(p + t + 1 for p in live for t in range(T))
        return {"bytes": keys * Hkv * 2 * d * size + io, "flops": 4 * d * H * pairs}
    pairs = sum(min(c["n_select"] * P, p + t + 1) for p in live for t in range(T))
    lists = len(past) * T * Hkv * c["n_select"] * 4
    # the window's tokens may list the same blocks: the cache rows that cannot be done without are those of one token
    return {"bytes": pairs // T * Hkv * 2 * d * size + lists + io, "flops": 4 * d * H * pairs}


# ----------------------------------------------------------------------------- inputs


def _cache_values(shape, c, g, std):
    """Cached keys or values: N(0, std^2); an 8-bit cache holds them over a scale that puts std near 24."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn if c["kv"] == "e4m3" else torch.bfloat16, device=DEV)
    flat, step = out.view(-1), 1 << 27
    unit = 24.0 if c["kv"] == "e4m3" else std
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV, dtype=torch.float16) * unit)
    return out


def _normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, T, H, Hkv, d, P = (c[k] for k in ("B", "T", "H", "Hkv", "d", "page"))
    new = _news(c)
    blocks = _blocks(c, new)
    n_pages, most = sum(blocks) + 3, max(max(blocks), 1)
    s = dict(case=c, n_pages=n_pages, most=most, scale=1.0 / math.sqrt(d))
    s["past"] = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)
    # pages handed out in random order; entries behind a sequence's last block are -1
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    count = torch.tensor(blocks, device=DEV)
    start = torch.cumsum(count, 0) - count
    at = torch.arange(most, device=DEV)
    table = order[(start[:, None] + at).clamp(max=n_pages - 1)]
    s["table"] = torch.where(at < count[:, None], table, torch.full_like(table, -1)).contiguous()
    s["k_scale"] = s["v_scale"] = None
    if c["kv"] == "e4m3":
        s["k_scale"] = (torch.rand(Hkv, generator=g, device=DEV) + 0.5) / 24.0
        s["v_scale"] = (torch.rand(Hkv, generator=g, device=DEV) + 0.5) / 24.0
    s["k"] = s["v"] = s["kmin"] = s["kmax"] = None
    if c["op"] != "select":
        s["k"] = _cache_values((n_pages, Hkv, P, d), c, g, 1.0)
        s["v"] = _cache_values((n_pages, Hkv, P, d), c, g, 1.0)
    if c["op"] == "append":
        N = sum(new)
        s["cu"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
        s["N"] = N
        s["q_in"], s["k_in"], s["v_in"] = _normal((N, H, d), g), _normal((N, Hkv, d), g), _normal((N, Hkv, d), g)
        half = c["rope"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / max(half, 1))
        s["kmin"] = torch.zeros(n_pages, Hkv, d, dtype=torch.bfloat16, device=DEV)
        s["kmax"] = torch.zeros_like(s["kmin"])
        s["q_out"] = torch.zeros_like(s["q_in"])
    else:
        s["q"] = _normal((B, T, H, d), g, 1.5)
    if c["op"] == "select":
        mid, wide = _normal((n_pages, Hkv, d), g, 1.0).float(), _normal((n_pages, Hkv, d), g, 0.7).float().abs()
        s["kmin"], s["kmax"] = (mid - wide).to(torch.bfloat16), (mid + wide).to(torch.bfloat16)
        s["sel"] = torch.empty(B, T, Hkv, c["n_select"], dtype=torch.int32, device=DEV)
    if c["op"] in ("decode", "sparse"):
        s["o"] = torch.empty(B, T, H, d, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
    if c["op"] == "sparse":
        # ascending distinct blocks of what each token sees, its newest block among them; -1 where it sees fewer
        n = c["n_select"]
        seen = (s["past"][:, None] + torch.arange(T, device=DEV)).div(P, rounding_mode="floor")  # [B, T]: the newest block
        width = max(most, n)
        at = torch.arange(width, device=DEV)
        key = torch.rand(B, T, Hkv, width, generator=g, device=DEV)
        key = torch.where(at == seen[:, :, None, None], 2.0, key)
        key = torch.where(at <= seen[:, :, None, None], key, -1.0)
        best = key.topk(n, -1)
        pick = torch.where(best.values >= 0, best.indices, width).sort(-1).values
        s["sel"] = torch.where(pick < width, pick, -1).to(torch.int32).contiguous()
    if own:  # the descriptor and the workspace that a program keeps beside the cache
        from hybrid_linear_attention_gated_gb300 import hla
        s["hla"] = hla
        s["C"] = C = hla.make_kv_cache(hla.HLA_E4M3 if c["kv"] == "e4m3" else hla.HLA_BF16, n_pages, P, Hkv, d,
                                       s["k"], s["v"], s["k_scale"], s["v_scale"], s["kmin"], s["kmax"])
        need = {"append": lambda: 0,
                "decode": lambda: hla.attn_paged_decode_workspace_size(C, B, T, H),
                "select": lambda: hla.attn_select_blocks_workspace_size(C, B, T, H, most),
                "sparse": lambda: hla.attn_paged_sparse_workspace_size(C, B, T, H)}[c["op"]]()
        s["ws"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------- one pass


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "decode": _decode, "select": _select, "sparse": _sparse}[state["case"]["op"]](state)


def _run_own(s):
    c, hla, C = s["case"], s["hla"], s["C"]
    B, T, H = c["B"], c["T"], c["H"]
    if c["op"] == "append":
        hla.kv_cache_append(C, s["N"], B, s["cu"], s["past"], s["most"], s["table"], H, s["q_in"], s["k_in"], s["v_in"],
                            c["rope"], int(c["inter"]), s["inv_freq"] if c["rope"] else None, s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"], "kmin": s["kmin"], "kmax": s["kmax"]}
    if c["op"] == "select":
        hla.attn_select_blocks(C, B, T, H, s["most"], s["table"], s["past"], c["n_select"], c["first"], c["last"], s["q"],
                               s["sel"], s["ws"], s["ws"].numel())
        return {"sel": s["sel"]}
    dt = hla.HLA_BF16 if c["out"] == "bf16" else hla.HLA_F32
    if c["op"] == "decode":
        hla.attn_paged_decode(C, B, T, H, s["most"], s["table"], s["past"], s["scale"], s["q"], s["o"], dt, s["ws"],
                              s["ws"].numel())
    else:
        hla.attn_paged_sparse(C, B, T, H, s["most"], s["table"], s["past"], c["n_select"], s["sel"], s["scale"], s["q"],
                              s["o"], dt, s["ws"], s["ws"].numel())
    return {"o": s["o"]}


def _rotate(x, pos, s):
    """x [N, heads, d] as fp32, its first rope channels rotated by pos * inv_freq (angles in fp64)."""
    c = s["case"]
    x = x.float()
    if not c["rope"]:
        return x
    a = pos.double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    r, rest = x[..., :c["rope"]], x[..., c["rope"]:]
    if c["inter"]:
        u, w = r[..., 0::2], r[..., 1::2]
        out = torch.stack((u * cos - w * sin, u * sin + w * cos), -1).flatten(-2)
    else:
        u, w = r.chunk(2, -1)
        out = torch.cat((u * cos - w * sin, u * sin + w * cos), -1)
    return torch.cat((out, rest), -1)


def _bytes(x):
    """A cache's values as bytes: torch indexes 8-bit floats only so."""
    return x.view(torch.uint8)


def _taken(x, *at):
    return _bytes(x)[at].view(x.dtype)


def _stored(x, scale, like):
    """fp32 values as the cache holds them."""
    if like.dtype == torch.bfloat16:
        return x.to(torch.bfloat16)
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(like.dtype)


def _places(s):
    """Sequence and position of every token, which of them are kept, and their page and row."""
    P, past = s["case"]["page"], s["past"].long()
    n = torch.arange(s["N"], device=DEV)
    b = torch.searchsorted(s["cu"].long(), n, right=True) - 1
    pos = past[b] + n - s["cu"].long()[b]
    live = past[b] >= 0
    return pos, live, s["table"].long()[b[live], pos[live] // P], pos[live] % P


def _append(s):
    c, P = s["case"], s["case"]["page"]
    pos, live, page, row = _places(s)
    q = _rotate(s["q_in"], pos, s).to(torch.bfloat16)
    s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"]))
    for name, x in (("k", _rotate(s["k_in"], pos, s)), ("v", s["v_in"].float())):
        _bytes(s[name])[page, :, row] = _bytes(_stored(x, s[name + "_scale"], s[name]))[live]
    past, end = s["past"].long(), s["past"].long() + s["cu"].long().diff()
    at = torch.arange(s["most"], device=DEV)
    touched = (past >= 0)[:, None] & (at >= (past // P)[:, None]) & (at * P < end[:, None])
    b, j = touched.nonzero(as_tuple=True)
    page = s["table"].long()[b, j]
    keys = _taken(s["k"], page).float()
    valid = (torch.arange(P, device=DEV) < (end[b] - j * P)[:, None])[:, None, :, None]
    s["kmin"][page] = torch.where(valid, keys, math.inf).amin(2).to(torch.bfloat16)
    s["kmax"][page] = torch.where(valid, keys, -math.inf).amax(2).to(torch.bfloat16)
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "kmin": s["kmin"], "kmax": s["kmax"]}


def _softmax_out(s, q, k, v, mask):
    """q [..., R, d], k and v [..., L, d] fp32, mask [..., R, L]: softmax(scale q k^T) v, zero rows where the mask has nothing."""
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~mask, LOWEST)
    top = score.amax(-1, keepdim=True)
    p = torch.exp_(score.sub_(torch.where(top == LOWEST, 0.0, top)))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, 1.0)


def _scaled(x, scale, shape):
    x = x.float()
    return x if scale is None else x.mul_(scale.view(shape))


def _decode(s):
    c = s["case"]
    B, T, H, Hkv, d = (c[k] for k in ("B", "T", "H", "Hkv", "d"))
    pages = s["table"].long().clamp(min=0)
    k = _scaled(_taken(s["k"], pages), s["k_scale"], (1, 1, Hkv, 1, 1)).transpose(1, 2).reshape(B, Hkv, -1, d)
    v = _scaled(_taken(s["v"], pages), s["v_scale"], (1, 1, Hkv, 1, 1)).transpose(1, 2).reshape(B, Hkv, -1, d)
    q = s["q"].float().view(B, T, Hkv, H // Hkv, d).transpose(1, 2).reshape(B, Hkv, -1, d)
    at = torch.arange(k.shape[2], device=DEV)
    newest = torch.where(s["past"] >= 0, s["past"], -T)[:, None] + torch.arange(T, device=DEV)  # [B, T]
    mask = (at <= newest[:, :, None]).repeat_interleave(H // Hkv, 1)[:, None]
    o = _softmax_out(s, q, k, v, mask)
    o = o.view(B, Hkv, T, H // Hkv, d).transpose(1, 2).reshape(B, T, H, d)
    s["o"].copy_(o)
    return {"o": s["o"]}


def _sparse(s):
    c = s["case"]
    B, T, H, Hkv, d, P = (c[k] for k in ("B", "T", "H", "Hkv", "d", "page"))
    sel = s["sel"].long()
    b = torch.arange(B, device=DEV)[:, None, None, None]
    page = s["table"].long()[b, sel.clamp(0, s["most"] - 1)].clamp(min=0)
    head = torch.arange(Hkv, device=DEV)[:, None]
    k = _scaled(_taken(s["k"], page, head), s["k_scale"], (1, 1, Hkv, 1, 1, 1)).reshape(B, T, Hkv, -1, d)
    v = _scaled(_taken(s["v"], page, head), s["v_scale"], (1, 1, Hkv, 1, 1, 1)).reshape(B, T, Hkv, -1, d)
    at = (sel[..., None] * P + torch.arange(P, device=DEV)).reshape(B, T, Hkv, -1)
    newest = (torch.where(s["past"] >= 0, s["past"], -T)[:, None] + torch.arange(T, device=DEV))[:, :, None, None]
    mask = ((at <= newest) & (sel >= 0).repeat_interleave(P, -1))[:, :, :, None]
    o = _softmax_out(s, s["q"].float().view(B, T, Hkv, H // Hkv, d), k, v, mask)
    s["o"].copy_(o.reshape(B, T, H, d))
    return {"o": s["o"]}


def _select(s):
    c = s["case"]
    B, T, H, Hkv, d, P, n = (c[k] for k in ("B", "T", "H", "Hkv", "d", "page", "n_select"))
    pages = s["table"].long().clamp(min=0)
    q = s["q"].double().view(B, T, Hkv, H // Hkv, d).transpose(1, 2).reshape(B, Hkv, -1, d)
    hi, lo = s["kmax"][pages].permute(0, 2, 3, 1).double(), s["kmin"][pages].permute(0, 2, 3, 1).double()
    # scores in fp64: two blocks at the border of the choice may differ by less than fp32 holds
    score = torch.matmul(q.clamp(min=0), hi) + torch.matmul(q.clamp(max=0), lo)
    score = score.view(B, Hkv, T, H // Hkv, -1).amax(3).transpose(1, 2)  # [B, T, Hkv, blocks]
    at = torch.arange(s["most"], device=DEV)
    newest = torch.where(s["past"] >= 0, s["past"], -T * P - P)[:, None] + torch.arange(T, device=DEV)
    newest = newest.div(P, rounding_mode="floor")[:, :, None, None]
    score = score.masked_fill((at < c["first"]) | (at > newest - c["last"]), math.inf).masked_fill(at > newest, -math.inf)
    order = score.sort(stable=True, dim=-1, descending=True).indices[..., :n]
    order = torch.where(order <= newest, order, s["most"]).sort(-1).values
    s["sel"].fill_(-1)
    s["sel"][..., :order.shape[-1]] = torch.where(order < s["most"], order, -1).to(torch.int32)
    return {"sel": s["sel"]}


# ----------------------------------------------------------------------------- the definitions in fp64


def exact(case, seed):
    c = case
    if c["op"] == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    B, T, H, Hkv, d, P = (c[k] for k in ("B", "T", "H", "Hkv", "d", "page"))
    past, table = _lengths(c), s["table"].tolist()
    ks = s["k_scale"].double() if s["k_scale"] is not None else torch.ones(Hkv, device=DEV, dtype=torch.float64)
    vs = s["v_scale"].double() if s["v_scale"] is not None else torch.ones(Hkv, device=DEV, dtype=torch.float64)
    if c["op"] == "append":
        k, v, q = s["k"].double(), s["v"].double(), s["q_out"].double()
        kmin, kmax = s["kmin"].double(), s["kmax"].double()
        i, half = 0, c["rope"] // 2
        lim = E4M3_MAX if c["kv"] == "e4m3" else math.inf
        for b, n in enumerate(_news(c)):
            if past[b] >= 0:
                pos = torch.arange(past[b], past[b] + n, device=DEV)
                turn = torch.polar(torch.ones(n, half, device=DEV, dtype=torch.float64), pos.double()[:, None] * s["inv_freq"])[:, None]

                def spin(x):
                    x = x[i:i + n].double()
                    r = x[..., :c["rope"]]
                    pair = r.unflatten(-1, (half, 2)) if c["inter"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
                    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
                    return torch.cat(((z if c["inter"] else z.transpose(-1, -2)).flatten(-2), x[..., c["rope"]:]), -1)

                q[i:i + n] = spin(s["q_in"]) if half else s["q_in"][i:i + n].double()
                kk = spin(s["k_in"]) if half else s["k_in"][i:i + n].double()
                page = s["table"][b].long()[pos // P]
                k[page, :, pos % P] = (kk / ks[:, None]).clamp(-lim, lim)
                v[page, :, pos % P] = (s["v_in"][i:i + n].double() / vs[:, None]).clamp(-lim, lim)
                for j in range(past[b] // P, (past[b] + n - 1) // P + 1):
                    rows = k[table[b][j], :, :min(P, past[b] + n - j * P)]
                    if c["kv"] == "e4m3":  # the bounds are those of the keys as they are held
                        rows = rows.to(s["k"].dtype).double()
                    kmin[table[b][j]], kmax[table[b][j]] = rows.amin(1), rows.amax(1)
            i += n
        return {"q": q, "k": k, "v": v, "kmin": kmin, "kmax": kmax}
    o = torch.zeros(B, T, H, d, dtype=torch.float64, device=DEV)
    sel = s["sel"] if c["op"] == "sparse" else None
    if sum(max(p, 0) for p in past) * H * d * T > 3e11 or (sel is not None and B * T * Hkv > 3000):
        return None  # too long in fp64
    for b in range(B):
        if past[b] < 0:
            continue
        rows = s["table"][b][:-(-(past[b] + T) // P)].long()
        if sel is None:
            kk = _taken(s["k"], rows).transpose(0, 1).reshape(Hkv, -1, d).double() * ks[:, None, None]
            vv = _taken(s["v"], rows).transpose(0, 1).reshape(Hkv, -1, d).double() * vs[:, None, None]
        for t in range(T):
            qq = s["q"][b, t].double().view(Hkv, H // Hkv, d) * s["scale"]
            if sel is None:
                w = torch.softmax(qq @ kk[:, :past[b] + t + 1].mT, -1)
                o[b, t] = (w @ vv[:, :past[b] + t + 1]).reshape(H, d)
                continue
            for h in range(Hkv):
                blocks = sel[b, t, h][sel[b, t, h] >= 0].long()
                seen = (blocks[:, None] * P + torch.arange(P, device=DEV)).flatten() <= past[b] + t
                kk = _taken(s["k"], rows[blocks], h).reshape(-1, d)[seen].double() * ks[h]
                vv = _taken(s["v"], rows[blocks], h).reshape(-1, d)[seen].double() * vs[h]
                o[b, t, h * (H // Hkv):(h + 1) * (H // Hkv)] = torch.softmax(qq[h] @ kk.mT, -1) @ vv
    return {"o": o}
