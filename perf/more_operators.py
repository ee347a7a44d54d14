"""The operators over 8-bit (e4m3) values with a scale for each block of 128 as measured cases: the conversion of
activations and weights, the matrix product, and the whole mixture-of-experts layer for a few tokens.

``run`` computes them in plain torch operations (fp32) or, with ``own`` set, calls this package's entry points.
``exact`` evaluates the definitions in fp64.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0
OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------------- cases


def listed():
    moe = dict(op="moe", Hd=7168, I=2048, E=256, k=8, shared=1, res=True)
    return [
        # one token's normalised activations before a projection: launch latency
        dict(name="quant_b1", op="quant", M=1, K=7168, x="bf16", rows=1),
        # the activations of a prompt of 8191 tokens
        dict(name="quant_prompt", op="quant", M=8191, K=7168, x="bf16", rows=1),
        # the input projection's weight matrix, once at load time, from fp32 with a ragged last group of rows
        dict(name="quant_weight", op="quant", M=16416, K=7168, x="f32", rows=128),
        # one token through the input projection (q, k, v, gate and one row per head)
        dict(name="mm_b1_in", op="mm", M=1, N=16416, K=7168, y="bf16", res=False),
        # a decode batch of 16 through the output projection, added to the residual stream
        dict(name="mm_b16_out", op="mm", M=16, N=7168, K=4096, y="bf16", res=True),
        # a decode batch of 64, fp32 output (the type that the epilogue of the input projection reads)
        dict(name="mm_b64_in_f32", op="mm", M=64, N=16416, K=7168, y="f32", res=False),
        # a mixed batch: odd numbers of tokens and outputs, K that ends inside a block of 128
        dict(name="mm_b333_odd", op="mm", M=333, N=7001, K=4112, y="bf16", res=True),
        # a prompt of 8192 tokens through the input projection
        dict(name="mm_prompt", op="mm", M=8192, N=16416, K=7168, y="bf16", res=False),
        # the smallest layer: 16 experts of 128, one token
        dict(moe, name="moe_tiny", M=1, Hd=256, I=128, E=16, k=2, shared=0, res=False),
        # one sequence decoding, a batch of 8, and a batch of 64 (nearly every expert has work)
        dict(moe, name="moe_b1", M=1),
        dict(moe, name="moe_b8", M=8),
        dict(moe, name="moe_b64", M=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "mm", "mm", "mm", "moe", "moe"])
    if op == "quant":
        rows = rng.choice([1, 1, 128])
        return dict(op=op, M=_log(rng, 1, 16000), K=16 * _log(rng, 1, 448), x=rng.choice(["bf16", "bf16", "f32"]), rows=rows)
    if op == "mm":
        return dict(op=op, M=_log(rng, 1, 8192) if rng.random() < 0.5 else _log(rng, 1, 64), N=_log(rng, 1, 16416),
                    K=16 * _log(rng, 1, 448), y=rng.choice(["bf16", "bf16", "f32"]), res=rng.random() < 0.5)
    E = rng.choice([8, 16, 60, 64, 128, 256])
    return dict(op=op, M=_log(rng, 1, 64), Hd=128 * _log(rng, 1, 56), I=128 * _log(rng, 1, 16), E=E,
                k=rng.randint(1, min(8, E)), shared=rng.choice([0, 1, 1, 2]), res=rng.random() < 0.5)


def _up(x, a):
    return -(-x // a)


def work(c):
    if c["op"] == "quant":
        n = c["M"] * c["K"]
        scales = _up(c["M"], c["rows"]) * _up(c["K"], BLOCK)
        return {"bytes": n * ((2 if c["x"] == "bf16" else 4) + 1) + 4 * scales, "flops": 3 * n}
    M = c["M"]
    if c["op"] == "mm":
        N, K = c["N"], c["K"]
        kb = _up(K, BLOCK)
        moved = (M + N) * K + 4 * kb * (M + _up(N, BLOCK)) + M * N * ((2 if c["y"] == "bf16" else 4) + (2 if c["res"] else 0))
        return {"bytes": moved, "flops": 2 * M * N * K}
    Hd, I, E = c["Hd"], c["I"], c["E"]
    # experts that a batch of M independent choices of k out of E reaches
    units = E * (1.0 - (1.0 - c["k"] / E) ** M) + c["shared"]
    weights = 3 * Hd * I * (1 + 4 / BLOCK ** 2)
    moved = units * weights + 2 * E * Hd + M * Hd * (2 + 2 + (2 if c["res"] else 0)) + M * c["k"] * 8
    return {"bytes": int(moved), "flops": M * (2 * E * Hd + (c["k"] + c["shared"]) * 6 * Hd * I)}


# ----------------------------------------------------------------------------- inputs


def _weights(rows, K, g):
    """e4m3 weights [rows, K] and their scales [ceil(rows / 128), ceil(K / 128)]: N(0, 0.02^2) in all, each block's own spread."""
    w = torch.empty(rows, K, dtype=torch.float8_e4m3fn, device=DEV)
    flat, step = w.view(-1), 1 << 27
    for i in range(0, flat.numel(), step):
        part = flat[i:i + step]
        part.copy_((torch.randn(part.numel(), generator=g, device=DEV, dtype=torch.float16) * 100.0).clamp_(-E4M3_MAX, E4M3_MAX))
    scale = (torch.rand(_up(rows, BLOCK), _up(K, BLOCK), generator=g, device=DEV) + 0.5) * (0.02 / 100.0)
    return w, scale


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=c)
    M = c["M"]
    if own:
        from hybrid_linear_attention_gated_gb300 import hla
        s["hla"] = hla
    if c["op"] == "quant":
        K = c["K"]
        # channels of different size, as activations and weights have them
        s["x"] = (_normal((M, K), g, torch.float32) * torch.exp(_normal((1, K), g, torch.float32))).to(OUT[c["x"]])
        s["q"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=DEV)
        s["scale"] = torch.empty(_up(M, c["rows"]), _up(K, BLOCK), device=DEV)
        return s
    if c["op"] == "mm":
        N, K = c["N"], c["K"]
        s["x"], s["x_scale"] = _quantize(_normal((M, K), g).float())
        s["w"], s["w_scale"] = _weights(N, K, g)
        s["residual"] = _normal((M, N), g) if c["res"] else None
        s["y"] = torch.empty(M, N, dtype=OUT[c["y"]], device=DEV)
        return s
    Hd, I, E = c["Hd"], c["I"], c["E"]
    s["w_router"] = (_normal((E, Hd), g, torch.float32) * 0.02).to(torch.bfloat16)
    s["x"] = _normal((M, Hd), g)
    for _ in range(50):  # no two of a token's first k + 1 scores closer than 1e-5: tokens that have such are drawn again
        top = (s["x"].double() @ s["w_router"].double().T).sort(-1, descending=True).values[:, :c["k"] + 1]
        near = (top.diff(dim=-1).neg() < 1e-5).any(-1)
        if not bool(near.any()):
            break
        s["x"][near] = _normal((int(near.sum()), Hd), g)
    for n, kind in ((E, ""), (c["shared"], "s")):
        for name, rows, K in (("gate", I, Hd), ("up", I, Hd), ("down", Hd, I)):
            w, scale = _weights(n * rows, K, g) if n else (None, None)
            s[f"w{kind}_{name}"] = w.view(n, rows, K) if n else None
            s[f"scale{kind}_{name}"] = scale.view(n, rows // BLOCK, K // BLOCK) if n else None
    s["residual"] = _normal((M, Hd), g) if c["res"] else None
    s["y"] = torch.empty(M, Hd, dtype=torch.bfloat16, device=DEV)
    s["topk_idx"] = torch.empty(M, c["k"], dtype=torch.int32, device=DEV)
    s["topk_w"] = torch.empty(M, c["k"], device=DEV)
    if own:  # the descriptor and the workspace that a program keeps beside the weights
        names = ("gate", "up", "down")
        s["layer"] = hla.make_moe_fp8(Hd, I, E, c["k"], c["shared"], s["w_router"], *(s["w_" + n] for n in names),
                                      *(s["scale_" + n] for n in names), *(s["ws_" + n] for n in names),
                                      *(s["scales_" + n] for n in names))
        s["ws"] = torch.empty(hla.moe_fp8_forward_workspace_size(s["layer"], M), dtype=torch.uint8, device=DEV)
    return s


# ----------------------------------------------------------------------------- one pass


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s)
    if c["op"] == "quant":
        q, scale = _quantize(s["x"].float(), c["rows"])
        s["q"].copy_(q)
        s["scale"].copy_(scale)
        return {"q": s["q"], "scale": s["scale"]}
    if c["op"] == "mm":
        y = torch.matmul(_values(s["x"], s["x_scale"], 1), _values(s["w"], s["w_scale"], BLOCK).T)
        s["y"].copy_(y if s["residual"] is None else y.add_(s["residual"]))
        return {"y": s["y"]}
    return _moe(s)


def _run_own(s):
    c, hla = s["case"], s["hla"]
    if c["op"] == "quant":
        hla.fp8_quantize(c["M"], c["K"], s["x"], hla.HLA_BF16 if c["x"] == "bf16" else hla.HLA_F32, c["rows"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    if c["op"] == "mm":
        hla.fp8_matmul(c["M"], c["N"], c["K"], s["x"], s["x_scale"], s["w"], s["w_scale"], s["residual"], s["y"],
                       hla.HLA_BF16 if c["y"] == "bf16" else hla.HLA_F32)
        return {"y": s["y"]}
    hla.moe_fp8_forward(s["layer"], c["M"], s["x"], s["residual"], s["y"], s["topk_idx"], s["topk_w"], s["ws"], s["ws"].numel())
    return {"y": s["y"], "topk_idx": s["topk_idx"], "topk_w": s["topk_w"]}


def _quantize(x, rows=1):
    """fp32 x [M, K] as e4m3 over the smallest power of two at or above max|x| / 448 of each block of rows x 128."""
    M, K = x.shape
    m, k = _up(M, rows), _up(K, BLOCK)
    if (M, K) != (m * rows, k * BLOCK):
        x = torch.nn.functional.pad(x, (0, k * BLOCK - K, 0, m * rows - M))
    x = x.view(m, rows, k, BLOCK)
    part, power = torch.frexp(x.abs().amax((1, 3)))  # part in [0.5, 1): 448 is 0.875 * 2^9
    power = torch.where(part > 0, power - 9 + (part > 0.875), -126).clamp(min=-126)
    scale = torch.ldexp(torch.ones_like(part), power)
    q = (x / scale[:, None, :, None]).view(m * rows, k * BLOCK)[:M, :K].contiguous()
    return q.to(torch.float8_e4m3fn), scale


def _values(q, scale, rows):
    """e4m3 [M, K] with its scales as fp32 values."""
    x = q.float()
    wide = scale.repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    return x.mul_(wide if rows == 1 else wide.repeat_interleave(rows, 0)[:x.shape[0]])


def _expert(s, kind, e, x):
    """Expert e (a number, or a tensor of one) of fp32 tokens x [M, Hd]: W_down of the 8-bit values of SiLU(W_gate x) * (W_up x)."""
    def w(name):
        q = s[f"w{kind}_{name}"].view(torch.uint8)[e].view(torch.float8_e4m3fn)
        return _values(q, s[f"scale{kind}_{name}"][e], BLOCK)

    gate, up = torch.matmul(x, w("gate").T), torch.matmul(x, w("up").T)
    h = gate / (1.0 + torch.exp(-gate)) * up
    return torch.matmul(_values(*_quantize(h), 1), w("down").T)


def _moe(s):
    c = s["case"]
    M, E, k = c["M"], c["E"], c["k"]
    # scores in fp64: two experts at the border of the choice may differ by less than fp32 holds
    logit = torch.matmul(s["x"].double(), s["w_router"].double().T)
    value, idx = logit.sort(stable=True, dim=-1, descending=True)
    idx, score = idx[:, :k], torch.sigmoid(value[:, :k])
    weight = (score / score.sum(-1, keepdim=True)).float()
    x = _values(*_quantize(s["x"].float()), 1)
    y = torch.zeros(M, c["Hd"], device=DEV) if s["residual"] is None else s["residual"].float()
    for e in range(c["shared"]):
        y += _expert(s, "s", e, x)
    if M * k <= E:  # an expert for each token and choice, or each expert for all tokens: whichever reads fewer weights
        for m in range(M):
            for j in range(k):
                y[m] += weight[m, j] * _expert(s, "", idx[m, j], x[m:m + 1])[0]
    else:
        for e in range(E):
            y += (weight * (idx == e)).sum(-1, keepdim=True) * _expert(s, "", e, x)
    s["y"].copy_(y)
    s["topk_idx"].copy_(idx)
    s["topk_w"].copy_(weight)
    return {"y": s["y"], "topk_idx": s["topk_idx"], "topk_w": s["topk_w"]}


# ----------------------------------------------------------------------------- the definitions in fp64


def _exact_scales(x, rows):
    """fp64 x [M, K] -> the scale of every element, [M, K], and of every block."""
    M, K = x.shape
    full = torch.empty_like(x)
    small = torch.empty(_up(M, rows), _up(K, BLOCK), dtype=torch.float64, device=DEV)
    for b in range(small.shape[1]):
        cols = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        top = x[:, cols].abs().amax(1)
        top = torch.nn.functional.pad(top, (0, small.shape[0] * rows - M)).view(-1, rows).amax(1)
        power = torch.floor(torch.log2((top / E4M3_MAX).clamp(min=2.0 ** -126)))
        low = torch.exp2(power)  # one step below the scale, or the scale itself where 448 of it reach the top
        small[:, b] = torch.where(low * E4M3_MAX < top, 2.0 * low, low)
        full[:, cols] = small[:, b].repeat_interleave(rows)[:M, None]
    return full, small


def _held(x):
    """fp64 x [M, K] after its conversion: the values that the 8 bits and their scales stand for."""
    full, _ = _exact_scales(x, 1)
    return (x / full).float().to(torch.float8_e4m3fn).double() * full


def _dense(q, scale):
    """e4m3 weights [N, K] with scales of 128 x 128 blocks in fp64."""
    w = q.double()
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= scale[i, j].double()
    return w


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "quant":
        x = s["x"].double()
        full, small = _exact_scales(x, c["rows"])
        return {"q": x / full, "scale": small}
    if c["op"] == "mm":
        x = s["x"].double() * s["x_scale"].double().repeat_interleave(BLOCK, 1)[:, :c["K"]]
        y = x @ _dense(s["w"], s["w_scale"]).T
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    M, k = c["M"], c["k"]
    x = s["x"].double()
    logits = x @ s["w_router"].double().T
    best = logits.topk(k, -1)
    share = 1.0 / (1.0 + torch.exp(-best.values))
    share = share / share.sum(-1, keepdim=True)
    y = torch.zeros(M, c["Hd"], dtype=torch.float64, device=DEV)
    if s["residual"] is not None:
        y += s["residual"].double()
    xq = _held(x)
    todo = [("s", e, list(range(M)), None) for e in range(c["shared"])]
    for e in range(c["E"]):
        hit = (best.indices == e).nonzero().tolist()
        if hit:
            todo.append(("", e, [m for m, _ in hit], share[tuple(zip(*hit))]))
    for kind, e, rows, weight in todo:
        gate, up, down = (s[f"w{kind}_{n}"][e].double() * s[f"scale{kind}_{n}"][e].double().kron(
            torch.ones(BLOCK, BLOCK, dtype=torch.float64, device=DEV)) for n in ("gate", "up", "down"))
        a, b = xq[rows] @ gate.T, xq[rows] @ up.T
        out = _held(a * torch.sigmoid(a) * b) @ down.T
        y[rows] += out if weight is None else weight[:, None] * out
    return {"y": y, "topk_idx": best.indices.int(), "topk_w": share}
