"""Inputs and tolerances of the GPU tests of the 8-bit operators (fp64 references on the GPU, written for speed)."""

import torch

BLOCK = 128


def up(x, a):
    return -(-x // a)


def generator(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def e4m3_weights(rows, K, g, dev, spread=100.0):
    w = (torch.randn(rows, K, generator=g, device=dev) * spread).clamp(-448, 448).to(torch.float8_e4m3fn)
    s = (torch.rand(up(rows, BLOCK), up(K, BLOCK), generator=g, device=dev) + 0.5) * (0.02 / spread)
    return w, s


def values64(q, s, rows):
    wide = s.double().repeat_interleave(BLOCK, 1)[:, :q.shape[1]]
    return q.double() * (wide if rows == 1 else wide.repeat_interleave(rows, 0)[:q.shape[0]])


def matmul64(x, xs, W, ws, residual=None):
    """(y, bound): the product in fp64 and how far an fp32 evaluation may be off.

    With A the product of the magnitudes: the 128 products of a block are exact and are added in fp32, each addition off by at
    most one unit in the last place, 2^-23, of what A's share of the block has reached: 128 * 2^-23 * A in all.  The two
    scales' product, its product with the block's sum and the additions over the blocks (and the join of up to 8 parts
    and the residual) are off by half a unit each: (blocks + 11) * 2^-24 * A.
    """
    a, b = values64(x, xs, 1), values64(W, ws, BLOCK)
    y, A = a @ b.T, a.abs() @ b.abs().T
    if residual is not None:
        y, A = y + residual.double(), A + residual.double().abs()
    blocks = xs.shape[1]
    return y, A * (128 * 2.0 ** -23 + (blocks + 11) * 2.0 ** -24)


def rounded(bound, y, dtype):
    """The bound after the rounding of y to its output type (half a step)."""
    return bound + (y.abs() + bound) * (torch.finfo(dtype).eps / 2)


def _e4m3(x):
    """fp64 -> nearest e4m3 value in fp64 (through fp32: the values here have far fewer bits than would round twice)."""
    return x.float().to(torch.float8_e4m3fn).double()


def quantized64(x):
    """fp64 x [M, K], K a multiple of 128, after its conversion (one row a block): values in fp64."""
    b = x.view(x.shape[0], -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True).clamp(min=448 * 2.0 ** -126)
    scale = torch.exp2(torch.floor(torch.log2(top / 448.0)))
    scale = torch.where(scale * 448.0 < top, 2 * scale, scale)
    return (_e4m3(b / scale) * scale).view_as(x)


class Moe:
    """A layer of 8-bit experts with the descriptor, and its fp64 reference with a bound on an fp32 evaluation's error."""

    def __init__(self, hla, dev, Hd, I, E, k, shared, seed):
        g = generator(dev, seed)
        self.hla, self.Hd, self.I, self.E, self.k, self.shared, self.dev = hla, Hd, I, E, k, shared, dev
        self.W_r = (torch.randn(E, Hd, generator=g, device=dev) * Hd ** -0.5 * 1.5).to(torch.bfloat16)
        self.w, self.s = {}, {}
        for kind, n in (("", E), ("s", shared)):
            for name, rows, K in (("gate", I, Hd), ("up", I, Hd), ("down", Hd, I)):
                if n:
                    w, s = e4m3_weights(n * rows, K, g, dev)
                    s *= 50.0 * K ** -0.5   # outputs near 1 whatever the width
                    self.w[kind + name], self.s[kind + name] = w.view(n, rows, K), s.view(n, rows // BLOCK, K // BLOCK)
        self.L = self.descriptor()

    def descriptor(self):
        n = ("gate", "up", "down")
        args = [self.w.get(x) for x in n] + [self.s.get(x) for x in n] + [self.w.get("s" + x) for x in n] + [self.s.get("s" + x) for x in n]
        return self.hla.make_moe_fp8(self.Hd, self.I, self.E, self.k, self.shared, self.W_r, *args)

    def tokens(self, M, seed):
        """Tokens whose first k + 1 scores are 1e-4 apart, so that fp32 logits order them as fp64 ones."""
        g = generator(self.dev, seed)
        x = torch.randn(M, self.Hd, generator=g, device=self.dev).to(torch.bfloat16)
        for _ in range(50):
            top = (x.double() @ self.W_r.double().T).sort(-1, descending=True).values[:, :self.k + 1]
            near = (top.diff(dim=-1).neg() < 1e-4).any(-1)
            if not bool(near.any()):
                return x
            x[near] = torch.randn(int(near.sum()), self.Hd, generator=g, device=self.dev).to(torch.bfloat16)
        raise AssertionError("no tokens without near ties")

    def workspace(self, M, fill=0xFF):
        n = self.hla.moe_fp8_forward_workspace_size(self.L, M)
        return torch.full((n,), fill, dtype=torch.uint8, device=self.dev)

    def run(self, x, residual=None, ws=None, **kw):
        M = x.shape[0]
        ws = self.workspace(M) if ws is None else ws
        y = torch.full_like(x, 7.0)
        idx = torch.full((M, self.k), -7, dtype=torch.int32, device=self.dev)
        w = torch.full((M, self.k), 7.0, device=self.dev)
        self.hla.moe_fp8_forward(self.L, M, x, residual, y, idx, w, ws, ws.numel(), **kw)
        return y, idx, w

    def reference(self, x, residual=None):
        """(y, bound, idx, w) in fp64.

        Sums as in matmul64.  SiLU by __expf is off by (2 + 1.173 |g|) units in the last place and three roundings more.
        Where the error of h can move a value across a rounding border of e4m3, or the block's largest magnitude across a
        power of two, the bound takes the distance between both conversions; w and the two scales add 2^-22.
        """
        logits = x.double() @ self.W_r.double().T
        val, idx = logits.sort(stable=True, dim=-1, descending=True)
        val, idx = val[:, :self.k], idx[:, :self.k]
        w = torch.sigmoid(val)
        w = w / w.sum(-1, keepdim=True)
        xq = quantized64(x.double())
        y = torch.zeros_like(xq) if residual is None else residual.double().clone()
        A, bound = y.abs(), torch.zeros_like(y)
        slack = 128 * 2.0 ** -23 + (self.Hd // BLOCK + 8) * 2.0 ** -24
        for kind, e in [("", int(e)) for e in idx.unique()] + [("s", e) for e in range(self.shared)]:
            if kind:
                rows, share = torch.arange(x.shape[0], device=self.dev), torch.ones(x.shape[0], dtype=torch.float64, device=self.dev)
            else:
                rows, slot = (idx == e).nonzero(as_tuple=True)
                share = w[rows, slot]
            m = {n: values64(self.w[kind + n][e], self.s[kind + n][e], BLOCK) for n in ("gate", "up", "down")}
            a = xq[rows]
            gate, up_ = a @ m["gate"].T, a @ m["up"].T
            dg, du = (a.abs() @ m["gate"].abs().T) * slack, (a.abs() @ m["up"].abs().T) * slack
            silu = gate * torch.sigmoid(gate)
            h = silu * up_
            dh = 1.1 * dg * (up_.abs() + du) + silu.abs() * du + h.abs() * (8 + 1.173 * gate.abs()) * 2.0 ** -23
            hq = quantized64(h)
            both = [quantized64(h + s * dh) for s in (-1, 1)]
            dq = torch.maximum((both[0] - hq).abs(), (both[1] - hq).abs())
            out, mag = hq @ m["down"].T, hq.abs() @ m["down"].abs().T
            y[rows] += share[:, None] * out
            A[rows] += share[:, None] * mag
            bound[rows] += share[:, None] * (dq @ m["down"].abs().T)
        units = x.shape[0] * self.k + self.shared
        bound += A * (128 * 2.0 ** -23 + 2.0 ** -21 + (units * (self.I // BLOCK) + 8) * 2.0 ** -24)
        return y, bound, idx, w
