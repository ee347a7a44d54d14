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
