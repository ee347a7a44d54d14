"""Operators over e4m3 values with a scale for each block of 128: conversion, matrix product, the mixture-of-experts layer.

Test infrastructure only (see ``oracle/__init__``).  float64 throughout.

"Kimi K3: From Day-0 Availability to Optimized Inference" (webinar summary), profiling paragraph, and "Hyper-optimizing
Kimi K3 in vLLM", Part 1 section 3: at low batch the cost is moving expert weights through GPU memory, which 8-bit
weights halve.  The pages give no 8-bit format.  The one here: a value is q * s, q an e4m3 value and s one number for
each block of ``rows`` x 128 values; the conversion takes for s the smallest power of two, 2^-126 at least, that
brings the block's largest magnitude to 448 or below.
"""

import math

import numpy as np

from .attention import E4M3_MAX, e4m3_round
from .moe import route_topk
from .numerics import f64, silu

BLOCK = 128


def block_scale(top):
    """The scale of a block whose largest magnitude is ``top`` (NaN for NaN and infinities)."""
    if not math.isfinite(top):
        return math.nan
    e = -126
    while E4M3_MAX * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def quantize(x, rows=1):
    """x [M, K] -> (q [M, K] of e4m3 values, scale [ceil(M / rows), ceil(K / 128)])."""
    x = f64(x)
    M, K = x.shape
    q = np.empty_like(x)
    scale = np.empty((-(-M // rows), -(-K // BLOCK)))
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            at = np.s_[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]
            top = np.abs(x[at]).max()
            scale[i, j] = block_scale(math.nan if np.isnan(top) else top)
            q[at] = e4m3_round(x[at] / scale[i, j])
    return q, scale


def values(q, scale, rows=1):
    """What q and its scales stand for."""
    q = f64(q)
    M, K = q.shape
    return q * np.repeat(np.repeat(f64(scale), rows, 0)[:M], BLOCK, 1)[:, :K]


def matmul(x, x_scale, W, w_scale, residual=None):
    y = values(x, x_scale) @ values(W, w_scale, BLOCK).T
    return y if residual is None else y + f64(residual)


def expert(x, gate, up, down):
    """One expert on values x [M, Hd]; gate, up, down: values of its matrices.  h is converted before the last product."""
    h = silu(x @ gate.T) * (x @ up.T)
    return values(*quantize(h)) @ down.T


def moe_layer(x, W_r, k, experts, shared=(), residual=None):
    """Router, routed and shared experts of tokens x [M, Hd]: (y, topk_idx, topk_w).

    experts: callable e -> (gate, up, down) as values; shared: a sequence of the same.  The router sees x itself, the
    experts its converted values.
    """
    idx, w, _ = route_topk(x, W_r, k)
    xq = values(*quantize(x))
    y = np.zeros(f64(x).shape) if residual is None else f64(residual).copy()
    for e in sorted(set(idx.flatten().tolist())):
        rows, slots = np.nonzero(idx == e)
        y[rows] += w[rows, slots][:, None] * expert(xq[rows], *experts(e))
    for s in shared:
        y += expert(xq, *s)
    return y, idx, w
