"""The fp64 oracle of the 8-bit operators, pinned by hand-worked values, scalar loops and invariants."""

import math

import numpy as np

import oracle
from oracle import fp8


def test_scales_are_the_least_power_of_two():
    assert fp8.block_scale(448.0) == 1.0 and fp8.block_scale(448.0001) == 2.0 and fp8.block_scale(224.0) == 0.5
    assert fp8.block_scale(1.75) == 2.0 ** -8 and fp8.block_scale(0.0) == 2.0 ** -126 and fp8.block_scale(1e-45) == 2.0 ** -126
    assert math.isnan(fp8.block_scale(math.inf)) and math.isnan(fp8.block_scale(math.nan))


def test_quantize_by_hand():
    x = np.zeros((3, 160))
    x[0, :4] = [896.0, 17.0, 34.0, -38.0]     # scale 2: 448, 8.5 (to the even 8), 17 -> 16, -19 -> -20
    x[1, 130] = 3.0                           # second block, 32 columns wide: 3 * 2^7 = 384 <= 448 < 768
    x[2, 0] = np.inf
    q, s = fp8.quantize(x)
    assert s[0].tolist() == [2.0, 2.0 ** -126] and q[0, :4].tolist() == [448.0, 8.0, 16.0, -20.0]
    assert s[1, 1] == 2.0 ** -7 and q[1, 130] == 384.0
    assert np.isnan(s[2, 0]) and np.all(np.isnan(q[2, :128])) and np.all(q[2, 128:] == 0)
    q, s = fp8.quantize(x[:2], 128)           # one block of two rows
    assert s.tolist() == [[2.0, 2.0 ** -7]] and q[0, 0] == 448.0
    g = np.random.default_rng(0)
    x = g.normal(size=(5, 300))
    q, s = fp8.quantize(x)
    back = fp8.values(q, s)
    # half a step of 3 mantissa bits, or of the smallest step 2^-9 of the scale
    assert np.all(np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(s, 128, 1)[:, :300] * 2.0 ** -10))
    again = fp8.quantize(back)
    assert np.array_equal(again[0] * np.repeat(again[1], 128, 1)[:, :300], back)


def test_matmul_by_scalar_loops():
    g = np.random.default_rng(1)
    M, N, K = 3, 140, 200
    x, W = g.normal(size=(M, K)), g.normal(size=(N, K))
    xs, ws, r = g.normal(size=(M, 2)), g.normal(size=(2, 2)), g.normal(size=(M, N))
    y = fp8.matmul(x, xs, W, ws, r)
    for m, n in ((0, 0), (1, 127), (2, 128), (2, 139)):
        want = r[m, n]
        for k in range(K):
            want += x[m, k] * xs[m, k // 128] * W[n, k] * ws[n // 128, k // 128]
        assert math.isclose(y[m, n], want, rel_tol=1e-10, abs_tol=1e-10)


def test_moe_layer_is_the_unconverted_layer_on_values_that_convert_exactly():
    g = np.random.default_rng(2)
    M, Hd, I, E, k = 4, 128, 128, 6, 2
    x = g.integers(-3, 4, size=(M, Hd)).astype(float)          # e4m3 holds these over any power of two
    W_r = g.normal(size=(E, Hd))
    gate, up = np.zeros((E + 1, I, Hd)), np.zeros((E + 1, I, Hd))
    down = g.normal(size=(E + 1, Hd, I))
    gate[:, :, 0] = 1000.0  # SiLU(+-1000 n) is 1000 n or 0, so h is a small whole multiple of 1000 * 2^j
    x[:, 0] = 1.0
    up[:, :, 1] = 1.0
    y, idx, w = fp8.moe_layer(x, W_r, k, lambda e: (gate[e], up[e], down[e]), [(gate[E], up[E], down[E])], x)
    assert np.array_equal(fp8.values(*fp8.quantize(x)), x)
    want_idx, want_w, _ = oracle.moe.route_topk(x, W_r, k)
    # 1000 = 2^3 * 125 takes 7 mantissa bits: h = 1000 x[1] is rounded; the reference layer gets the rounded gate
    held = {v: float(fp8.values(*fp8.quantize(np.full((1, 128), 1000.0 * v)))[0, 0]) for v in range(-3, 4)}
    for m in range(M):
        h = np.full(I, held[int(x[m, 1])])
        want = x[m] + down[E] @ h + sum(want_w[m, j] * (down[want_idx[m, j]] @ h) for j in range(k))
        assert np.allclose(y[m], want, rtol=1e-12)
    assert np.array_equal(idx, want_idx) and np.array_equal(w, want_w)
