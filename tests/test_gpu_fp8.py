"""fp8_quantize and fp8_matmul on the GPU: against the fp64 oracle, bit for bit where nothing but the rounding to e4m3 is
involved, within the bounds of fp32 sums otherwise."""

import numpy as np
import pytest
import torch

import oracle
from hybrid_linear_attention_gated_gb300 import hla
from tests.fp8_common import e4m3_weights, generator, matmul64, rounded, up
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
CODE = {BF: hla.HLA_BF16, F32: hla.HLA_F32}
E4M3 = torch.float8_e4m3fn


def quantize(x, rows):
    M, K = x.shape
    q = torch.empty(M, K, dtype=E4M3, device=x.device)
    s = torch.empty(up(M, rows), up(K, 128), device=x.device)
    hla.fp8_quantize(M, K, x, CODE[x.dtype], rows, q, s)
    return q, s


# ----------------------------------------------------------------------------- conversion


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (7, 4112), (130, 400), (257, 1040), (64, 7168)])
def test_quantize_bit_for_bit(M, K, dtype, rows):
    dev = require_gpu()
    g = generator(dev, M * 1000 + K)
    x = (torch.randn(M, K, generator=g, device=dev) * torch.exp(3 * torch.randn(M, K, generator=g, device=dev))).to(dtype)
    x[0, 0] = 1.75 * 2.0 ** 5   # the largest value that scale 2^-3 holds, often the block's largest
    q, s = quantize(x, rows)
    want_q, want_s = oracle.fp8.quantize(x.double().cpu().numpy(), rows)
    assert np.array_equal(s.double().cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().double().numpy(), want_q)


def test_quantize_extremes():
    dev = require_gpu()
    x = torch.zeros(8, 256, device=dev)
    x[1, 5] = 1e-45                       # the smallest fp32 subnormal
    x[2, 7] = torch.finfo(F32).max
    x[3, 9] = float("inf")
    x[4, 11] = float("nan")
    x[5, 3], x[5, 130] = -float("inf"), 2.0
    x[6, :] = 448.0 * 2.0 ** -126
    x[7, :] = torch.tensor([1.75, 1.7500001], device=dev).repeat(128)
    x[0, 0] = -0.0
    for rows in (1, 128):
        q, s = quantize(x, rows)
        want_q, want_s = oracle.fp8.quantize(x.double().cpu().numpy(), rows)
        assert np.array_equal(s.double().cpu().numpy(), want_s, equal_nan=True)
        assert np.array_equal(q.cpu().double().numpy(), want_q, equal_nan=True)


def test_quantize_leaves_its_neighbours():
    dev = require_gpu()
    M, K = 131, 272
    x = torch.randn(M, K, device=dev)
    for rows in (1, 128):
        q = torch.full((M * K + 64,), 7, dtype=torch.uint8, device=dev)
        s = torch.full((up(M, rows) * 3 + 16,), 7.0, device=dev)
        hla.fp8_quantize(M, K, x, hla.HLA_F32, rows, q.view(E4M3), s)
        assert torch.all(q[M * K:] == 7) and torch.all(s[up(M, rows) * 3:] == 7.0)


# ----------------------------------------------------------------------------- product


def product_inputs(M, N, K, dev, seed, residual):
    g = generator(dev, seed)
    x, xs = e4m3_weights(M, K, g, dev, 60.0)
    xs = (torch.rand(M, up(K, 128), generator=g, device=dev) + 0.5) / 60.0
    W, ws = e4m3_weights(N, K, g, dev)
    r = torch.randn(M, N, generator=g, device=dev).to(BF) if residual else None
    return x, xs, W, ws, r


def check_product(M, N, K, dtype, residual, dev, seed):
    x, xs, W, ws, r = product_inputs(M, N, K, dev, seed, residual)
    y = torch.full((M * N + 32,), 7.0, dtype=dtype, device=dev)
    hla.fp8_matmul(M, N, K, x, xs, W, ws, r, y, CODE[dtype])
    torch.cuda.synchronize()
    assert hla.hla_device_status() == 0
    want, bound = matmul64(x, xs, W, ws, r)
    err = (y[:M * N].view(M, N).double() - want).abs()
    worst = (err / rounded(bound, want, dtype)).max().item()
    print(f"{hla.hla_last_variant()} M {M} N {N} K {K}: {worst:.3f} of the bound, rel {float(err.norm() / want.norm()):.2e}")
    assert worst <= 1.0
    assert torch.all(y[M * N:] == 7.0)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 63, 64])
@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (130, 144), (1000, 1040), (384, 4112)])
def test_matmul_few_tokens(M, N, K):
    dev = require_gpu()
    check_product(M, N, K, F32 if (M + N) % 2 else BF, M % 3 == 0, dev, M + N + K)


@pytest.mark.parametrize("M,N,K", [(65, 1, 16), (128, 128, 128), (129, 130, 144), (200, 1000, 1040), (333, 701, 4112), (257, 4097, 512),
                                   (1000, 127, 2048), (2049, 2500, 272), (4096, 5000, 640)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_matmul_more_tokens(M, N, K, dtype):
    dev = require_gpu()
    check_product(M, N, K, dtype, N % 2 == 1, dev, M + N + K)


@pytest.mark.parametrize("M", [1, 16, 64, 256])
def test_matmul_of_the_projections(M):
    dev = require_gpu()
    check_product(M, 16416, 7168, BF, False, dev, M)
    check_product(M, 7168, 4096, BF, True, dev, M)
