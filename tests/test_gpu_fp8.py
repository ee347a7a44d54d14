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


# ----------------------------------------------------------------------------- the calls that programs make


def test_matmul_into_its_residual():
    dev = require_gpu()
    for M, N, K in ((5, 300, 272), (70, 300, 272), (600, 7200, 144)):
        x, xs, W, ws, r = product_inputs(M, N, K, dev, M, True)
        y = torch.empty(M, N, dtype=BF, device=dev)
        hla.fp8_matmul(M, N, K, x, xs, W, ws, r, y, hla.HLA_BF16)
        hla.fp8_matmul(M, N, K, x, xs, W, ws, r, r, hla.HLA_BF16)
        assert torch.equal(y, r)


@pytest.mark.parametrize("M,N,K", [(3, 300, 400), (20, 1000, 2048), (100, 500, 1040), (300, 9000, 528), (1000, 12000, 144)])
def test_nan_and_infinity_stay_in_their_rows_and_columns(M, N, K):
    dev = require_gpu()
    x, xs, W, ws, _ = product_inputs(M, N, K, dev, 3, False)
    y = torch.empty(M, N, device=dev)
    hla.fp8_matmul(M, N, K, x, xs, W, ws, None, y, hla.HLA_F32)
    x2, W2, xs2 = x.clone(), W.clone(), xs.clone()
    x2.view(torch.uint8)[1, 5] = 0x7F                  # NaN in token 1
    W2.view(torch.uint8)[N - 2, K - 1] = 0x7F          # and in weight row N - 2
    xs2[2, 0] = float("inf")                           # token 2: inf or NaN, as the sum of its first block is signed or 0
    z = torch.empty(M, N, device=dev)
    hla.fp8_matmul(M, N, K, x2, xs2, W2, ws, None, z, hla.HLA_F32)
    assert torch.all(z[1].isnan()) and torch.all(z[:, N - 2].isnan())
    assert not torch.any(z[2].isfinite())
    rows = [m for m in range(M) if m not in (1, 2)]
    cols = [n for n in range(N) if n != N - 2]
    assert torch.equal(z[rows][:, cols], y[rows][:, cols])


def test_matmul_wait_timeout_is_reported():
    dev = require_gpu()
    for M, N, K in ((4, 300, 272), (100, 300, 272), (600, 9000, 144)):
        x, xs, W, ws, _ = product_inputs(M, N, K, dev, M, False)
        y = torch.full((M, N), 7.0, device=dev)
        torch.cuda.synchronize()
        assert hla.hla_device_status() == 0
        try:
            hla.hla_test_force_wait_timeout(1)
            hla.fp8_matmul(M, N, K, x, xs, W, ws, None, y, hla.HLA_F32)
            torch.cuda.synchronize()
        finally:
            hla.hla_test_force_wait_timeout(0)
        assert hla.hla_device_status() == 6 and hla.hla_device_status() == 0 and torch.all(y == 7.0)
        check_product(M, N, K, F32, False, dev, M)


def test_graph_stream_and_chain_give_the_same_bits():
    dev = require_gpu()
    M, N, K = 48, 1500, 1040
    g = generator(dev, 9)
    a = torch.randn(M, K, generator=g, device=dev).to(BF)
    W, ws = e4m3_weights(N, K, g, dev)
    q, s = torch.empty(M, K, dtype=E4M3, device=dev), torch.empty(M, up(K, 128), device=dev)
    y = torch.empty(M, N, dtype=BF, device=dev)

    def step():
        hla.fp8_quantize(M, K, a, hla.HLA_BF16, 1, q, s)
        hla.fp8_matmul(M, N, K, q, s, W, ws, None, y, hla.HLA_BF16)

    step()
    want = y.clone()
    # another stream, in a launch chain
    st = torch.cuda.Stream()
    y.fill_(7)
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        hla.hla_chain_begin()
        step()
        step()
        hla.hla_chain_end()
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(y, want)
    # a graph, replayed on other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    a.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want.neg())


def test_offsets_beyond_32_bits():
    dev = require_gpu()
    M, N, K = 139000, 16001, 16          # 2.2e9 outputs, rows that keep no alignment
    x, xs, W, ws, _ = product_inputs(M, N, K, dev, 5, False)
    y = torch.empty(M, N, dtype=BF, device=dev)
    hla.fp8_matmul(M, N, K, x, xs, W, ws, None, y, hla.HLA_BF16)
    for rows in (slice(0, 70), slice(134100, 134300), slice(M - 70, M)):
        want, bound = matmul64(x[rows], xs[rows], W, ws)
        assert torch.all((y[rows].double() - want).abs() <= rounded(bound, want, BF))
    del y
    M, K = 300000, 7168                  # 2.15e9 values
    a = torch.randn(M, K, dtype=BF, device=dev)
    for per in (1, 128):
        q, s = quantize(a, per)
        for r0 in (0, 299520, 299904):
            want_q, want_s = quantize(a[r0:r0 + 96].contiguous(), per)
            if per == 1 or r0 == 299904:  # the last block of 128 rows has 96
                assert torch.equal(q[r0:r0 + 96].view(torch.uint8), want_q.view(torch.uint8))
                assert torch.equal(s[r0 // per:r0 // per + want_s.shape[0]], want_s)


def test_random_sizes():
    dev = require_gpu()
    rng = np.random.default_rng(11)
    for i in range(40):
        M, N = (int(round(np.exp(rng.uniform(0, np.log(top))))) for top in (3000, 6000))
        K = 16 * int(round(np.exp(rng.uniform(0, np.log(200)))))
        check_product(M, N, K, F32 if i % 2 else BF, i % 3 == 0, dev, i)
