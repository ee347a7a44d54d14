"""Every variant of fp8_matmul by name, over what callers vary: something added or not, in place, rows that keep alignment or
not, both output types, views that are aligned to 16 bytes only, scales that are not finite, and waits that give up."""

import pytest
import torch

from hybrid_linear_attention_gated_gb300 import hla
from tests.fp8_common import matmul64, rounded, up
from tests.gpu_common import require_gpu
from tests.test_gpu_fp8 import BF, CODE, F32, product_inputs, quantize

pytestmark = pytest.mark.gpu

# variant, tokens, outputs of aligned and of unaligned rows, K; the rules that choose them count 152 SMs
VARIANTS = [
    ("fp8_matmul<tokens16,split1>", 5, 304, 301, 272),
    ("fp8_matmul<tokens16,split8>", 13, 496, 499, 2064),
    ("fp8_matmul<tokens32,split1>", 32, 304, 301, 272),
    ("fp8_matmul<tokens32,split8>", 20, 496, 499, 2064),
    ("fp8_matmul<tile128x128,split1>", 200, 6000, 6001, 272),
    ("fp8_matmul<tile128x128,split4>", 100, 496, 499, 2064),
    ("fp8_matmul<pair256x192>", 500, 7184, 7001, 528),
    ("fp8_matmul<pair256x192>", 1024, 10928, 10943, 144),   # several tiles a pair
    ("fp8_matmul<pair256x256>", 300, 9008, 9001, 528),
    ("fp8_matmul<pair256x256>", 1000, 12000, 11999, 144),
]
each_variant = pytest.mark.parametrize("variant,M,N,odd,K", VARIANTS)


def device():
    dev = require_gpu()
    if torch.cuda.get_device_properties(dev).multi_processor_count != 152:
        pytest.skip("the variants are named for 152 SMs")
    return dev


def product(variant, M, N, K, x, xs, W, ws, r, y):
    hla.fp8_matmul(M, N, K, x, xs, W, ws, r, y, CODE[y.dtype])
    assert hla.hla_last_variant() == variant
    return y


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@each_variant
def test_each_variant(variant, M, N, odd, K, dtype, residual):
    dev = device()
    for n in (N, odd):
        x, xs, W, ws, r = product_inputs(M, n, K, dev, M + n, residual)
        y = product(variant, M, n, K, x, xs, W, ws, r, torch.full((M + 1, n), 7.0, dtype=dtype, device=dev))
        want, bound = matmul64(x, xs, W, ws, r)
        assert torch.all((y[:M].double() - want).abs() <= rounded(bound, want, dtype))
        assert torch.all(y[M] == 7.0)
    assert hla.hla_device_status() == 0


@each_variant
def test_in_place(variant, M, N, odd, K):
    dev = device()
    for n in (N, odd):
        x, xs, W, ws, r = product_inputs(M, n, K, dev, M, True)
        y = product(variant, M, n, K, x, xs, W, ws, r, torch.empty_like(r))
        assert torch.equal(product(variant, M, n, K, x, xs, W, ws, r, r), y)


def view_off(t, offset=16):
    """t at an address that is 16 bytes past a multiple of 512."""
    raw = torch.zeros(t.numel() * t.element_size() + 512, dtype=torch.uint8, device=t.device)
    assert raw.data_ptr() % 512 == 0
    v = raw[offset:offset + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    v.view(torch.uint8).copy_(t.contiguous().view(torch.uint8))
    return v


@pytest.mark.parametrize("dtype", [BF, F32])
@each_variant
def test_views_aligned_to_16_bytes(variant, M, N, odd, K, dtype):
    dev = device()
    x, xs, W, ws, r = product_inputs(M, N, K, dev, M, True)
    y = product(variant, M, N, K, x, xs, W, ws, r, torch.empty(M, N, dtype=dtype, device=dev))
    z = view_off(torch.full_like(y, 7.0))
    product(variant, M, N, K, *(view_off(t) for t in (x, xs, W, ws, r)), z)
    assert torch.equal(z, y)
    z = torch.full_like(y, 7.0)   # the output alone keeps its alignment
    assert torch.equal(product(variant, M, N, K, *(view_off(t) for t in (x, xs, W, ws, r)), z), y)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_of_views_aligned_to_16_bytes(dtype, rows):
    dev = device()
    M, K = 131, 400
    x = torch.randn(M, K, device=dev).to(dtype)
    q, s = quantize(x, rows)
    q2, s2 = view_off(torch.zeros_like(q.view(torch.uint8))).view(q.dtype), view_off(torch.zeros_like(s))
    hla.fp8_quantize(M, K, view_off(x), CODE[dtype], rows, q2, s2)
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)


@each_variant
def test_scales_that_are_not_finite_stay_in_their_columns(variant, M, N, odd, K):
    dev = device()
    x, xs, W, ws, _ = product_inputs(M, odd, K, dev, 3, False)
    y = product(variant, M, odd, K, x, xs, W, ws, None, torch.empty(M, odd, device=dev))
    blocks = ws.shape[0]
    for at in sorted({0, 1, 2, blocks // 2, blocks - 1}):  # in tiles of 192 columns: either of a tile's blocks, and the border inside one
        for v in (float("nan"), float("inf")):
            ws2 = ws.clone()
            ws2[at, -1] = v
            z = product(variant, M, odd, K, x, xs, W, ws2, None, torch.empty(M, odd, device=dev))
            cols = slice(at * 128, min(odd, at * 128 + 128))
            assert not torch.any(z[:, cols].isfinite())
            z[:, cols] = y[:, cols]
            assert torch.equal(z, y)


@each_variant
def test_a_wait_that_gives_up_is_reported(variant, M, N, odd, K):
    dev = device()
    x, xs, W, ws, r = product_inputs(M, N, K, dev, M, True)
    y = torch.full((M, N), 7.0, dtype=BF, device=dev)
    torch.cuda.synchronize()
    assert hla.hla_device_status() == 0
    try:
        hla.hla_test_force_wait_timeout(1)
        product(variant, M, N, K, x, xs, W, ws, r, y)
        torch.cuda.synchronize()
    finally:
        hla.hla_test_force_wait_timeout(0)
    assert hla.hla_device_status() == 6 and hla.hla_device_status() == 0 and torch.all(y == 7.0)
    product(variant, M, N, K, x, xs, W, ws, r, y)
    want, bound = matmul64(x, xs, W, ws, r)
    assert torch.all((y.double() - want).abs() <= rounded(bound, want, BF)) and hla.hla_device_status() == 0


@pytest.mark.parametrize("variant,M,N,odd,K", VARIANTS + [
    ("fp8_matmul<tokens16,split8>", 8, 1000, 1001, 7168),
    ("fp8_matmul<tile128x128,split8>", 64, 1000, 1001, 7168),
    ("fp8_matmul<pair256x256>", 256, 16400, 16401, 7168),
])
def test_fp32_outputs_as_a_whole(variant, M, N, odd, K):
    """The norm of the error over the norm of the product.

    A block's sum is made by four instructions; each may lose a unit in the last place (2^-23) where it aligns its 32 products
    and another where it adds them to the accumulator: 4 * 2 * 2^-23 = 2^-20.  The two products of scales and the additions
    over the blocks, of a join's parts and of what is added are off by half a unit each, with either sign: the root of their
    number times 2^-24, of sums that are no larger than the result in the mean over its elements.
    """
    dev = device()
    x, xs, W, ws, _ = product_inputs(M, N, K, dev, K, False)
    y = product(variant, M, N, K, x, xs, W, ws, None, torch.empty(M, N, device=dev))
    want, _ = matmul64(x, xs, W, ws)
    rel = float((y.double() - want).norm() / want.norm())
    print(f"{variant} K {K}: rel {rel:.2e}")
    assert rel <= 2.0 ** -20 + (up(K, 128) + 11) ** 0.5 * 2.0 ** -24
