"""moe_fp8_forward on the GPU: against its fp64 definition over sizes, batches and routings, and the calls that a program
makes of it (graphs, streams, workspaces, chains), alone and with the other 8-bit operators."""

import numpy as np
import pytest
import torch

import oracle
from hybrid_linear_attention_gated_gb300 import hla
from tests.fp8_common import Moe, rounded, up, values64
from tests.gpu_common import MOE_FROB_REL, require_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HLA_ERR_DEVICE_TIMEOUT = 6


def check(layer, x, residual=None, got=None):
    y, idx, w = got or layer.run(x, residual)
    torch.cuda.synchronize()
    assert hla.hla_device_status() == 0
    want, bound, want_idx, want_w = layer.reference(x, residual)
    assert torch.equal(idx.long(), want_idx)
    assert torch.all((w.double() - want_w).abs() <= 2e-6 * want_w)   # logits of fp32 sums, exp, three roundings
    err = (y.double() - want).abs()
    worst = (err / rounded(bound, want, BF)).max().item()
    rel = float(err.norm() / want.norm())
    print(f"{hla.hla_last_variant()} M {x.shape[0]} Hd {layer.Hd} I {layer.I} E {layer.E} k {layer.k}+{layer.shared}: {worst:.3f} of the bound, rel {rel:.2e}")
    assert worst <= 1.0 and rel < MOE_FROB_REL


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("Hd,I,E,k,shared", [(128, 128, 1, 1, 0), (256, 128, 16, 2, 0), (384, 256, 5, 3, 1), (1024, 384, 60, 8, 2)])
def test_sizes(M, Hd, I, E, k, shared):
    dev = require_gpu()
    layer = Moe(hla, dev, Hd, I, E, k, shared, seed=Hd + I + E)
    x = layer.tokens(M, M)
    residual = torch.randn(M, Hd, device=dev, generator=torch.Generator(dev).manual_seed(M)).to(BF) if (M + E) % 2 else None
    check(layer, x, residual)


@pytest.mark.parametrize("E,k,shared", [(300, 16, 1), (1008, 4, 16), (257, 1, 0)])
def test_many_experts(E, k, shared):
    dev = require_gpu()
    layer = Moe(hla, dev, 256, 128, E, k, shared, seed=E)
    for M in (1, 24, 64):
        check(layer, layer.tokens(M, M))
