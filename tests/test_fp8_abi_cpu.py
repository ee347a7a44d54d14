"""Refusals of the 8-bit entry points on the host, before any launch."""

import ctypes

import pytest
import torch

from hybrid_linear_attention_gated_gb300 import build, hla

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = range(5)
FAKE = 0x10000  # never dereferenced: validation fails before any launch


@pytest.fixture(scope="module")
def lib():
    build.build()
    return hla.load()


def quantize(lib, **kw):
    a = dict(M=4, K=256, x=FAKE, x_dtype=hla.HLA_BF16, rows=1, q=FAKE, scale=FAKE)
    a.update(kw)
    return lib.fp8_quantize(*a.values(), None)


def matmul(lib, **kw):
    a = dict(M=4, N=256, K=256, x=FAKE, xs=FAKE, W=FAKE, ws=FAKE, residual=None, y=FAKE, y_dtype=hla.HLA_BF16)
    a.update(kw)
    return lib.fp8_matmul(*a.values(), None)


def moe(lib, M=4, ws=FAKE, n=1 << 40, x=FAKE, residual=None, y=FAKE, idx=None, w=None, L=None, null=False, **kw):
    a = dict(hidden=256, inter=128, n_experts=8, top_k=2, n_shared=1)
    a.update({k: v for k, v in kw.items() if k in a})
    L = hla.hla_moe_fp8(*a.values())
    for name, _ in hla.hla_moe_fp8._fields_[5:]:
        setattr(L, name, kw.get(name, FAKE))
    return lib.moe_fp8_forward(None if null else ctypes.byref(L), M, x, residual, y, idx, w, ws, n, None)


def test_moe_refusals(lib):
    assert moe(lib, null=True) == INVALID
    for kw in (dict(hidden=0), dict(inter=0), dict(n_experts=0), dict(top_k=0), dict(n_shared=-1), dict(top_k=9), dict(M=0), dict(x=None),
               dict(y=None), *({n: None} for n, _ in hla.hla_moe_fp8._fields_[5:])):
        assert moe(lib, **kw) == INVALID, kw
    for kw in (dict(hidden=192), dict(inter=64), dict(top_k=17, n_experts=64), dict(n_experts=1024), dict(n_shared=17), dict(M=65),
               dict(hidden=1 << 21)):
        assert moe(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(x=FAKE + 2), dict(residual=FAKE + 8), dict(y=FAKE + 2), dict(idx=FAKE + 4), dict(w=FAKE + 4), dict(ws=FAKE + 8),
               *({n: FAKE + 4} for n, _ in hla.hla_moe_fp8._fields_[5:])):
        assert moe(lib, **kw) == MISALIGNED, kw
    for kw in (dict(ws=None), dict(n=1024)):
        assert moe(lib, **kw) == WORKSPACE, kw


def test_moe_workspace(lib):
    L = hla.hla_moe_fp8(256, 128, 8, 2, 1)
    sizes = [hla.moe_fp8_forward_workspace_size(L, M) for M in (1, 2, 16, 17, 33, 64)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert [hla.moe_fp8_forward_workspace_size(L, M) for M in (0, -1, 65)] == [0, 0, 0]
    assert hla.moe_fp8_forward_workspace_size(hla.hla_moe_fp8(200, 128, 8, 2, 1), 4) == 0


def test_quantize_refusals(lib):
    for kw in (dict(M=0), dict(M=-1), dict(K=0), dict(x=None), dict(q=None), dict(scale=None), dict(x_dtype=hla.HLA_E4M3), dict(x_dtype=7)):
        assert quantize(lib, **kw) == INVALID, kw
    for kw in (dict(K=24), dict(K=250), dict(rows=0), dict(rows=2), dict(rows=64), dict(M=2**31 - 1, K=2**31 - 16, rows=128)):
        assert quantize(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(x=FAKE + 8), dict(q=FAKE + 4), dict(scale=FAKE + 4)):
        assert quantize(lib, **kw) == MISALIGNED, kw


def test_matmul_refusals(lib):
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(x=None), dict(xs=None), dict(W=None), dict(ws=None), dict(y=None),
               dict(y_dtype=hla.HLA_E4M3), dict(K=-16)):
        assert matmul(lib, **kw) == INVALID, kw
    for kw in (dict(K=40), dict(K=8), dict(M=2**31 - 1), dict(N=2**31 - 1), dict(K=2**31 - 16)):
        assert matmul(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(x=FAKE + 8), dict(xs=FAKE + 4), dict(W=FAKE + 1), dict(ws=FAKE + 8), dict(residual=FAKE + 2), dict(y=FAKE + 2)):
        assert matmul(lib, **kw) == MISALIGNED, kw


def test_binding_checks_tensors(lib):
    e4m3, bf = torch.float8_e4m3fn, torch.bfloat16
    x, q, s = torch.zeros(4, 256, dtype=bf), torch.zeros(4, 256, dtype=e4m3), torch.zeros(4, 2)
    good = dict(M=4, K=256, x=x, x_dtype=hla.HLA_BF16, rows_per_scale=1, q=q, scale=s, stream=0)
    # host tensors are on no CUDA device; types, sizes and strides are refused the same way
    for kw in (dict(), dict(x=x.float()), dict(q=q[:3]), dict(x=x.t()), dict(scale=s[:, :1])):
        with pytest.raises(hla.HlaError):
            hla.fp8_quantize(**{**good, **kw})
    with pytest.raises(hla.HlaError):
        hla.fp8_matmul(4, 4, 256, q, s, q, s[:1], None, torch.zeros(4, 4, dtype=bf), hla.HLA_BF16, stream=0)
