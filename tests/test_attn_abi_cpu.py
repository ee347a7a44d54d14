"""Refusals of the paged-cache entry points on the host, before any launch, and their workspace queries."""

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


def cache(**kw):
    a = dict(dtype=hla.HLA_BF16, n_pages=8, page_size=64, kv_heads=2, head_dim=128, k=FAKE, v=FAKE, k_scale=None, v_scale=None,
             k_min=FAKE, k_max=FAKE)
    a.update(kw)
    return hla.make_kv_cache(**a)


def append(lib, C, **kw):
    a = dict(N=4, B=2, cu=FAKE, past=FAKE, max_blocks=4, table=FAKE, H=8, q=FAKE, k=FAKE, v=FAKE, rope=128, inter=0, f=FAKE, out=FAKE)
    a.update(kw)
    return lib.kv_cache_append(ctypes.byref(C) if C else None, *a.values(), None)


def decode(lib, C, **kw):
    a = dict(B=2, T=1, H=8, max_blocks=4, table=FAKE, past=FAKE, scale=1.0, q=FAKE, o=FAKE, o_dtype=0, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.attn_paged_decode(ctypes.byref(C) if C else None, *a.values(), None)


def sparse(lib, C, **kw):
    a = dict(B=2, T=1, H=8, max_blocks=4, table=FAKE, past=FAKE, n_select=4, sel=FAKE, scale=1.0, q=FAKE, o=FAKE, o_dtype=0, ws=FAKE,
             n=1 << 40)
    a.update(kw)
    return lib.attn_paged_sparse(ctypes.byref(C) if C else None, *a.values(), None)


def select(lib, C, **kw):
    a = dict(B=2, T=1, H=8, max_blocks=4, table=FAKE, past=FAKE, n_select=4, n_first=0, n_last=1, q=FAKE, sel=FAKE, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.attn_select_blocks(ctypes.byref(C) if C else None, *a.values(), None)


@pytest.mark.parametrize("call", [append, decode, sparse, select])
def test_descriptor_is_checked(lib, call):
    assert call(lib, None) == INVALID
    for kw in (dict(n_pages=0), dict(page_size=0), dict(kv_heads=0), dict(head_dim=0), dict(dtype=9), dict(k_min=None),
               dict(k_max=None)):
        assert call(lib, cache(**kw)) == INVALID, kw
    for kw in (dict(page_size=48), dict(page_size=8), dict(page_size=256), dict(head_dim=96), dict(head_dim=256), dict(kv_heads=257), dict(dtype=hla.HLA_F32)):
        assert call(lib, cache(**kw)) == UNSUPPORTED, kw
    assert call(lib, cache(k_min=FAKE + 2)) == MISALIGNED
    if call is select:
        assert call(lib, cache(k_min=None, k_max=None)) == INVALID
    else:
        for kw in (dict(k=None), dict(v=None), dict(dtype=hla.HLA_E4M3), dict(dtype=hla.HLA_E4M3, k_scale=FAKE)):
            assert call(lib, cache(**kw)) == INVALID, kw
        assert call(lib, cache(k=FAKE + 8)) == MISALIGNED
        assert call(lib, cache(dtype=hla.HLA_E4M3, k_scale=FAKE, v_scale=FAKE + 4)) == MISALIGNED


@pytest.mark.parametrize("call", [decode, sparse, select])
def test_window_sizes_are_checked(lib, call):
    C = cache()
    for kw in (dict(B=0), dict(T=0), dict(H=0), dict(H=7), dict(max_blocks=0), dict(table=None), dict(past=None), dict(q=None)):
        assert call(lib, C, **kw) == INVALID, kw
    for kw in (dict(B=1025), dict(T=9), dict(H=1026), dict(max_blocks=1 << 25)):
        assert call(lib, C, **kw) == UNSUPPORTED, kw
    for kw in (dict(table=FAKE + 4), dict(past=FAKE + 8), dict(q=FAKE + 2), dict(ws=FAKE + 8)):
        assert call(lib, C, **kw) == MISALIGNED, kw
    for kw in (dict(ws=None), dict(n=16)):
        assert call(lib, C, **kw) == WORKSPACE, kw


def test_own_arguments_are_checked(lib):
    C = cache()
    for call in (decode, sparse):
        for kw in (dict(o=None), dict(o_dtype=2), dict(o_dtype=-1), dict(scale=float("nan")), dict(scale=float("inf"))):
            assert call(lib, C, **kw) == INVALID, kw
        assert call(lib, C, o=FAKE + 4) == MISALIGNED
    for kw in (dict(sel=None), dict(n_select=0)):
        assert sparse(lib, C, **kw) == INVALID
    assert sparse(lib, C, n_select=1 << 24) == UNSUPPORTED
    assert sparse(lib, C, sel=FAKE + 4) == MISALIGNED
    for kw in (dict(sel=None), dict(n_select=0), dict(n_first=-1), dict(n_last=-1), dict(n_first=4), dict(n_first=5, n_last=0),
               dict(n_first=2 ** 31 - 1, n_last=2 ** 31 - 1)):
        assert select(lib, C, **kw) == INVALID, kw
    assert select(lib, C, max_blocks=65537) == UNSUPPORTED
    for kw in (dict(N=0), dict(B=0), dict(H=9), dict(cu=None), dict(out=None), dict(k=None), dict(v=None), dict(f=None), dict(rope=-16),
               dict(inter=2)):
        assert append(lib, C, **kw) == INVALID, kw
    for kw in (dict(rope=144), dict(rope=24), dict(B=2000)):
        assert append(lib, C, **kw) == UNSUPPORTED, kw
    for kw in (dict(cu=FAKE + 4), dict(k=FAKE + 2), dict(out=FAKE + 8), dict(f=FAKE + 8)):
        assert append(lib, C, **kw) == MISALIGNED, kw


def test_workspace_queries(lib):
    C = cache()
    assert 0 < hla.attn_paged_decode_workspace_size(C, 1, 1, 8) < hla.attn_paged_decode_workspace_size(C, 1, 8, 32)
    assert hla.attn_paged_sparse_workspace_size(C, 4, 2, 8) > 0
    assert hla.attn_select_blocks_workspace_size(C, 2, 1, 8, 100) < hla.attn_select_blocks_workspace_size(C, 2, 2, 8, 100)
    for bad in ((0, 1, 8), (1, 9, 8), (1, 1, 7)):
        assert hla.attn_paged_decode_workspace_size(C, *bad) == 0
        assert hla.attn_paged_sparse_workspace_size(C, *bad) == 0
        assert hla.attn_select_blocks_workspace_size(C, *bad, 4) == 0


def test_binding_refuses_tensors_a_kernel_would_misread(lib):
    """Host tensors, wrong types, short and strided ones never reach the library."""
    with pytest.raises(hla.HlaError) as e:
        hla.make_kv_cache(hla.HLA_BF16, 2, 16, 1, 64, torch.zeros(2, 1, 16, 64), FAKE)  # fp32
    assert e.value.status == INVALID and "k must be" in str(e.value)
    with pytest.raises(hla.HlaError):
        hla.make_kv_cache(hla.HLA_BF16, 2, 16, 1, 64, FAKE, torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16))  # too few pages
    C = cache()
    table = torch.zeros(2, 4, dtype=torch.int64)
    with pytest.raises(hla.HlaError):
        hla.attn_paged_decode(C, 2, 1, 8, 4, table, FAKE, 1.0, FAKE, FAKE, 0, FAKE, 1 << 40, stream=0)
    if torch.cuda.is_available():
        with pytest.raises(hla.HlaError):
            hla.attn_paged_decode(C, 2, 1, 8, 4, table.int(), FAKE, 1.0, FAKE, FAKE, 0, FAKE, 1 << 40, stream=0)  # a host tensor


def test_binding_refuses_a_cache_of_another_device(lib):
    """The descriptor's tensors are on the device that was current when it was made."""
    C = cache()
    assert C.device is None
    C.device = 5
    for call in (lambda: hla.kv_cache_append(C, 1, 1, FAKE, FAKE, 4, FAKE, 8, FAKE, FAKE, FAKE, 0, 0, None, FAKE, stream=0),
                 lambda: hla.attn_paged_decode(C, 1, 1, 8, 4, FAKE, FAKE, 1.0, FAKE, FAKE, 0, FAKE, 1 << 40, stream=0),
                 lambda: hla.attn_select_blocks(C, 1, 1, 8, 4, FAKE, FAKE, 2, 0, 0, FAKE, FAKE, FAKE, 1 << 40, stream=0),
                 lambda: hla.attn_paged_sparse(C, 1, 1, 8, 4, FAKE, FAKE, 2, FAKE, 1.0, FAKE, FAKE, 0, FAKE, 1 << 40, stream=0)):
        with pytest.raises(hla.HlaError) as e:
            call()
        assert e.value.status == INVALID and "device 5" in str(e.value)
