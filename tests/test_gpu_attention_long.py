"""Paged attention with enough cached tokens that every CTA runs tens of tiles of a unit: the running maximum and sums over a
long piece, the copy ring's reuse, the page look-ahead and the pieces' join, against fp64 on the GPU."""

import numpy as np
import pytest
import torch

from hybrid_linear_attention_gated_gb300 import hla, inputs
from tests.attn_common import BF16, FP8, I32, Problem, attention_tolerance
from tests.gpu_common import require_gpu

pytestmark = pytest.mark.gpu

BF, E4 = hla.HLA_BF16, hla.HLA_E4M3


def long_problem(T, H, Hkv, d, dtype, B, n, seed):
    """B sequences of about n tokens on the same pages.  Along the sequence the keys grow in one channel, and a query row's
    value in that channel is 0, +-1/4, +-1/2 or +-1 of the largest: some rows of a warp meet a maximum that rises hundreds of
    powers of two over the sequence, others one that stays or that came first."""
    p = Problem(require_gpu(), [n], T, H, Hkv, d, 64, dtype, seed=seed, poison=False)
    at = torch.zeros(p.n_pages, 64)
    at[p.table[0].long()] = torch.arange(p.max_blocks * 64).view(-1, 64) / n
    ramp, top = (640.0, 4.0) if dtype == BF else (448.0, 64.0)
    p.k[..., d - 1] = (ramp * at)[:, None].expand(-1, Hkv, -1).to(p.k.dtype)
    p.B, p.past = B, [n - (37 * b) % 1000 for b in range(B)]
    p.past[B // 2] = -1
    p.table = p.table.repeat(B, 1)
    p.q = torch.randn((B, T, H, d), generator=inputs.generator(seed + 1)).to(BF16)
    steps = torch.tensor([0.0, 0.25, 0.5, 1.0, -0.25, -0.5, -1.0, 1.0])
    p.q[..., d - 1] = top * steps[torch.randint(0, 8, (B, T, H), generator=inputs.generator(seed + 2))]
    return p


def reference(p, sel=None):
    """o, the same sums over |v|, and the largest |score|, in fp64 from the definition."""
    B, T, H, Hkv, d, P, dev = p.B, p.T, p.H, p.Hkv, p.d, p.page, p.dev
    pages = p.table[0].long().to(dev)
    as_values = lambda x, s: x.to(dev).double()[pages] * (1.0 if s is None else s.to(dev).double()[:, None, None])  # noqa: E731
    k, v = as_values(p.k, p.k_scale), as_values(p.v, p.v_scale)  # [blocks, Hkv, P, d]
    q = p.q.to(dev).double().view(B, T, Hkv, H // Hkv, d)
    o, mag, top = torch.zeros_like(q), torch.zeros_like(q), 0.0
    for b in range(B):
        if p.past[b] < 0:
            continue
        for h in range(Hkv):
            for t in [None] if sel is None else range(T):  # a list is a token's own
                blocks = torch.arange(p.max_blocks, device=dev) if t is None else sel[b, t, h].to(dev).long()
                pos = (blocks[:, None] * P + torch.arange(P, device=dev)).flatten()
                rows = q[b, :, h] if t is None else q[b, t:t + 1, h]
                seen = pos[None] <= p.past[b] + (torch.arange(T, device=dev)[:, None] if t is None else t)  # [T or 1, keys]
                s = p.scale * rows @ k[blocks, h].reshape(-1, d).T
                top = max(top, s.abs().max().item())
                w = torch.softmax(s.masked_fill(~seen[:, None], -torch.inf), -1)
                x = v[blocks, h].reshape(-1, d)
                if t is None:
                    o[b, :, h], mag[b, :, h] = w @ x, w @ x.abs()
                else:
                    o[b, t, h], mag[b, t, h] = (w @ x)[0], (w @ x.abs())[0]
    return [x.view(B, T, H, d).cpu().numpy() for x in (o, mag)] + [top]


def check_long(p, o_dtype, n_keys, sel=None):
    o = p.decode(o_dtype, None if sel is None else sel.to(p.dev)).double().cpu().numpy()
    ref, mag, top = reference(p, sel)
    assert np.all(np.isfinite(o)) and np.all(o[p.past.index(-1)] == 0)
    # (the terms of a score add up to no more than the ramp's, which is the score, and those of 127 normal products)
    size = top + p.scale * 127 * 6 * 6
    assert np.all(np.abs(o - ref) <= attention_tolerance(ref, mag, n_keys, p.d, size, o_dtype, p.dtype))
    # On average far closer: the output's rounding (a bf16 weight's is as large), and fp32 scores, which d / 16 products add up
    # with an error of 2^-23 of the sum each
    rel = np.linalg.norm(o - ref) / np.linalg.norm(ref)
    assert rel < (2.0 ** -8 if o_dtype == BF else 2e-5) + 2 * p.d / 16 * 2.0 ** -23 * top, rel


def tiles_per_cta(p, rows, o_dtype, keys):
    """Tiles of 64 or 128 keys that a CTA gets of all units' `keys` keys."""
    sms = torch.cuda.get_device_properties(p.dev).multi_processor_count
    tc = rows > 64 and p.dtype == BF and o_dtype == BF
    tile = 64 if tc or (p.d == 128 and p.dtype == BF) else 128
    row_tiles = 1 if tc else -(-rows // 64)
    return keys * p.Hkv * row_tiles / tile / ((2 if p.d == 128 else 3) * sms)


@pytest.mark.parametrize("T,H,d,dtype,o_dtype", [
    (1, 16, 128, BF, BF), (4, 4, 128, E4, hla.HLA_F32), (2, 8, 64, BF, hla.HLA_F32), (1, 16, 64, E4, BF),   # 16 rows
    (4, 8, 128, E4, BF), (4, 8, 64, BF, hla.HLA_F32), (2, 16, 128, BF, BF),                                 # 32
    (8, 8, 128, BF, hla.HLA_F32), (4, 16, 64, E4, BF), (4, 16, 128, BF, BF),                                # 64
    (8, 9, 128, E4, hla.HLA_F32),                                                                           # two tiles of 64
    (8, 9, 128, BF, BF), (8, 16, 64, BF, BF),                                                               # tcgen05
])
def test_decode_over_many_tiles(T, H, d, dtype, o_dtype):
    B, n = 128, 19500 if d == 64 else 13500
    p = long_problem(T, H, 1, d, dtype, B, n, seed=30).upload()
    assert tiles_per_cta(p, T * H, o_dtype, sum(x + T for x in p.past if x >= 0)) > 40
    check_long(p, o_dtype, n + T)


@pytest.mark.parametrize("H,Hkv,d,dtype,o_dtype", [(16, 2, 128, BF, BF), (32, 1, 64, E4, hla.HLA_F32), (64, 1, 128, BF, hla.HLA_F32),
                                                   (72, 1, 64, BF, BF), (128, 1, 128, BF, BF)])
def test_sparse_over_many_tiles(H, Hkv, d, dtype, o_dtype):
    """Long lists in random order, each of its own."""
    B, T, n, listed = 96, 2, 18000, 260
    p = long_problem(T, H, Hkv, d, dtype, B, n, seed=31).upload()
    g = inputs.generator(32)
    newest = torch.tensor([max(x, 0) for x in p.past]) // 64  # (visible to every token of the window)
    key = torch.rand((B, T, Hkv, p.max_blocks), generator=g)
    key[torch.arange(p.max_blocks) > newest[:, None, None, None].expand(-1, T, Hkv, 1)] = -1
    sel = key.topk(listed, -1).indices.to(I32)
    sel[p.past.index(-1)] = 0
    assert tiles_per_cta(p, H // Hkv, o_dtype, (B - 1) * T * listed * 64) > 40
    check_long(p, o_dtype, listed * 64, sel)
