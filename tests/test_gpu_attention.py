"""Paged attention of the newest tokens, dense and over listed blocks, against the fp64 oracle."""

import numpy as np
import pytest
import torch

import oracle
from hybrid_linear_attention_gated_gb300 import hla, inputs
from tests.attn_common import BF16, I32, Problem, attention_tolerance, bits
from tests.gpu_common import f64, require_gpu

pytestmark = pytest.mark.gpu


def check(p, o, o_dtype, sel=None):
    k, v = p.values()
    q = p.q.double().numpy()
    table = p.table.numpy()
    ref, mag = oracle.attention.attend(q, k, v, table, p.past, p.scale, sel)
    n = max([x + p.T for x in p.past] + [1]) if sel is None else sel.shape[-1] * p.page
    size = p.scale * np.abs(q).sum(-1).max() * np.nanmax(np.abs(np.where(np.isfinite(k), k, 0.0)))
    tol = attention_tolerance(ref, mag, n, p.d, size, o_dtype, p.dtype)
    got = f64(o)
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - ref) - tol)
    assert worst <= 0, worst
    # and far closer on average than the elementwise bound: rounding of the output, or fp32
    rel = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    assert rel < (2.0 ** -8 if o_dtype == hla.HLA_BF16 else 2e-5), rel
    return ref


# (past per sequence, T, H, Hkv, d, page): 16-, 32- and 64-row tiles, one key, page and tile borders, idle slots
CASES = [
    ([0], 1, 1, 1, 64, 16),
    ([0, 1, 15, 16, 17, -1], 1, 8, 2, 128, 16),
    ([62, 63, 64, 65, 127, 128], 1, 32, 8, 128, 64),
    ([300, -1, 5, 1021], 4, 16, 4, 128, 32),        # 16 rows
    ([97, 2000], 5, 10, 2, 128, 128),               # 25 rows
    ([31, 500, 0], 8, 16, 4, 64, 64),               # 32 rows
    ([700, 12], 8, 16, 1, 128, 16),                 # 128 rows: two tiles of 64
    ([130, 64, -1], 3, 24, 1, 64, 32),              # 72 rows: a full tile and a ragged one
    ([4093], 2, 6, 2, 128, 64),
    ([-1, -1], 2, 4, 2, 64, 16),
]


@pytest.mark.parametrize("o_dtype", [hla.HLA_BF16, hla.HLA_F32])
@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_decode_matches_oracle(case, dtype, o_dtype):
    past, T, H, Hkv, d, page = CASES[case]
    p = Problem(require_gpu(), past, T, H, Hkv, d, page, dtype, seed=case).upload()
    o = p.decode(o_dtype)
    rows = T * H // Hkv
    m = 16 if rows <= 16 else 32 if rows <= 32 else 64
    if rows > 64 and dtype == hla.HLA_BF16 and o_dtype == hla.HLA_BF16:
        m = 128  # tcgen05
    assert hla.hla_last_variant() == f"attn_paged<d{d},{'e4m3' if dtype == hla.HLA_E4M3 else 'bf16'},m{m}>"
    torch.cuda.synchronize()
    check(p, o, o_dtype)
    again = p.decode(o_dtype)
    assert torch.equal(bits(again), bits(o))  # fixed order of all sums


@pytest.mark.parametrize("T,H,Hkv", [(1, 8, 2), (4, 16, 2), (8, 8, 1), (8, 24, 2)])
def test_many_ragged_sequences(T, H, Hkv):
    """More units than CTAs and fewer, with pieces joined across CTAs: every sequence against the oracle."""
    g = np.random.default_rng(5)
    past = [int(x) for x in g.integers(-1, 700, size=70)]
    p = Problem(require_gpu(), past, T, H, Hkv, 64, 32, seed=9).upload()
    for o_dtype in (hla.HLA_F32, hla.HLA_BF16):
        check(p, p.decode(o_dtype), o_dtype)


@pytest.mark.parametrize("d,T,H,Hkv,page", [(128, 8, 9, 1, 64), (64, 8, 32, 1, 16), (128, 5, 40, 2, 128), (64, 3, 24, 1, 32)])
def test_tcgen05_rows_over_lengths(d, T, H, Hkv, page):
    """More than 64 rows of a bf16 cache: lengths around the 64-key tiles, windows across page and tile borders, negative
    scale, pieces joined across CTAs, and the status word stays clear."""
    dev = require_gpu()
    past = [0, 1, 120, 121, 126, 127, 128, 129, 255, 256, 511, 3000, -1, 900]
    p = Problem(dev, past, T, H, Hkv, d, page, seed=d + T).upload()
    for scale in (p.scale, -0.05, 0.7):
        p.scale = scale
        o = p.decode(hla.HLA_BF16)
        assert hla.hla_last_variant().endswith("m128>")
        torch.cuda.synchronize()
        assert hla.hla_device_status() == 0
        check(p, o, hla.HLA_BF16)
        assert torch.equal(bits(o), bits(p.decode(hla.HLA_BF16)))


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
def test_large_scores_and_flat_scores(dtype):
    """Scores of hundreds (one key takes all) and of zero (all keys alike)."""
    dev = require_gpu()
    for scale in (8.0, 0.0, -1.0):
        p = Problem(dev, [513, 64], 2, 8, 2, 128, 64, dtype, seed=3).upload()
        p.scale = scale
        k, v = p.values()
        ref, mag = oracle.attention.attend(p.q.double().numpy(), k, v, p.table.numpy(), p.past, scale)
        got = f64(p.decode(hla.HLA_F32))
        # a score's error is d 2^-23 of its terms' magnitudes: about 128 x 2^-23 x 8 x 128 x 3 at scale 8
        assert np.all(np.abs(got - ref) <= (1e-5 + abs(scale) * 0.012) * mag + 1e-6)


def test_small_and_large_queries_with_an_8_bit_cache():
    """Query rows go to fp16 by a power of two of their own: tiny, huge, zero and one-element rows keep their precision."""
    dev = require_gpu()
    p = Problem(dev, [200], 1, 8, 1, 128, 64, hla.HLA_E4M3, seed=4)
    q = p.q.float()
    q[0, 0, 0] *= 2.0 ** -60
    q[0, 0, 1] *= 1e-30
    q[0, 0, 2] = 0
    q[0, 0, 3, 1:] = 0
    q[0, 0, 4] *= 2.0 ** 3
    q[0, 0, 5, 7] = 2.0 ** 17      # beyond fp16
    q[0, 0, 5, :7] = 0
    p.q = q.to(BF16)
    p.scale = 1.0 / 128
    p.upload()
    k, v = p.values()
    ref, mag = oracle.attention.attend(p.q.double().numpy(), k, v, p.table.numpy(), p.past, p.scale)
    got = f64(p.decode(hla.HLA_F32))
    qs = np.abs(p.q.double().numpy()).sum(-1)
    size = p.scale * qs * np.nanmax(np.abs(k))
    # elements below 2^-38 of a row's largest may vanish in fp16: within d 2^-23 of the score's size as well
    tol = (2 * (128 * 2.0 ** -23 * size + 2.0 ** -21) + 2.0 ** -21 + 400 * 2.0 ** -23)[..., None] * mag + 1e-7
    assert np.all(np.abs(got - ref) <= tol)


def test_masked_places_may_hold_anything():
    """Infinities and NaN at keys and values a row does not see: the window's later tokens, rows behind the last token (the
    problem's poison), whole foreign pages; a row sees its own infinities."""
    dev = require_gpu()
    for dtype in (hla.HLA_BF16, hla.HLA_E4M3):
        for H, Hkv in ((4, 2), (16, 2), (16, 1), (24, 1)):  # 16-, 32- and 64-row tiles, and tcgen05's, at T = 4
            for past in (62, 64, 13):              # the window across a page and tile border, at its start, inside
                p = Problem(dev, [past, 100], 4, H, Hkv, 64, 16, dtype, seed=past)
                q = Problem(dev, [past, 100], 4, H, Hkv, 64, 16, dtype, seed=past).upload()
                clean, clean16 = q.decode(hla.HLA_F32), q.decode(hla.HLA_BF16)
                for t, what in ((2, float("nan")), (3, float("inf") if dtype == hla.HLA_BF16 else float("nan"))):
                    c = past + t
                    p.v[p.table[0, c // 16], :, c % 16] = torch.tensor(what).to(p.v.dtype)
                    p.k[p.table[0, c // 16], :, c % 16] = torch.tensor(what).to(p.k.dtype)
                o = p.upload().decode(hla.HLA_F32)
                torch.cuda.synchronize()
                # rows 0 and 1 of sequence 0 and all of sequence 1 see none of it; sums may run in another order
                assert torch.isfinite(o[0, :2]).all() and torch.isfinite(o[1]).all()
                assert torch.allclose(o[0, :2], clean[0, :2], rtol=1e-4, atol=1e-5)
                assert torch.equal(o[1], clean[1])
                assert torch.isnan(o[0, 2:]).all()
                o = p.decode(hla.HLA_BF16)
                assert torch.isfinite(o[0, :2]).all() and torch.isnan(o[0, 2:]).all() and torch.equal(o[1], clean16[1])
                assert torch.allclose(o[0, :2].float(), clean16[0, :2].float(), rtol=2.0 ** -6, atol=2.0 ** -8)


def test_blocks_without_a_page_hold_no_keys():
    dev = require_gpu()
    for sel in (False, True):
        p = Problem(dev, [500, 90, 40], 2, 8, 2, 128, 32, seed=6)
        p.table[0, 0], p.table[0, 3], p.table[0, 15] = -1, p.n_pages, 2 ** 31 - 1
        p.table[1] = -(2 ** 31)
        p.upload()
        lists = None
        if sel:
            lists = torch.arange(16, dtype=I32).repeat(3, 2, 2, 1)
        o = p.decode(hla.HLA_F32, None if lists is None else lists.to(dev))
        torch.cuda.synchronize()
        check(p, o, hla.HLA_F32, None if lists is None else lists.numpy())
        assert torch.all(o[1] == 0)


def test_positions_behind_the_table_are_dropped():
    dev = require_gpu()
    p = Problem(dev, [200, 100], 2, 4, 2, 64, 16, seed=7, max_blocks=5)
    p.upload()
    o = p.decode(hla.HLA_F32)
    check(p, o, hla.HLA_F32)
    # lengths far behind the table: every row sees the whole table
    far = p.D["past"]
    far.copy_(torch.tensor([2 ** 31 - 1, 2 ** 30], dtype=I32))
    o = p.decode(hla.HLA_F32)
    p.past = [10 ** 6, 10 ** 6]
    k, v = p.values()
    ref, _ = oracle.attention.attend(p.q.double().numpy(), k, v, p.table.numpy(), p.past, p.scale)
    assert np.allclose(f64(o), ref, rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("T,H,Hkv,d,page,n_sel", [(1, 8, 2, 128, 64, 5), (3, 12, 4, 64, 16, 9), (2, 40, 2, 128, 32, 3),
                                                  (1, 48, 1, 64, 128, 2), (2, 144, 2, 64, 16, 6)])
def test_sparse_matches_oracle(T, H, Hkv, d, page, n_sel, dtype):
    """Arbitrary lists: unsorted, repeated, behind the token, outside the table, empty."""
    dev = require_gpu()
    p = Problem(dev, [40 * page // 8, 11 * page + 3, -1, 0], T, H, Hkv, d, page, dtype, seed=n_sel, max_blocks=13).upload()
    g = np.random.default_rng(n_sel)
    sel = g.integers(-2, 15, size=(4, T, Hkv, n_sel))
    sel[1, 0, 0] = -1                       # nothing listed
    sel[0, -1, -1] = 2                      # one block, n_sel times
    lists = torch.from_numpy(sel).to(I32).to(dev)
    check(p, p.decode(hla.HLA_BF16, lists), hla.HLA_BF16, sel)
    o = p.decode(hla.HLA_F32, lists)
    assert hla.hla_last_variant().startswith("attn_sparse<")
    check(p, o, hla.HLA_F32, sel)
    assert torch.all(o[2] == 0) and torch.all(o[1, 0, :H // Hkv] == 0)


def test_listing_every_block_is_the_dense_form():
    dev = require_gpu()
    p = Problem(dev, [333, 64, 5], 2, 8, 2, 128, 32, seed=8).upload()
    sel = torch.arange(p.max_blocks, dtype=I32, device=dev).repeat(3, 2, 2, 1)
    dense, sparse = p.decode(hla.HLA_F32), p.decode(hla.HLA_F32, sel)
    assert torch.allclose(dense, sparse, rtol=1e-5, atol=1e-6)


def test_cache_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^31 and 2^32, in a pool that is written only where it is used."""
    dev = require_gpu()
    p = Problem(dev, [150, 70], 1, 8, 8, 128, 64, seed=10)
    page_elems = 8 * 64 * 128
    n_pages = 2 ** 32 // page_elems + 64
    k, v = (torch.empty(n_pages, 8, 64, 128, dtype=BF16, device=dev) for _ in range(2))
    moved = p.table.clone()
    places = [n_pages - 1, 2 ** 31 // page_elems, 2 ** 32 // page_elems + 1, 2 ** 31 // page_elems - 1, 3]
    for n, (b, j) in enumerate([(0, 0), (0, 1), (0, 2), (1, 0), (1, 1)]):
        moved[b, j] = places[n]
        k[places[n]], v[places[n]] = p.k[p.table[b, j]].to(dev), p.v[p.table[b, j]].to(dev)
    small = p.upload().decode(hla.HLA_F32)
    C = hla.make_kv_cache(hla.HLA_BF16, n_pages, 64, 8, 128, k, v)
    o = torch.empty_like(small)
    ws = torch.empty(hla.attn_paged_decode_workspace_size(C, 2, 1, 8), dtype=torch.uint8, device=dev)
    hla.attn_paged_decode(C, 2, 1, 8, p.max_blocks, moved.to(dev), p.D["past"], p.scale, p.D["q"], o, hla.HLA_F32, ws, ws.numel())
    assert torch.equal(o, small)
    check(p, o, hla.HLA_F32)


@pytest.mark.parametrize("H,Hkv,o_dtype", [(8, 2, hla.HLA_F32), (80, 2, hla.HLA_BF16)])
def test_one_captured_graph_serves_any_lengths_and_pages(H, Hkv, o_dtype):
    dev = require_gpu()
    p = Problem(dev, [700, 300, 20], 2, H, Hkv, 64, 32, seed=11, poison=False).upload()
    o = torch.empty(3, 2, H, 64, device=dev, dtype=torch.float32 if o_dtype == hla.HLA_F32 else BF16)
    ws = torch.empty(hla.attn_paged_decode_workspace_size(p.C, 3, 2, H), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        p.decode(o_dtype, ws=ws, o=o)
    side.synchronize()
    graphs = []
    for _ in range(2):  # two graphs that share the workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.decode(o_dtype, ws=ws, o=o)
        graphs.append(g)
    for past in ([700, 300, 20], [1, 640, -1], [0, 0, 0], [650, 2, 33]):
        p.D["past"].copy_(torch.tensor(past, dtype=I32))
        eager = p.decode(o_dtype)
        for g in graphs:
            ws.fill_(255)
            o.fill_(3.0)
            g.replay()
            assert torch.equal(o, eager)


def test_two_streams_at_once_with_their_own_workspaces():
    dev = require_gpu()
    ps = [Problem(dev, [900 + 40 * n, 100], 4, 16, 4, 128, 64, seed=12 + n).upload() for n in range(2)]
    want = [p.decode(hla.HLA_F32) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for p, s in zip(ps, streams):
            with torch.cuda.stream(s):
                got.append(p.decode(hla.HLA_F32))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_largest_batch_and_most_heads_per_kv_head():
    """1024 sequences (some idle), and 512 query heads on one kv head (four tcgen05 row tiles, eight of 64)."""
    dev = require_gpu()
    g = np.random.default_rng(16)
    past = [int(x) for x in g.integers(-1, 40, size=1024)]
    p = Problem(dev, past, 1, 2, 1, 64, 16, seed=16).upload()
    check(p, p.decode(hla.HLA_F32), hla.HLA_F32)
    p = Problem(dev, [90, 700], 1, 512, 1, 64, 32, seed=17).upload()
    for o_dtype in (hla.HLA_BF16, hla.HLA_F32):
        check(p, p.decode(o_dtype), o_dtype)


def test_output_and_workspace_stay_inside_their_bounds():
    dev = require_gpu()
    for T, H, Hkv, d, o_dtype in ((1, 8, 2, 128, 0), (5, 8, 2, 64, 0), (8, 16, 1, 128, 0), (8, 12, 1, 128, 1), (7, 10, 1, 64, 1)):
        p = Problem(dev, [500, 33], T, H, Hkv, d, 16, seed=13).upload()
        n = hla.attn_paged_decode_workspace_size(p.C, 2, T, H)
        ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=dev)
        elems = 2 * T * H * d
        o = torch.full((elems + 1024,), 5.0, device=dev, dtype=BF16 if o_dtype == hla.HLA_BF16 else torch.float32)
        hla.attn_paged_decode(p.C, 2, T, H, p.max_blocks, p.D["table"], p.D["past"], p.scale, p.D["q"], o, o_dtype, ws, n)
        torch.cuda.synchronize()
        assert torch.all(ws[n:] == 0x5A) and torch.all(o[elems:] == 5.0) and not torch.any(o[:elems] == 5.0)


def test_inside_a_launch_chain():
    dev = require_gpu()
    p = Problem(dev, [400, 60], 1, 8, 2, 128, 64, seed=14).upload()
    want = p.decode(hla.HLA_F32)
    o = torch.zeros_like(want)
    ws = torch.empty(hla.attn_paged_decode_workspace_size(p.C, 2, 1, 8), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    hla.hla_chain_begin()
    try:
        for _ in range(4):
            p.decode(hla.HLA_F32, ws=ws, o=o)
    finally:
        hla.hla_chain_end()
    assert torch.equal(o, want)


def test_forced_wait_timeout_is_reported_and_nothing_is_written():
    """A tcgen05 launch whose wait gives up reports it once through the status word and leaves the output alone; the
    next launch is right."""
    dev = require_gpu()
    p = Problem(dev, [300, 70], 8, 16, 1, 64, 32, seed=15).upload()
    torch.cuda.synchronize()
    assert hla.hla_device_status() == 0
    try:
        hla.hla_test_force_wait_timeout(1)
        o = p.decode(hla.HLA_BF16)
        torch.cuda.synchronize()
    finally:
        hla.hla_test_force_wait_timeout(0)
    assert hla.hla_device_status() == 6 and hla.hla_device_status() == 0  # HLA_ERR_DEVICE_TIMEOUT, then cleared
    assert torch.all(o == 7.0)
    check(p, p.decode(hla.HLA_BF16), hla.HLA_BF16)


def test_sequences_that_share_a_prefix():
    """Four sequences on the same first pages, each with its own last one, through the dense, listed and chosen forms."""
    dev = require_gpu()
    for H, Hkv, o_dtype in ((8, 2, hla.HLA_F32), (36, 1, hla.HLA_BF16)):
        p = Problem(dev, [70, 75, 64, 79], 2, H, Hkv, 64, 16, seed=18, poison=False)
        p.table[1:, :4] = p.table[0, :4]
        p.upload()
        check(p, p.decode(o_dtype), o_dtype)
        sel = np.tile(np.array([3, 0, 4]), (4, 2, Hkv, 1))
        check(p, p.decode(o_dtype, torch.from_numpy(sel).to(I32).to(dev)), o_dtype, sel)


def test_largest_batch_on_tcgen05():
    """1024 windows of 8 tokens, 72 rows each, some idle: every CTA runs many short units."""
    dev = require_gpu()
    g = np.random.default_rng(19)
    for d in (64, 128):
        p = Problem(dev, [int(x) for x in g.integers(-1, 9, size=1024)], 8, 9, 1, d, 16, seed=19).upload()
        check(p, p.decode(hla.HLA_BF16), hla.HLA_BF16)
        assert hla.hla_last_variant().endswith("m128>")


def test_stream_argument():
    """The stream given by object or by handle, with another one current."""
    dev = require_gpu()
    p = Problem(dev, [300, 40], 2, 8, 2, 64, 16, seed=20).upload()
    want = p.decode(hla.HLA_F32)
    ws = torch.empty(hla.attn_paged_decode_workspace_size(p.C, 2, 2, 8), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        o = torch.zeros_like(want)
        torch.cuda.synchronize()
        p.decode(hla.HLA_F32, stream=stream, ws=ws, o=o)
        side.synchronize()
        assert torch.equal(o, want)


def test_a_list_is_read_up_to_the_blocks_the_token_sees():
    """Entries behind those are not read: neither a visible block there nor a further mention counts."""
    dev = require_gpu()
    p = Problem(dev, [17, 3], 1, 4, 2, 64, 16, seed=21).upload()
    lists = torch.tensor([[-1, 1, 0, 0], [0, 0, 0, 0]], dtype=I32).view(2, 1, 1, 4).repeat(1, 1, 2, 1)
    short = torch.tensor([[-1, 1, -1, -1], [0, -1, -1, -1]], dtype=I32).view(2, 1, 1, 4).repeat(1, 1, 2, 1)
    a, b = p.decode(hla.HLA_F32, lists.to(dev)), p.decode(hla.HLA_F32, short.to(dev))
    assert torch.equal(a, b)
    check(p, a, hla.HLA_F32, short.numpy())


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("o_dtype", [hla.HLA_BF16, hla.HLA_F32])
@pytest.mark.parametrize("T,H,Hkv,d", [(1, 8, 8, 128), (2, 16, 8, 64), (8, 9, 1, 128), (3, 40, 4, 64)])
def test_more_units_than_run_at_once(T, H, Hkv, d, o_dtype, dtype):
    """Sequences of no, few and thousands of tokens in one call: units of many CTAs, many units of one, and none."""
    dev = require_gpu()
    g = np.random.default_rng(22)
    past = [int(x) for x in g.integers(-1, 60, size=640 // Hkv)]
    past[0], past[7], past[-1] = -1, 3000, 1500
    past[20:30] = [-1] * 10
    p = Problem(dev, past, T, H, Hkv, d, 32, dtype, seed=22).upload()
    check(p, p.decode(o_dtype), o_dtype)
    sel = g.integers(-1, 95, size=(len(past), T, Hkv, 12))
    check(p, p.decode(o_dtype, torch.from_numpy(sel).to(I32).to(dev)), o_dtype, sel)


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("T,H,Hkv,d", [(1, 8, 8, 128), (1, 32, 8, 64), (4, 16, 4, 128), (2, 24, 3, 128), (5, 3, 1, 64)])
def test_a_bf16_output_is_off_by_its_rounding_alone(T, H, Hkv, d, dtype):
    """Up to 16 rows: the weights lose nothing that the output would show."""
    p = Problem(require_gpu(), [1500, 700, 2100, 33], T, H, Hkv, d, 64, dtype, seed=23).upload()
    k, v = p.values()
    lists = np.tile(np.arange(0, 34, 2), (4, T, Hkv, 1))
    for sel in (None, lists):
        ref, _ = oracle.attention.attend(p.q.double().numpy(), k, v, p.table.numpy(), p.past, p.scale, sel)
        o = f64(p.decode(hla.HLA_BF16, None if sel is None else torch.from_numpy(sel).to(I32).to(p.dev)))
        size, rounding = np.linalg.norm(ref), np.linalg.norm(torch.from_numpy(ref).to(BF16).double().numpy() - ref)
        # An error e before the output's rounding shifts a value's distance from its rounded self by |e| at most, and adds |e|.
        # Two bf16 parts hold a weight to 2^-16, and independent errors of weights over values of either sign add up to that
        # much of the output (twice that with what fp32 sums and scores err); fp16 holds 2^-11 worst, which is one error
        # among independent others: a square root of squares.
        err = np.linalg.norm(o - ref)
        if dtype == hla.HLA_BF16:
            assert err <= rounding + 2 * 2.0 ** -15 * size, (err / size, rounding / size)
        else:
            assert err <= np.hypot(rounding, 2.0 ** -11 * size) + 2 * 2.0 ** -15 * size, (err / size, rounding / size)


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("T,H,Hkv,d", [(1, 8, 2, 128), (4, 16, 2, 64), (8, 8, 1, 128), (8, 9, 1, 128), (8, 16, 1, 64)])
def test_equal_values_come_back_as_they_are(T, H, Hkv, d, dtype):
    """Numerator and denominator hold the same rounded weights: over keys whose values are all alike an output is that value,
    whatever the scores (a few keys dominate here, and their weights are no powers of two).  Where they differ, the largest
    mantissa shows it first: a step of its own is 2^-8 of it."""
    p = Problem(require_gpu(), [3000], T, H, Hkv, d, 64, dtype, seed=24, poison=False)
    # sequences on the same pages: several tiles for every CTA, over which a row's maximum rises
    p.B, p.past = 64, [3000 - 40 * b for b in range(64)]
    p.table = p.table.repeat(64, 1)
    p.q = torch.randn((64, T, H, d), generator=inputs.generator(25)).to(BF16)
    value = 255 / 128 if dtype == hla.HLA_BF16 else 1.875
    p.v = torch.full_like(p.v.float(), value).to(p.v.dtype)
    if dtype == hla.HLA_E4M3:
        p.v_scale[:] = 1
    p.upload()
    for scale in (4 * d ** -0.5, 16 * d ** -0.5, 40 * d ** -0.5):
        p.scale = scale
        o = p.decode(hla.HLA_BF16)
        assert torch.all(o == value), (scale, torch.unique(o.float(), return_counts=True))


def test_tcgen05_keeps_its_pace_with_the_batch():
    """The time per cached token does not jump where a batch grows: 119 and 120 sequences, and 800, on the same pages.  (Two
    CTAs to an SM or one is a factor of 1.6; units that end and begin cost the larger batch some of its time.)"""
    dev = require_gpu()

    def us_per_token(B, n, d):
        p = Problem(dev, [n], 8, 16, 1, d, 64, seed=26, poison=False)
        p.B, p.past, p.table = B, [n] * B, p.table.repeat(B, 1)
        p.q = p.q.repeat(B, 1, 1, 1)
        p.upload()
        o = torch.empty(B, 8, 16, d, dtype=BF16, device=dev)
        ws = torch.empty(hla.attn_paged_decode_workspace_size(p.C, B, 8, 16), dtype=torch.uint8, device=dev)
        times = []
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            p.decode(hla.HLA_BF16, ws=ws, o=o)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        return sorted(times[3:])[4] / (B * n)

    for d in (128, 64):
        small, large, many = us_per_token(119, 24000, d), us_per_token(120, 24000, d), us_per_token(800, 24000, d)
        assert large < 1.2 * small and many < 1.2 * small, (d, small, large, many)


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("T,H,Hkv,d", [(1, 8, 2, 128), (4, 16, 2, 64), (8, 8, 1, 128), (8, 9, 1, 128), (8, 16, 1, 64)])
def test_scores_beyond_the_precision_of_their_differences(T, H, Hkv, d, dtype):
    """Scores of 2^31 and far beyond, exact in fp32: one product each.  The highest key of a row takes all, so the row is that
    key's value; the fp32 spacing of such scores is no weight."""
    dev = require_gpu()
    for past, top in (([300, 40, 0], 2.0 ** 31), ([2500, 100, 7], 2.0 ** 36), ([900, 333, 64], 2.0 ** 120)):
        p = Problem(dev, past, T, H, Hkv, d, 16, dtype, seed=27, poison=False)
        # keys of 1 to 1.9375 (bf16 and e4m3 both hold 1, 1.125, ...) over 2^(x) in one channel, the others zero
        g = inputs.generator(28)
        p.k = torch.zeros(p.k.shape)
        p.k[..., 3] = -(1 + torch.randint(0, 8, p.k.shape[:-1], generator=g) / 8)
        for b in range(3):  # one key per kv head above all others, seen by every token of the window
            for h in range(Hkv):
                c = (past[b] * (h + 1) * 5) // 7 % (past[b] + 1)
                p.k[p.table[b, c // 16], h, c % 16, 3] = 2.0
        p.k = p.k.to(p.v.dtype)
        p.q = torch.zeros(p.q.shape, dtype=BF16)
        p.q[..., 3] = top
        p.scale = 1.0
        if dtype == hla.HLA_E4M3:
            p.k_scale[:] = 1
        p.upload()
        k, v = p.values()
        ref, _ = oracle.attention.attend(p.q.double().numpy(), k, v, p.table.numpy(), p.past, 1.0)
        for o_dtype, half in ((hla.HLA_F32, 2.0 ** -23), (hla.HLA_BF16, 2.0 ** -8)):
            # a weight of 1 and zeros: the value, times its scale in fp32
            assert np.all(np.abs(f64(p.decode(o_dtype)) - ref) <= half * np.abs(ref)), (top, o_dtype)


@pytest.mark.parametrize("T,H,dtype,o_dtype", [(8, 8, hla.HLA_BF16, hla.HLA_BF16), (8, 16, hla.HLA_E4M3, hla.HLA_BF16),
                                               (8, 16, hla.HLA_BF16, hla.HLA_F32)])
def test_forms_without_bounded_waits_ignore_the_forced_timeout(T, H, dtype, o_dtype):
    """At most 64 rows, an 8-bit cache or an fp32 output: the hook changes nothing and the status word stays clear."""
    dev = require_gpu()
    p = Problem(dev, [300, 70], T, H, 1, 64, 32, dtype, seed=29).upload()
    want = p.decode(o_dtype)
    torch.cuda.synchronize()
    try:
        hla.hla_test_force_wait_timeout(1)
        o = p.decode(o_dtype)
        torch.cuda.synchronize()
    finally:
        hla.hla_test_force_wait_timeout(0)
    assert hla.hla_device_status() == 0
    assert torch.equal(bits(o), bits(want))


@pytest.mark.parametrize("B", [112, 113, 224, 225, 449, 897])
def test_tcgen05_finds_its_sequences_in_any_batch(B):
    """Around the batches from which a CTA keeps every 2nd, 4th, ... prefix sum: idle sequences alone, in runs and at the ends,
    lengths of nothing to many tiles."""
    g = np.random.default_rng(B)
    past = [int(x) for x in g.integers(-1, 200, size=B)]
    past[B // 3:B // 3 + 19], past[0], past[1], past[-2:] = [-1] * 19, -1, 1700, [900, -1]
    for T, H, sparse in ((8, 9, False), (1, 66, True)):
        p = Problem(require_gpu(), past, T, H, 1, 128, 64, seed=B).upload()
        sel = g.integers(-1, 28, size=(B, T, 1, 5)) if sparse else None
        check(p, p.decode(hla.HLA_BF16, None if sel is None else torch.from_numpy(sel).to(I32).to(p.dev)), hla.HLA_BF16, sel)
        assert hla.hla_last_variant().endswith("m128>")


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("T,H,Hkv,d", [(1, 8, 2, 128), (4, 8, 1, 64), (8, 8, 1, 128), (8, 9, 1, 128), (8, 16, 1, 64)])
def test_rows_of_scores_of_minus_infinity(T, H, Hkv, d, dtype):
    """An infinite query channel against negative keys: rows all of whose scores are -infinity are zero, beside rows that are
    not, whole units and joined ones."""
    p = Problem(require_gpu(), [900, 20, 0], T, H, Hkv, d, 16, dtype, seed=33)
    p.k[..., 0] = torch.where(torch.isnan(p.k[..., 0].float()), p.k[..., 0].float(), -2.0).to(p.k.dtype)
    plain = p.upload().decode(hla.HLA_BF16)
    p.q[:, :, ::2, 0] = float("inf")
    p.upload()
    for o_dtype in (hla.HLA_BF16, hla.HLA_F32):
        o = p.decode(o_dtype)
        assert torch.all(o[:, :, ::2] == 0)
        if o_dtype == hla.HLA_BF16:
            assert torch.equal(bits(o[:, :, 1::2]), bits(plain[:, :, 1::2]))
