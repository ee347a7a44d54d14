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


def check(layer, x, residual=None, got=None, rel_limit=MOE_FROB_REL):
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
    assert worst <= 1.0 and rel < rel_limit


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


@pytest.mark.parametrize("M,Hd,I,E,k,shared", [
    (8, 128, 256, 40, 8, 1), (9, 128, 256, 40, 8, 1), (8, 256, 128, 300, 3, 0), (9, 256, 128, 300, 16, 0),  # either place of the choice
    (1, 256, 2048, 16, 4, 1), (23, 384, 768, 8, 2, 1), (53, 512, 256, 60, 4, 2), (64, 128, 1024, 64, 8, 1), (2, 2048, 128, 4, 1, 0)])
def test_few_items_and_either_choice(M, Hd, I, E, k, shared):
    """Layers of so few output blocks that not all CTAs share them, the choice in the last kernel and in its own."""
    dev = require_gpu()
    layer = Moe(hla, dev, Hd, I, E, k, shared, seed=M + Hd)
    x = layer.tokens(M, M)
    first = layer.run(x)
    check(layer, x, got=first)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(layer.run(x), first))


def test_full_size():
    dev = require_gpu()
    layer = Moe(hla, dev, 7168, 2048, 256, 8, 1, seed=1)
    for M in (1, 3, 16, 20, 64):
        x = layer.tokens(M, M)
        # one of 18432 values of h on another side of a rounding border moves y by 2^-4 / 136 of itself: bf16 rounding dominates
        check(layer, x, torch.randn(M, 7168, device=dev, generator=torch.Generator(dev).manual_seed(M)).to(BF), rel_limit=2.0 ** -8)
        ws = layer.workspace(M)
        first = layer.run(x, ws=ws)[0]
        for _ in range(3):  # the same bits, however the CTAs' work falls
            assert torch.equal(layer.run(x, ws=ws)[0], first)


@pytest.mark.parametrize("M", [16, 24, 40, 64])
def test_crowded_experts(M):
    """All tokens the same: every chosen expert has all of them; and half of them the same: experts with 9 or more tokens of a half
    of the batch beside others with few."""
    dev = require_gpu()
    layer = Moe(hla, dev, 512, 256, 24, 4, 1, seed=M)
    x = layer.tokens(M, 5)
    check(layer, x[:1].expand(M, -1).contiguous())
    x[::2] = x[0]
    check(layer, x)
    x[: M // 2] = x[1]
    check(layer, x)


def test_outputs_and_workspace_stay_in_their_bounds():
    dev = require_gpu()
    layer = Moe(hla, dev, 384, 256, 20, 3, 1, seed=2)
    for M in (1, 5, 17, 64):
        x = layer.tokens(M, M)
        n = hla.moe_fp8_forward_workspace_size(layer.L, M)
        ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device=dev)
        y = torch.full((M + 2, 384), 7.0, dtype=BF, device=dev)
        idx = torch.full((M + 2, 3), -7, dtype=torch.int32, device=dev)
        w = torch.full((M + 2, 3), 7.0, device=dev)
        hla.moe_fp8_forward(layer.L, M, x, None, y, idx, w, ws, n)
        torch.cuda.synchronize()
        assert torch.all(ws[n:] == 0xAB) and torch.all(y[M:] == 7.0) and torch.all(idx[M:] == -7) and torch.all(w[M:] == 7.0)
        check(layer, x, got=(y[:M], idx[:M], w[:M]))


def test_bits_do_not_depend_on_workspace_outputs_or_aliasing():
    dev = require_gpu()
    layer = Moe(hla, dev, 1024, 384, 60, 8, 1, seed=3)
    for M in (1, 9, 30, 64):
        x = layer.tokens(M, M)
        residual = torch.randn(M, 1024, device=dev).to(BF)
        y, idx, w = layer.run(x, residual)
        for fill in (0x00, 0x7F, 0x80):
            again, _, _ = layer.run(x, residual, ws=layer.workspace(M, fill))
            assert torch.equal(again, y)
        ws = layer.workspace(M)
        r = residual.clone()
        hla.moe_fp8_forward(layer.L, M, x, r, r, None, None, ws, ws.numel())   # y in place of the residual
        xx = x.clone()
        hla.moe_fp8_forward(layer.L, M, xx, residual, xx, None, None, ws, ws.numel())  # and of x
        assert torch.equal(r, y) and torch.equal(xx, y)


@pytest.mark.parametrize("M", [3, 20, 64])
def test_nan_reaches_only_its_tokens(M):
    dev = require_gpu()
    layer = Moe(hla, dev, 256, 256, 12, 2, 0, seed=4)
    x = layer.tokens(M, M)
    x[M // 2:] = x[M // 2]                      # crowded beside sparse experts
    y, idx, _ = layer.run(x)
    bad = int(idx[0, 1])                        # an expert of token 0 gets a NaN weight in each matrix
    for name in ("gate", "up", "down"):
        layer.w[name].view(torch.uint8)[bad, 3, 7] = 0x7F
    z, idx2, _ = layer.run(x)
    hit = (idx == bad).any(-1)
    assert torch.equal(idx, idx2) and bool(hit[0])
    assert torch.all(z[hit].isnan().any(-1)) and torch.equal(z[~hit], y[~hit])
    # a token with a NaN or an infinity: its row only
    layer = Moe(hla, dev, 256, 256, 12, 2, 1, seed=4)
    y, _, _ = layer.run(x)
    for v in (float("nan"), float("inf")):
        xx = x.clone()
        xx[1, 9] = v
        z, idx, _ = layer.run(xx)
        assert torch.all(z[1].isnan()) and torch.equal(z[0], y[0]) and torch.equal(z[2:], y[2:])
        assert torch.all((idx >= 0) & (idx < 12))


def test_scores_below_fp32_keep_their_weights():
    """Logits near -150: every sigmoid is below the smallest fp32 number, their shares are not."""
    dev = require_gpu()
    layer = Moe(hla, dev, 256, 128, 20, 4, 1, seed=13)
    layer.W_r = (layer.W_r.float() - 150.0 / 256).to(BF)
    layer.L = layer.descriptor()
    x = torch.ones(5, 256, device=dev).to(BF) + layer.tokens(5, 1) * 0.05
    y, idx, w = layer.run(x.contiguous())
    logits = (x.double() @ layer.W_r.double().T).sort(-1, descending=True).values[:, :5]
    assert logits.max() < -104 and logits.diff(dim=-1).abs().min() > 1e-3
    want, bound, want_idx, want_w = layer.reference(x)
    assert torch.equal(idx.long(), want_idx)
    # fp32 sums of 256 products of size 0.6 move a logit by 256 * 2^-24 * 150 at most, and a share by as much of itself
    assert torch.all((w.double() - want_w).abs() <= 3e-3 * want_w) and torch.all(y.isfinite())
    check_rel = float((y.double() - want).norm() / want.norm())
    assert check_rel < MOE_FROB_REL


def test_graphs_share_a_workspace_and_see_new_inputs():
    dev = require_gpu()
    a, b = Moe(hla, dev, 512, 256, 40, 4, 1, seed=5), Moe(hla, dev, 256, 128, 16, 2, 0, seed=6)
    n = max(hla.moe_fp8_forward_workspace_size(a.L, 64), hla.moe_fp8_forward_workspace_size(b.L, 7))
    ws = torch.full((n,), 0xEE, dtype=torch.uint8, device=dev)
    xa, xb = a.tokens(64, 1), b.tokens(7, 2)
    ya, yb = torch.empty_like(xa), torch.empty_like(xb)
    graphs = []
    for layer, x, y in ((a, xa, ya), (b, xb, yb)):
        hla.moe_fp8_forward(layer.L, x.shape[0], x, None, y, None, None, ws, n)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hla.moe_fp8_forward(layer.L, x.shape[0], x, None, y, None, None, ws, n)
        graphs.append(g)
    for i in range(3):
        xa.copy_(a.tokens(64, 10 + i))
        xb.copy_(b.tokens(7, 20 + i))
        for g in graphs:
            g.replay()
        assert torch.equal(ya, a.run(xa)[0]) and torch.equal(yb, b.run(xb)[0])


def test_two_streams_at_once():
    dev = require_gpu()
    layer = Moe(hla, dev, 1024, 512, 32, 4, 1, seed=7)
    xs = [layer.tokens(M, M) for M in (64, 40)]
    want = [layer.run(x)[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ws = [layer.workspace(x.shape[0]) for x in xs]
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                y = torch.empty_like(xs[i])
                hla.moe_fp8_forward(layer.L, xs[i].shape[0], xs[i], None, y, None, None, ws[i], ws[i].numel())
                got[i].append(y)
    torch.cuda.synchronize()
    assert hla.hla_device_status() == 0
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_wait_timeout_is_reported():
    dev = require_gpu()
    layer = Moe(hla, dev, 256, 128, 16, 2, 0, seed=8)
    x = layer.tokens(4, 4)
    torch.cuda.synchronize()
    assert hla.hla_device_status() == 0
    try:
        hla.hla_test_force_wait_timeout(1)
        y, _, _ = layer.run(x)
        torch.cuda.synchronize()
    finally:
        hla.hla_test_force_wait_timeout(0)
    assert hla.hla_device_status() == HLA_ERR_DEVICE_TIMEOUT and hla.hla_device_status() == 0
    assert torch.all(y == 7.0)
    check(layer, x)


def test_a_decode_step_of_the_8_bit_operators():
    """bf16 weights converted once; then projection + residual, norm and the experts in one launch chain, each stage against the
    fp64 oracle on what the stage before left."""
    dev = require_gpu()
    g = torch.Generator(dev).manual_seed(12)
    M, Hd, I, E, k, K = 6, 256, 128, 10, 2, 512

    def weight(rows, cols):
        w = (torch.randn(rows, cols, generator=g, device=dev) * 0.05).to(BF)
        q, s = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=dev), torch.empty(up(rows, 128), up(cols, 128), device=dev)
        hla.fp8_quantize(rows, cols, w, hla.HLA_BF16, 128, q, s)
        return q, s

    W_o, s_o = weight(Hd, K)
    W_r = (torch.randn(E, Hd, generator=g, device=dev) * 0.1).to(BF)
    stacks = {n: weight(E * r, c) for n, r, c in (("gate", I, Hd), ("up", I, Hd), ("down", Hd, I))}
    shared = {n: weight(r, c) for n, r, c in (("gate", I, Hd), ("up", I, Hd), ("down", Hd, I))}
    names = ("gate", "up", "down")
    L = hla.make_moe_fp8(Hd, I, E, k, 1, W_r, *(stacks[n][0] for n in names), *(stacks[n][1] for n in names),
                         *(shared[n][0] for n in names), *(shared[n][1] for n in names))
    o, x = (torch.randn(M, n, generator=g, device=dev).to(BF) for n in (K, Hd))
    gamma = torch.ones(Hd, dtype=BF, device=dev)
    oq, os_ = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=dev), torch.empty(M, K // 128, device=dev)
    r, xn, y = (torch.empty(M, Hd, dtype=BF, device=dev) for _ in range(3))
    idx, w = torch.empty(M, k, dtype=torch.int32, device=dev), torch.empty(M, k, device=dev)
    ws = torch.empty(hla.moe_fp8_forward_workspace_size(L, M), dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    hla.hla_chain_begin()
    hla.fp8_quantize(M, K, o, hla.HLA_BF16, 1, oq, os_)
    hla.fp8_matmul(M, Hd, K, oq, os_, W_o, s_o, x, r, hla.HLA_BF16)
    hla.hla_rmsnorm(M, Hd, r, gamma, 1e-6, xn)
    hla.moe_fp8_forward(L, M, xn, r, y, idx, w, ws, ws.numel())
    hla.hla_chain_end()
    torch.cuda.synchronize()
    assert hla.hla_device_status() == 0
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    q, s = oracle.fp8.quantize(f(o))
    assert np.array_equal(f(oq), q) and np.array_equal(f(os_), s)
    want = oracle.fp8.matmul(q, s, f(W_o), f(s_o), f(x))
    assert np.all(np.abs(f(r) - want) <= np.abs(want) * 2.0 ** -8 * 1.01 + 1e-4)  # half a step of bf16; sums of fp32 lose less than 1e-4
    val = lambda n, t: f(values64(t[n][0], t[n][1], 128))  # noqa: E731
    full = {n: val(n, stacks) for n in names}
    cut = lambda n, e: full[n].reshape(E, -1, full[n].shape[1])[e]  # noqa: E731
    want, want_idx, want_w = oracle.fp8.moe_layer(f(xn), f(W_r), k, lambda e: tuple(cut(n, e) for n in names),
                                                  [tuple(val(n, shared) for n in names)], f(r))
    assert np.array_equal(idx.cpu().numpy(), want_idx) and np.allclose(f(w), want_w, rtol=2e-6)
    assert np.linalg.norm(f(y) - want) / np.linalg.norm(want) < MOE_FROB_REL


@pytest.mark.parametrize("M", [3, 20, 64])
@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_nan_and_infinite_scales_reach_only_tokens_of_their_expert(M, name):
    """A block of weights that holds a NaN or an infinity is converted to a NaN scale; scales may be infinite, too."""
    dev = require_gpu()
    for v in (float("nan"), float("inf"), -float("inf")):
        layer = Moe(hla, dev, 256, 256, 12, 2, 0, seed=4)
        x = layer.tokens(M, M)
        x[M // 2:] = x[M // 2]
        y, idx, _ = layer.run(x)
        count = torch.bincount(idx.flatten().long(), minlength=12).cpu()
        scale = layer.s[name]
        for bad in {int(count.argmax()), int(count.masked_fill(count == 0, M + 1).argmin()), int(idx[0, 1])}:  # crowded, and few tokens'
            keep = scale[bad, 0, 1].clone()
            scale[bad, 0, 1] = v
            z, idx2, _ = layer.run(x)
            scale[bad, 0, 1] = keep
            hit = (idx == bad).any(-1)
            assert torch.equal(idx, idx2) and bool(hit.any())
            assert torch.equal(z[~hit], y[~hit])
            if name == "down":  # 128 of the output's rows
                assert not torch.any(z[hit][:, :128].isfinite()) and torch.equal(z[:, 128:], y[:, 128:])
            else:               # 128 of h, whose scale is then NaN: all of the output
                assert not torch.any(z[hit].isfinite())


@pytest.mark.parametrize("M", [3, 20, 64])
def test_a_scale_of_zero_hides_no_nan(M):
    """NaN times a scale of 0 is NaN for the tokens of the expert, however many they are, and nothing for the others."""
    dev = require_gpu()
    layer = Moe(hla, dev, 256, 256, 12, 2, 0, seed=4)
    x = layer.tokens(M, M)
    x[M // 2:] = x[M // 2]
    y, idx, _ = layer.run(x)
    count = torch.bincount(idx.flatten().long(), minlength=12).cpu()
    for bad in (int(count.argmax()), int(count.masked_fill(count == 0, M + 1).argmin())):
        w, scale = layer.w["down"].view(torch.uint8), layer.s["down"]
        keep, byte = scale[bad, 0, 1].clone(), w[bad, 3, 200].clone()
        hit = (idx == bad).any(-1)
        scale[bad, 0, 1] = 0.0
        z, _, _ = layer.run(x)                      # zeros alone: finite
        assert torch.all(z.isfinite()) and torch.equal(z[~hit], y[~hit]) and torch.equal(z[:, 128:], y[:, 128:])
        w[bad, 3, 200] = 0x7F
        again, _, _ = layer.run(x)
        scale[bad, 0, 1], w[bad, 3, 200] = keep, byte
        assert torch.all(again[hit][:, 3].isnan())
        again[hit, 3] = z[hit, 3]
        assert torch.equal(again, z)


def test_views_aligned_to_16_bytes():
    dev = require_gpu()

    def off(t):  # t at an address that is 16 bytes past a multiple of 512
        raw = torch.zeros(t.numel() * t.element_size() + 512, dtype=torch.uint8, device=dev)
        v = raw[16:16 + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        v.view(torch.uint8).copy_(t.view(torch.uint8))
        assert v.data_ptr() % 512 == 16
        return v

    layer = Moe(hla, dev, 384, 256, 20, 3, 1, seed=2)
    for M in (3, 20, 64):
        x = layer.tokens(M, M)
        residual = torch.randn(M, 384, device=dev).to(BF)
        y, idx, w = layer.run(x, residual)
        keep = layer.W_r, dict(layer.w), dict(layer.s)
        layer.W_r = off(layer.W_r)
        layer.w = {n: off(t) for n, t in layer.w.items()}
        layer.s = {n: off(t) for n, t in layer.s.items()}
        L = layer.descriptor()
        layer.W_r, layer.w, layer.s = keep
        ws = off(layer.workspace(M))
        y2, idx2, w2 = off(torch.full_like(y, 7.0)), off(torch.full_like(idx, -7)), off(torch.full_like(w, 7.0))
        hla.moe_fp8_forward(L, M, off(x), off(residual), y2, idx2, w2, ws, ws.numel())
        assert torch.equal(y2, y) and torch.equal(idx2, idx) and torch.equal(w2, w)


def test_parallel_branches_of_a_graph():
    """Two layers, and products beside them, on branches of one graph that nothing orders: each with its own workspace."""
    dev = require_gpu()
    a, b = Moe(hla, dev, 1024, 512, 32, 4, 1, seed=7), Moe(hla, dev, 2048, 256, 16, 4, 0, seed=8)
    xa, xb = a.tokens(64, 1), b.tokens(5, 2)
    want_a, want_b = a.run(xa)[0], b.run(xb)[0]
    M, N, K = 600, 4000, 1024
    q, W = (torch.randn(n, K, device=dev).to(torch.float8_e4m3fn) for n in (M, N))
    s, ws = torch.ones(M, up(K, 128), device=dev), torch.ones(up(N, 128), up(K, 128), device=dev)
    y = torch.empty(M, N, dtype=BF, device=dev)
    hla.fp8_matmul(M, N, K, q, s, W, ws, None, y, hla.HLA_BF16)
    want_y = y.clone()
    ya, yb = torch.empty_like(xa), torch.empty_like(xb)
    spaces = a.workspace(64), b.workspace(5)
    torch.cuda.synchronize()
    graph, side, third = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        third.wait_stream(main)
        for _ in range(4):
            hla.moe_fp8_forward(a.L, 64, xa, None, ya, None, None, spaces[0], spaces[0].numel())
            with torch.cuda.stream(side):
                hla.moe_fp8_forward(b.L, 5, xb, None, yb, None, None, spaces[1], spaces[1].numel())
            with torch.cuda.stream(third):
                hla.fp8_matmul(M, N, K, q, s, W, ws, None, y, hla.HLA_BF16)
        main.wait_stream(side)
        main.wait_stream(third)
    for _ in range(10):
        ya.zero_(), yb.zero_(), y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert hla.hla_device_status() == 0
        assert torch.equal(ya, want_a) and torch.equal(yb, want_b) and torch.equal(y, want_y)
