"""Appending to the paged cache (rotation, both cache types, key bounds), block choice, and the operators together,
against the fp64 oracle."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from hybrid_linear_attention_gated_gb300 import hla, inputs
from tests.attn_common import BF16, F32, FP8, I32, Problem, bits
from tests.gpu_common import f64, require_gpu

pytestmark = pytest.mark.gpu


def freqs(n, base=10000.0):
    return base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))


class Append:
    def __init__(self, dev, past, new, H=8, Hkv=2, d=128, page=64, dtype=hla.HLA_BF16, rope=128, inter=0, seed=0, behind=3,
                 bounds=True, max_blocks=None):
        g = inputs.generator(seed)
        need = [-(-(p + n) // page) if p >= 0 else 0 for p, n in zip(past, new)]
        self.max_blocks = max_blocks or max(need + [1])
        self.n_pages = sum(need) + 2
        order, at = torch.randperm(self.n_pages, generator=g).to(I32), 0
        self.table = torch.full((len(past), self.max_blocks), -1, dtype=I32)
        for b, n in enumerate(need):
            m = min(n, self.max_blocks)
            self.table[b, :m] = order[at:at + m]
            at += n
        self.past, self.new, self.cu = past, new, np.concatenate([[0], np.cumsum(new)])
        self.N = int(self.cu[-1]) + behind
        store = FP8 if dtype == hla.HLA_E4M3 else BF16
        shape = (self.n_pages, Hkv, page, d)
        self.kc, self.vc = ((torch.randn(shape, generator=g) * 3).to(store) for _ in range(2))
        self.q = torch.randn(self.N, H, d, generator=g).to(BF16)
        self.k, self.v = ((torch.randn(self.N, Hkv, d, generator=g) * 2).to(BF16) for _ in range(2))
        self.ks = self.vs = None
        if dtype == hla.HLA_E4M3:
            self.ks, self.vs = (torch.rand(Hkv, generator=g) * 0.2 + 0.01 for _ in range(2))
        self.lo = torch.full((self.n_pages, Hkv, d), 11.0, dtype=BF16) if bounds else None
        self.hi = torch.full((self.n_pages, Hkv, d), -11.0, dtype=BF16) if bounds else None
        self.f, self.rope, self.inter, self.dtype = freqs(rope // 2), rope, inter, dtype
        self.dev, self.H, self.Hkv, self.d, self.page = dev, H, Hkv, d, page

    def run(self, in_place=False, times=1):
        up = lambda t: None if t is None else t.to(self.dev)  # noqa: E731
        kc, vc, lo, hi = up(self.kc), up(self.vc), up(self.lo), up(self.hi)
        ks, vs = up(self.ks), up(self.vs)
        C = hla.make_kv_cache(self.dtype, self.n_pages, self.page, self.Hkv, self.d, kc, vc, ks, vs, lo, hi)
        q = up(self.q)
        out = q if in_place else torch.full_like(q, 9.0)
        cu = torch.from_numpy(self.cu).to(I32).to(self.dev)
        past, table = torch.tensor(self.past, dtype=I32, device=self.dev), up(self.table)
        for _ in range(times):
            hla.kv_cache_append(C, self.N, len(self.past), cu, past, self.max_blocks, table, self.H, q, up(self.k), up(self.v),
                                self.rope, self.inter, up(self.f) if self.rope else None, out)
        torch.cuda.synchronize()
        return kc, vc, lo, hi, out

    def check(self, kc, vc, lo, hi, out, in_place=False):
        n = lambda t: None if t is None else t.double().numpy()  # noqa: E731
        k_ref, v_ref, q_ref = oracle.attention.append(n(self.kc), n(self.vc), self.table.numpy(), self.past, self.cu, n(self.q),
                                                      n(self.k), n(self.v), n(self.f), bool(self.inter), n(self.ks), n(self.vs))
        # q: untouched rows keep what the output held
        live = np.zeros(self.N, bool)
        for b, p in enumerate(self.past):
            if p >= 0:
                live[self.cu[b]:self.cu[b + 1]] = True
        got = f64(out)
        rest = f64(self.q) if in_place else np.full(got.shape, 9.0)
        assert np.array_equal(got[~live], rest[~live])
        # a rotated value is two fp32 products and a sum of terms of size r = |x| + |y|, with sine and cosine off by
        # 2^-22 (2 ulp) + 2^-30 (angle): off by 2^-21 r; rounding to bf16 is half a step, 2^-8
        rq = np.abs(f64(self.q)).max()
        assert np.all(np.abs(got - q_ref)[live] <= 2.0 ** -8 * np.abs(q_ref[live]) + 2.0 ** -20 * rq)
        # the cache: bf16, or e4m3 (half a step is 2^-4 of the value and 2^-10 in the subnormals), saturated
        for c, c0, ref, x, s in ((kc, self.kc, k_ref, self.k, self.ks), (vc, self.vc, v_ref, self.v, self.vs)):
            g, before = f64(c.float()), f64(self.kc.float() if c is kc else self.vc.float())
            size = np.abs(f64(x)).max() / (1.0 if s is None else float(s.min()))
            if self.dtype == hla.HLA_E4M3:
                ref = np.clip(ref, -448, 448)
                tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10) + 2.0 ** -20 * size
            else:
                tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size
            same = ref == before  # places the append does not reach
            assert np.array_equal(g[same], before[same])
            assert np.all(np.abs(g - ref) <= tol)
        if lo is not None:
            lo_ref, hi_ref = oracle.attention.bounds(f64(kc.float()), f64(self.lo), f64(self.hi), self.table.numpy(), self.past,
                                                     self.cu)
            assert np.array_equal(f64(lo), lo_ref) and np.array_equal(f64(hi), hi_ref)


CASES = [
    dict(past=[0], new=[1], H=1, Hkv=1, d=64, page=16, rope=64),
    dict(past=[0, 15, 16, 17, 31], new=[1, 1, 1, 1, 1], page=16, inter=1),
    dict(past=[60, 61, 62, 63, 64, -1, 500], new=[4] * 7, H=32, Hkv=8),
    dict(past=[5, 100, 0, 7, 63], new=[0, 1, 130, 0, 200], H=6, Hkv=3, d=64, page=32, rope=32, inter=1),
    dict(past=[0, 33], new=[257, 64], H=12, Hkv=4, page=128, rope=64),
    dict(past=[3, 90], new=[17, 1], H=4, Hkv=4, page=64, rope=0, bounds=False),
    dict(past=[100, 20], new=[1, 16], H=10, Hkv=2, d=64, page=16, rope=16),
]


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_matches_oracle(case, dtype):
    a = Append(require_gpu(), dtype=dtype, seed=case, **CASES[case])
    got = a.run()
    assert hla.hla_last_variant().startswith("kv_append<")
    a.check(*got)


def test_append_many_sequences_and_long_prompts():
    """More sequences than a block scans at once, and enough pages and tokens that CTAs take several heads and tokens."""
    dev = require_gpu()
    g = np.random.default_rng(1)
    a = Append(dev, [int(x) for x in g.integers(-1, 90, 300)], [int(x) for x in g.integers(0, 4, 300)], H=4, Hkv=2, d=64, page=16,
               rope=64, seed=2)
    a.check(*a.run())
    a = Append(dev, [10, 0], [3001, 2990], H=4, Hkv=4, d=64, page=16, rope=64, seed=3)
    a.check(*a.run())


def test_largest_batch():
    """1024 sequences through the append and the block choice."""
    dev = require_gpu()
    g = np.random.default_rng(9)
    a = Append(dev, [int(x) for x in g.integers(-1, 60, 1024)], [int(x) for x in g.integers(0, 3, 1024)], H=2, Hkv=1, d=64, page=16,
               rope=64, seed=9)
    a.check(*a.run())
    p = bounded(Problem(dev, [int(x) for x in g.integers(-1, 300, 1024)], 1, 2, 1, 64, 16, seed=9, poison=False), 9)
    select_check(p, 5, 1, 1)


def test_block_choice_keeps_inside_its_buffers():
    dev = require_gpu()
    p = bounded(Problem(dev, [900, -1, 40], 2, 4, 2, 64, 16, seed=11, poison=False), 11)
    n, m = hla.attn_select_blocks_workspace_size(p.C, 3, 2, 4, p.max_blocks), 3 * 2 * 2 * 7
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=dev)
    sel = torch.full((m + 64,), -7, dtype=I32, device=dev)
    hla.attn_select_blocks(p.C, 3, 2, 4, p.max_blocks, p.D["table"], p.D["past"], 7, 1, 1, p.D["q"], sel, ws, n)
    torch.cuda.synchronize()
    assert torch.all(ws[n:] == 0x5A) and torch.all(sel[m:] == -7) and torch.all(sel[:m] >= -1)


def test_append_in_place_and_again():
    """q rotated in its own buffer; the same append twice gives the same cache."""
    dev = require_gpu()
    a = Append(dev, [30, 62], [5, 4], seed=4)
    got = a.run(in_place=True)
    a.check(*got, in_place=True)
    one, two = a.run(), a.run(times=2)
    for x, y in zip(one, two):
        assert torch.equal(bits(x), bits(y))


def test_far_positions_keep_their_angles():
    """At position 2^29 a radian per token leaves fp32 no digit of the angle."""
    dev = require_gpu()
    page, far = 128, 2 ** 29 - 300
    g = inputs.generator(5)
    H, d, N = 2, 64, 3
    q, k = torch.randn(N, H, d, generator=g).to(BF16), torch.randn(N, 1, d, generator=g).to(BF16)
    blocks = far // page + 2
    table = torch.full((1, blocks), -1, dtype=I32, device=dev)
    table[0, far // page:] = torch.tensor([1, 0], dtype=I32)
    kc, vc = (torch.zeros(2, 1, page, d, dtype=BF16, device=dev) for _ in range(2))
    C = hla.make_kv_cache(hla.HLA_BF16, 2, page, 1, d, kc, vc)
    f = torch.cat([freqs(30), torch.tensor([6.0, 0.0], dtype=torch.float64)])
    out = torch.empty_like(q, device=dev)
    hla.kv_cache_append(C, N, 1, torch.tensor([0, N], dtype=I32, device=dev), torch.tensor([far], dtype=I32, device=dev), blocks,
                        table, H, q.to(dev), k.to(dev), k.to(dev), 64, 0, f.to(dev), out)
    for n in range(N):
        # fp64 holds the angle 3e9 to 2^-21 only: compare with the angle taken modulo a turn in exact integers
        turns = [(int(round(x / (2 * np.pi) * 2 ** 80)) * (far + n)) % 2 ** 80 / 2 ** 80 * 2 * np.pi for x in f.tolist()]
        ref = oracle.attention.rotate(q[n].double().numpy(), 1, turns, False)
        # the frequency itself is an fp64 value: its rounding, 2^-53 relative, times 5e8 positions is 2^-22 radian at 6
        assert np.all(np.abs(f64(out[n]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18)


def test_angles_near_quarter_turns():
    """Where a sine or cosine is nearly zero its bf16 value shows the angle's absolute error, here at the positions below 2^31
    that come nearest to a quarter turn (denominators of the continued fraction of quarters per position)."""
    dev = require_gpu()
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    f = [1.0, 0.75, 0.1, 10000.0 ** (-1 / 64), 10000.0 ** (-3 / 8), 6.0, -37.25, 1e-3]
    past = []
    for x in f:
        a, q0, q1 = abs(Fraction(x)) * 2 / pi, 1, 0
        while True:
            whole = a.numerator // a.denominator
            q0, q1 = q1, whole * q1 + q0
            if q1 >= 2 ** 31 - 1:
                break
            past += [q1] * (q1 > 0)
            a = 1 / (a - whole)
    B, d = len(past), 64
    q = torch.zeros(B, 1, d, dtype=BF16)
    q[..., 0:16:2] = 1  # (1, 0) turns to (cos, sin)
    cache = torch.zeros(1, 1, 16, d, dtype=BF16, device=dev)
    C = hla.make_kv_cache(hla.HLA_BF16, 1, 16, 1, d, cache, cache.clone())
    out = torch.empty_like(q, device=dev)
    kv = torch.zeros(B, 1, d, dtype=BF16, device=dev)
    hla.kv_cache_append(C, B, B, torch.arange(B + 1, dtype=I32, device=dev), torch.tensor(past, dtype=I32, device=dev), 1,
                        torch.full((B, 1), -1, dtype=I32, device=dev), 1, q.to(dev), kv, kv, 16, 1,
                        torch.tensor(f, dtype=torch.float64, device=dev), out)
    got, near = f64(out)[:, 0, :16].reshape(B, 8, 2), 0
    for b, pos in enumerate(past):
        for i, x in enumerate(f):
            quarters = Fraction(x) * pos * 2 / pi
            whole = round(quarters)
            rest = float(quarters - whole) * np.pi / 2  # from the nearest quarter turn
            c, s = np.cos(rest), np.sin(rest)
            ref = np.array([(c, s), (-s, c), (-c, -s), (s, -c)][whole % 4])
            near += abs(s) < 1e-5
            # bf16 2^-8, fp32 sine and cosine 2^-21, and 2^-32 of a turn is 1.5e-9 radian, below 2^-29
            assert np.all(np.abs(got[b, i] - ref) <= (2.0 ** -8 + 2.0 ** -21) * np.abs(ref) + 2.0 ** -29), (pos, x, got[b, i], ref)
    assert near > 40


def test_append_drops_tokens_without_a_page_or_behind_the_table():
    dev = require_gpu()
    a = Append(dev, [10, 30, 2], [40, 60, 5], H=4, Hkv=2, d=64, page=16, rope=64, seed=6, max_blocks=4)
    a.table[0, 1], a.table[2, 0] = -1, a.n_pages
    a.check(*a.run())


def test_bounds_forget_rejected_tokens():
    """A rollback (a shorter past) leaves no trace of the rejected keys in the bounds, and a NaN key shows."""
    dev = require_gpu()
    a = Append(dev, [20], [8], H=2, Hkv=2, d=64, page=64, rope=0, seed=7)
    a.k[:8] = 100.0
    kc, vc, lo, hi, _ = a.run()
    assert torch.all(hi[a.table[0, 0]] == 100.0)
    b = Append(dev, [22], [1], H=2, Hkv=2, d=64, page=64, rope=0, seed=7)  # two of the eight were accepted
    b.kc, b.vc, b.lo, b.hi, b.table = kc.cpu(), vc.cpu(), lo.cpu(), hi.cpu(), a.table
    b.k[0] = -50.0
    b.k[0, 1, 3] = float("nan")
    kc, vc, lo, hi, _ = b.run()
    pg = int(a.table[0, 0])
    assert torch.all(lo[pg, 0] == -50.0) and torch.all(hi[pg, 0] == 100.0)
    assert torch.isnan(lo[pg, 1, 3]) and torch.isnan(hi[pg, 1, 3]) and torch.isfinite(lo[pg, 1, :3]).all()


def test_e4m3_saturates():
    dev = require_gpu()
    a = Append(dev, [0], [3], H=2, Hkv=2, d=64, page=16, rope=0, dtype=hla.HLA_E4M3, seed=8)
    a.k[0], a.k[1], a.k[2] = 1e30, float("-inf"), float("nan")
    kc, _, lo, hi, _ = a.run()
    pg = int(a.table[0, 0])
    rows = kc[pg, :, :3].float()
    assert torch.all(rows[:, 0] == 448) and torch.all(rows[:, 1] == -448) and torch.isnan(rows[:, 2]).all()


# ----------------------------------------------------------------------------- block choice


def bounded(p, seed, kind="random"):
    g = inputs.generator(seed + 100)
    shape = (p.n_pages, p.Hkv, p.d)
    mid, wide = torch.randn(shape, generator=g), torch.randn(shape, generator=g).abs()
    p.k_min, p.k_max = (mid - wide).to(BF16), (mid + wide).to(BF16)
    if kind == "equal":          # all blocks alike
        p.k_min[:], p.k_max[:] = p.k_min[0].clone(), p.k_max[0].clone()
    elif kind == "few":          # four kinds of blocks
        n = torch.arange(p.n_pages) % 4
        p.k_min, p.k_max = p.k_min[n].clone(), p.k_max[n].clone()
    elif kind == "zero":
        p.k_min[:], p.k_max[:] = 0, -0.0
    elif kind == "near":         # scores apart by less than fp32 sums hold: large shared parts, small differences
        p.k_min[:], p.k_max[:] = -1e4, 1e4
        p.k_max[:, :, 5] = (torch.randn(p.n_pages, p.Hkv, generator=g) * 2 ** -7).to(BF16)
        p.k_min[:, :, 5] = -p.k_max[:, :, 5]
    elif kind == "strange":
        p.k_max[3, 0, 0], p.k_max[5, :, 1], p.k_min[7, :, 2] = float("nan"), float("inf"), float("-inf")
    elif kind == "huge":
        p.k_min, p.k_max = (p.k_min.float() * 1e37).to(BF16), (p.k_max.float() * 1e37).to(BF16)
    return p.upload()


def select_check(p, n_select, n_first, n_last):
    got = p.select(n_select, n_first, n_last).cpu().numpy()
    ref = oracle.attention.select(p.q.double().numpy(), p.k_min.double().numpy(), p.k_max.double().numpy(), p.table.numpy(), p.past,
                                  p.page, n_select, n_first, n_last)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("kind", ["random", "equal", "few", "zero", "near", "huge"])
@pytest.mark.parametrize("T,H,Hkv,d,page,n_sel,first,last", [(1, 8, 2, 128, 16, 7, 1, 2), (4, 12, 2, 64, 16, 16, 0, 0),
                                                            (2, 40, 2, 128, 32, 3, 1, 1), (8, 16, 1, 64, 16, 9, 0, 1)])
def test_select_matches_oracle(kind, T, H, Hkv, d, page, n_sel, first, last):
    p = Problem(require_gpu(), [1500, 16 * 9 - 1, -1, 3, 700], T, H, Hkv, d, page, seed=T, poison=False)
    select_check(bounded(p, T, kind), n_sel, first, last)


def test_select_with_infinities_and_nan():
    """Scores of +-infinity and NaN: never a hang or a bad index, and the finite rest in order."""
    p = bounded(Problem(require_gpu(), [400], 1, 4, 2, 64, 16, seed=1, poison=False), 1, "strange")
    sel = p.select(6, 0, 1).cpu().numpy()
    for h in range(2):
        row = sel[0, 0, h]
        assert np.all(np.diff(row) > 0) and row[0] >= 0 and row[-1] == 25
    with np.errstate(invalid="ignore"):
        select_check(p, 6, 0, 1)


@pytest.mark.parametrize("blocks", [20, 1500])
def test_blocks_without_a_page_tie_with_scores_of_minus_infinity(blocks):
    """An infinite query channel against negative bounds: every score is -infinity, so the lowest blocks are chosen, those
    without a page among them (few blocks, and more than are listed in shared memory)."""
    p = Problem(require_gpu(), [16 * blocks - 1], 1, 4, 2, 64, 16, seed=12, poison=False)
    p.q[..., 0] = float("inf")
    p.k_min, p.k_max = (torch.randn((p.n_pages, 2, 64), generator=inputs.generator(n)).to(BF16) for n in (1, 2))
    p.k_min, p.k_max = torch.minimum(p.k_min, p.k_max), torch.maximum(p.k_min, p.k_max)
    p.k_min[..., 0], p.k_max[..., 0] = -2.0, -1.0
    p.table[0, 1], p.table[0, 2], p.table[0, 9] = -1, p.n_pages, -7
    p.upload()
    for n, first, last in ((5, 0, 0), (2, 0, 1), (11, 1, 2)):
        select_check(p, n, first, last)


def test_select_extremes():
    dev = require_gpu()
    p = bounded(Problem(dev, [999], 1, 4, 2, 64, 16, seed=2, poison=False), 2)
    select_check(p, 1, 0, 0)
    select_check(p, 62, 0, 0)
    select_check(p, 63, 0, 0)      # every visible block
    select_check(p, 100, 30, 70)
    select_check(p, 10, 10, 0)     # nothing left to choose
    select_check(p, 10, 4, 6)
    # blocks without a page come last
    p.table[0, 3], p.table[0, 40] = -1, p.n_pages
    p.upload()
    select_check(p, 61, 0, 0)
    select_check(p, 62, 0, 0)


@pytest.mark.parametrize("kind", ["random", "equal", "few"])
def test_select_long_rows(kind):
    """More blocks than are kept in shared memory, and more equals than are listed there."""
    p = Problem(require_gpu(), [130000], 1, 8, 1, 64, 16, seed=3, poison=False)
    select_check(bounded(p, 3, kind), 64, 1, 2)


@pytest.mark.parametrize("kind", ["random", "equal", "few", "near", "huge"])
@pytest.mark.parametrize("d,H,Hkv", [(128, 4, 2), (64, 10, 2)])
def test_select_more_rows_than_run_at_once(kind, d, H, Hkv):
    """800 rows, on sequences that share their pages, some with more equals than are listed in shared memory."""
    p = Problem(require_gpu(), [17000], 8, H, Hkv, d, 16, seed=5, poison=False)
    p.B, p.past = 50, [17000 - 340 * b for b in range(50)]
    p.table = p.table.repeat(50, 1)
    p.q = torch.randn((50, 8, H, d), generator=inputs.generator(6)).to(BF16)
    select_check(bounded(p, 5, kind), 24, 1, 2)


# ----------------------------------------------------------------------------- together


@pytest.mark.parametrize("dtype", [hla.HLA_BF16, hla.HLA_E4M3])
def test_decode_loop_with_speculative_windows(dtype):
    """Prompt, then windows of 4 drafted tokens: append, dense and sparse attention, acceptance, and the next window from the
    committed length, which the same array holds for every call.  One graph replays the steps; the keys and values that the
    oracle attends to are rebuilt from the accepted tokens alone."""
    dev = require_gpu()
    B, T, H, Hkv, d, page, blocks = 3, 4, 8, 2, 64, 16, 12
    g = inputs.generator(20)
    n_pages = B * blocks
    store = FP8 if dtype == hla.HLA_E4M3 else BF16
    kc, vc = (torch.zeros(n_pages, Hkv, page, d, dtype=F32, device=dev).fill_(float("nan")).to(store) for _ in range(2))
    lo, hi = (torch.zeros(n_pages, Hkv, d, dtype=BF16, device=dev) for _ in range(2))
    scales = [torch.full((Hkv,), 0.02, device=dev) if dtype == hla.HLA_E4M3 else None for _ in range(2)]
    C = hla.make_kv_cache(dtype, n_pages, page, Hkv, d, kc, vc, *scales, lo, hi)
    table = torch.randperm(n_pages, generator=g).to(I32).view(B, blocks).to(dev)
    f = freqs(d // 2).to(dev)
    committed = torch.zeros(B, dtype=I32, device=dev)

    def tokens(n):
        return [torch.randn(n, h, d, generator=g).to(BF16) for h in (H, Hkv, Hkv)]

    # prompts of 60, 1 and 37 tokens in one ragged append
    lens = [60, 1, 37]
    cu = torch.tensor([0, 60, 61, 98], dtype=I32, device=dev)
    q, k, v = tokens(98)
    q_rot = torch.empty(98, H, d, dtype=BF16, device=dev)
    hla.kv_cache_append(C, 98, B, cu, committed, blocks, table, H, q.to(dev), k.to(dev), v.to(dev), d, 0, f, q_rot)
    committed += torch.tensor(lens, dtype=I32, device=dev)
    hist = [[(k[cu[b] + i], v[cu[b] + i]) for i in range(lens[b])] for b in range(B)]

    # one speculative step, captured
    qw, kw, vw = (torch.zeros(B * T, h, d, dtype=BF16, device=dev) for h in (H, Hkv, Hkv))
    cu_w = torch.arange(0, B * T + 1, T, dtype=I32, device=dev)
    draft, target = (torch.zeros(B, T, dtype=I32, device=dev) for _ in range(2))
    accepted = torch.zeros(B, dtype=I32, device=dev)
    dense, sparse = (torch.zeros(B, T, H, d, device=dev) for _ in range(2))
    sel = torch.zeros(B, T, Hkv, 5, dtype=I32, device=dev)
    ws = torch.empty(max(hla.attn_paged_decode_workspace_size(C, B, T, H), hla.attn_paged_sparse_workspace_size(C, B, T, H),
                         hla.attn_select_blocks_workspace_size(C, B, T, H, blocks)), dtype=torch.uint8, device=dev)

    def step():
        hla.kv_cache_append(C, B * T, B, cu_w, committed, blocks, table, H, qw, kw, vw, d, 0, f, qw)
        hla.attn_paged_decode(C, B, T, H, blocks, table, committed, d ** -0.5, qw, dense, hla.HLA_F32, ws, ws.numel())
        hla.attn_select_blocks(C, B, T, H, blocks, table, committed, 5, 1, 2, qw, sel, ws, ws.numel())
        hla.attn_paged_sparse(C, B, T, H, blocks, table, committed, 5, sel, d ** -0.5, qw, sparse, hla.HLA_F32, ws, ws.numel())
        hla.spec_accept_prefix(B, T, draft, target, accepted, committed)

    graph, first = torch.cuda.CUDAGraph(), True
    for it in range(6):
        q, k, v = tokens(B * T)
        past = committed.cpu().numpy().copy()
        take = [(it * 2 + b) % (T + 1) for b in range(B)]
        for dst, src in ((qw, q), (kw, k), (vw, v)):
            dst.copy_(src)
        target.zero_()
        draft.copy_(torch.tensor([[0 if t < take[b] else 1 for t in range(T)] for b in range(B)], dtype=I32))
        if first:
            with torch.cuda.graph(graph):
                hla.hla_chain_begin()  # the step's calls as one launch chain
                try:
                    step()
                finally:
                    hla.hla_chain_end()
            first = False
        graph.replay()
        torch.cuda.synchronize()
        assert committed.cpu().tolist() == [int(past[b]) + take[b] for b in range(B)]
        chosen = sel.cpu().numpy()
        for b in range(B):
            window = [(k[b * T + t], v[b * T + t]) for t in range(T)]
            seq = hist[b] + window
            scale = 1.0 if dtype == hla.HLA_BF16 else 0.02
            rounded = (lambda x: oracle.numerics.round_bf16(x)) if dtype == hla.HLA_BF16 else oracle.attention.e4m3_round
            keys = np.stack([rounded(oracle.attention.rotate(x[0].double().numpy(), n, f.cpu().numpy(), False) / scale) * scale
                             for n, x in enumerate(seq)])
            vals = np.stack([rounded(x[1].double().numpy() / scale) * scale for x in seq])
            for t in range(T):
                n = int(past[b]) + t + 1
                qq = oracle.numerics.round_bf16(oracle.attention.rotate(q[b * T + t].double().numpy(), n - 1, f.cpu().numpy(), False))
                for h in range(H):
                    hk = h // (H // Hkv)
                    seen = np.zeros(n, bool)
                    for j in chosen[b, t, hk]:
                        if j >= 0:
                            seen[j * page:(j + 1) * page] = True
                    for got, rows in ((dense, np.ones(n, bool)), (sparse, seen)):
                        s = np.exp((keys[:n, hk] @ qq[h]) * d ** -0.5)[rows]
                        ref = (s / s.sum()) @ vals[:n, hk][rows]
                        # a rotated value near a rounding border may be stored a step away on either side: a bf16 step is 2^-7,
                        # an e4m3 step 2^-3 of one key channel in rare places
                        err = np.abs(got[b, t, h].cpu().double().numpy() - ref).max()
                        assert err < (2e-2 if dtype == hla.HLA_BF16 else 8e-2), (it, b, t, h, err)
                # the sparse choice covers the first and the last two blocks
                for hk in range(Hkv):
                    have = [j for j in chosen[b, t, hk] if j >= 0]
                    nb = (n - 1) // page + 1
                    assert len(have) == min(5, nb) and have == sorted(have) and 0 in have and nb - 1 in have
            hist[b] += window[:take[b]]
