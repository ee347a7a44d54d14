"""The fp64 oracle of the paged-cache operators, pinned by hand-worked values, scalar loops and invariants."""

import math

import numpy as np
import pytest

from oracle import attention as at


def test_e4m3_values_and_rounding():
    v = at.e4m3_values()
    assert len(v) == 127 and v[0] == 0.0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[-1] == 448.0
    assert np.all(np.diff(v) > 0)
    assert np.array_equal(at.e4m3_round(v), v) and np.array_equal(at.e4m3_round(-v), -v)
    # 17 is halfway between 16 (mantissa 0, even) and 18; 19 between 18 and 20 (even); 1e9 and inf saturate
    got = at.e4m3_round([17.0, 19.0, 17.01, 1e9, -np.inf, 2.0 ** -10, 3 * 2.0 ** -10])
    assert got.tolist() == [16.0, 20.0, 18.0, 448.0, -448.0, 0.0, 2.0 ** -8]
    assert np.isnan(at.e4m3_round(np.nan))


def test_rotation_by_a_quarter_turn_and_its_pairings():
    x = np.arange(1.0, 7.0)  # 4 rotated channels, 2 left alone
    f = [math.pi / 2, math.pi]
    # half pairs (0, 2), (1, 3): position 1 turns the first by 90 degrees, the second by 180
    assert np.allclose(at.rotate(x, 1, f, False), [-3, -2, 1, -4, 5, 6], atol=1e-15)
    # neighbours (0, 1), (2, 3)
    assert np.allclose(at.rotate(x, 1, f, True), [-2, 1, -3, -4, 5, 6], atol=1e-15)
    assert np.array_equal(at.rotate(x, 0, f, True), x) and np.array_equal(at.rotate(x, 9, [], False), x)
    # a product of two rotated vectors depends on the distance of their positions only
    g = np.random.default_rng(0)
    a, b, f = g.normal(size=8), g.normal(size=8), [0.3, 0.01, 1.7]
    assert math.isclose(at.rotate(a, 107, f, False) @ at.rotate(b, 100, f, False),
                        at.rotate(a, 7, f, False) @ at.rotate(b, 0, f, False), rel_tol=1e-12)


def test_append_places_tokens_and_bounds_valid_rows():
    k = np.full((3, 1, 2, 2), 9.0)  # 3 pages of 2 rows, one head of 2 channels
    v = k.copy()
    table = np.array([[2, 0], [1, -1]])
    new = np.array([[[1.0, -1.0]], [[2.0, -2.0]], [[3.0, 3.0]], [[4.0, 4.0]]])
    # sequence 0: rows 0-1 at positions 1, 2; sequence 1: rows 2-3 at positions 1, 2 (its block 1 has no page)
    past, cu = np.array([1, 1]), np.array([0, 2, 4])
    k2, v2, q2 = at.append(k, v, table, past, cu, new, new, 10 * new, [], False, k_scale=[2.0], v_scale=[1.0])
    assert k2[2, 0].tolist() == [[9, 9], [0.5, -0.5]] and k2[0, 0].tolist() == [[1, -1], [9, 9]]
    assert k2[1, 0].tolist() == [[9, 9], [1.5, 1.5]] and v2[0, 0, 0].tolist() == [20, -20]
    assert np.array_equal(q2, new) and np.all(k == 9)
    lo, hi = at.bounds(k2, np.zeros((3, 1, 2)), np.zeros((3, 1, 2)), table, past, cu)
    assert lo[2, 0].tolist() == [0.5, -0.5] and hi[2, 0].tolist() == [9, 9]   # old row 0 and new row 1
    assert lo[0, 0].tolist() == hi[0, 0].tolist() == [1, -1]                  # row 1 is not valid
    assert lo[1, 0].tolist() == [1.5, 1.5] and hi[1, 0].tolist() == [9, 9]
    idle = at.append(k, v, table, np.array([-1, -1]), cu, new, new, new, [], False)
    assert np.array_equal(idle[0], k) and np.array_equal(idle[2], new)


def test_attend_by_scalar_loops():
    g = np.random.default_rng(1)
    B, T, H, Hkv, d, P = 2, 2, 4, 2, 3, 2
    k, v = g.normal(size=(5, Hkv, P, d)), g.normal(size=(5, Hkv, P, d))
    q = g.normal(size=(B, T, H, d))
    table, past = np.array([[3, 0, 4], [1, 7, 2]]), np.array([3, 3])  # sequence 1's block 1 has no page
    o, mag = at.attend(q, k, v, table, past, 0.7)
    for b in range(B):
        for t in range(T):
            for h in range(H):
                num, den, top = np.zeros(d), 0.0, np.zeros(d)
                for pos in range(past[b] + t + 1):
                    pg = table[b, pos // P]
                    if not 0 <= pg < 5:
                        continue
                    w = math.exp(0.7 * sum(q[b, t, h, c] * k[pg, h // 2, pos % P, c] for c in range(d)))
                    den += w
                    for c in range(d):
                        num[c] += w * v[pg, h // 2, pos % P, c]
                        top[c] += w * abs(v[pg, h // 2, pos % P, c])
                assert np.allclose(o[b, t, h], num / den, rtol=1e-12) and np.allclose(mag[b, t, h], top / den, rtol=1e-12)


def test_attend_special_rows_and_lists():
    g = np.random.default_rng(2)
    k, v = g.normal(size=(4, 1, 2, 3)), g.normal(size=(4, 1, 2, 3))
    q, table = g.normal(size=(1, 1, 2, 3)), np.array([[2, 1, 0]])
    # one key: its value; an idle slot and a listless row: zeros
    assert np.allclose(at.attend(q, k, v, table, np.array([0]), 1.0)[0][0, 0], v[2, 0, 0])
    assert np.all(at.attend(q, k, v, table, np.array([-1]), 1.0)[0] == 0)
    assert np.all(at.attend(q, k, v, table, np.array([5]), 1.0, sel=np.full((1, 1, 1, 3), -1))[0] == 0)
    # all blocks listed, in any order, is the dense form; a block twice weighs double (two copies of its keys)
    dense = at.attend(q, k, v, table, np.array([4]), 1.0)[0]
    assert np.allclose(at.attend(q, k, v, table, np.array([4]), 1.0, sel=np.array([[[[2, 0, 1]]]]))[0], dense)
    twice = at.attend(q, k, v, table, np.array([5]), 1.0, sel=np.array([[[[1, 1, 2]]]]))[0]
    table4 = np.array([[1, 1, 0, 3]])
    assert np.allclose(twice, at.attend(q, k, v, table4, np.array([5]), 1.0)[0])
    # a token that sees two blocks reads two entries
    short = at.attend(q, k, v, table, np.array([3]), 1.0, sel=np.array([[[[0, -1, 1]]]]))[0]
    assert np.allclose(short, at.attend(q, k, v, table, np.array([1]), 1.0)[0])


def test_scores_bound_every_key_and_selection_by_hand():
    g = np.random.default_rng(3)
    keys, q = g.normal(size=(6, 4, 5)), g.normal(size=(2, 5))
    s = at.block_scores(q, keys.min(1), keys.max(1))
    assert np.all(s >= np.einsum("nrd,gd->nrg", keys, q).max((1, 2)) - 1e-12)
    # one channel, q = +-1: the score is kmax of the one head, -kmin of the other, whichever is larger
    assert at.block_scores([[1.0], [-1.0]], [[-3.0], [0.0]], [[1.0], [2.0]]).tolist() == [3.0, 2.0]
    # blocks 0..5 with scores 1 5 5 2 9 0 and 12 positions of page size 2; first and last forced, then 9, then the lower 5
    k_max = np.array([1.0, 5, 5, 2, 9, 0]).reshape(6, 1, 1)
    sel = at.select(np.ones((1, 1, 1, 1)), -k_max, k_max, np.arange(6)[None], np.array([11]), 2, 4, 1, 1)
    assert sel[0, 0, 0].tolist() == [0, 1, 4, 5]
    sel = at.select(np.ones((1, 1, 1, 1)), -k_max, k_max, np.arange(6)[None], np.array([5]), 2, 4, 1, 1)
    assert sel[0, 0, 0].tolist() == [0, 1, 2, -1]
    k_max[3] = np.nan
    sel = at.select(np.ones((1, 1, 1, 1)), k_max, k_max, np.array([[0, 1, 2, 3, -1, 5]]), np.array([11]), 2, 2, 0, 0)
    assert sel[0, 0, 0].tolist() == [1, 3]  # NaN above all, block 4 without a page


@pytest.mark.parametrize("wrong", ["last", "scale", "head"])
def test_attend_pins_catch_planted_mistakes(wrong):
    """The scalar-loop pin tells a shifted mask, a lost scale and a wrong kv head from the definition."""
    g = np.random.default_rng(4)
    k, v, q = g.normal(size=(3, 2, 2, 3)), g.normal(size=(3, 2, 2, 3)), g.normal(size=(1, 1, 4, 3))
    table, past = np.array([[0, 1, 2]]), np.array([3])
    good = at.attend(q, k, v, table, past, 0.5)[0]
    bad = {"last": lambda: at.attend(q, k, v, table, past + 1, 0.5)[0],
           "scale": lambda: at.attend(q, k, v, table, past, 1.0)[0],
           "head": lambda: at.attend(q, k[:, ::-1], v[:, ::-1], table, past, 0.5)[0]}[wrong]()
    assert np.max(np.abs(good - bad)) > 1e-3
