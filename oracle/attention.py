"""Softmax attention over a paged key-value cache, its append with rotation, and block choice by key bounds.

Test infrastructure only (see ``oracle/__init__``).  float64 throughout.

"Kimi K3: From Day-0 Availability to Optimized Inference" (webinar summary), opening paragraph: next to KDA's
fixed-size state the model's other layers keep an attention cache that grows with the sequence.  The page gives
no layout; the one here is a pool of pages and a table of pages per sequence.

Arrays: k, v [n_pages, Hkv, P, d] as the values the cache stands for (scales applied by the caller); table
[B, max_blocks]; past [B]; q [B, T, H, d].  A position holds a key when its block has a table entry in
[0, n_pages).
"""

import numpy as np

from .numerics import f64

E4M3_MAX = 448.0


def e4m3_values():
    """The 127 non-negative e4m3 values in order: 4 exponent bits (bias 7), 3 mantissa bits, no infinity."""
    out = []
    for bits in range(0x7F):
        e, m = bits >> 3, bits & 7
        out.append(m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
    return np.array(out)


def e4m3_round(x):
    """Nearest e4m3 value, ties to the even mantissa, saturating; NaN stays NaN."""
    x = f64(x)
    v = e4m3_values()
    a = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.clip(np.searchsorted(v, np.where(np.isnan(a), 0.0, a)), 1, len(v) - 1)
    lo = hi - 1
    below, above = a - v[lo], v[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    r = np.where(up, v[hi], v[lo])
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def rotate(x, pos, inv_freq, interleaved):
    """x [..., d] at position pos: its first 2 len(inv_freq) channels turned pair by pair."""
    x = f64(x).copy()
    n = len(inv_freq)
    a = float(pos) * f64(inv_freq)
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    u, w = x[..., first].copy(), x[..., second].copy()
    x[..., first] = u * np.cos(a) - w * np.sin(a)
    x[..., second] = u * np.sin(a) + w * np.cos(a)
    return x


def append(k_cache, v_cache, table, past, cu, q, k, v, inv_freq, interleaved, k_scale=None, v_scale=None):
    """The stored (unscaled) values and q after an append, before any rounding; inputs are not modified."""
    k_cache, v_cache, q_out = (f64(x).copy() for x in (k_cache, v_cache, q))
    n_pages, Hkv, P, _ = k_cache.shape
    ks = np.ones(Hkv) if k_scale is None else f64(k_scale)
    vs = np.ones(Hkv) if v_scale is None else f64(v_scale)
    for b in range(len(past)):
        for i in range(int(cu[b + 1] - cu[b]) if past[b] >= 0 else 0):
            row, pos = int(cu[b]) + i, int(past[b]) + i
            q_out[row] = rotate(q[row], pos, inv_freq, interleaved)
            if pos // P < table.shape[1] and 0 <= table[b, pos // P] < n_pages:
                pg = int(table[b, pos // P])
                k_cache[pg, :, pos % P] = rotate(k[row], pos, inv_freq, interleaved) / ks[:, None]
                v_cache[pg, :, pos % P] = f64(v[row]) / vs[:, None]
    return k_cache, v_cache, q_out


def bounds(k_cache, k_min, k_max, table, past, cu):
    """Key bounds after an append that left the stored keys k_cache: touched pages only, valid rows only."""
    k_min, k_max = f64(k_min).copy(), f64(k_max).copy()
    n_pages, _, P, _ = k_cache.shape
    for b in range(len(past)):
        n = int(cu[b + 1] - cu[b])
        if past[b] < 0 or n <= 0:
            continue
        for j in range(int(past[b]) // P, (int(past[b]) + n - 1) // P + 1):
            if j < table.shape[1] and 0 <= table[b, j] < n_pages:
                rows = f64(k_cache[int(table[b, j]), :, :min(P, int(past[b]) + n - j * P)])
                k_min[int(table[b, j])], k_max[int(table[b, j])] = rows.min(1), rows.max(1)
    return k_min, k_max


def _row(q, keys, values, scale):
    """softmax(scale q.k) v over the listed keys, and sum of weight x |value| (for error bounds); zeros for none."""
    if len(keys) == 0:
        return np.zeros(values.shape[-1]), np.zeros(values.shape[-1])
    s = scale * (keys @ q)
    w = np.exp(s - s.max())
    w /= w.sum()
    return w @ values, w @ np.abs(values)


def attend(q, k, v, table, past, scale, sel=None):
    """o [B, T, H, d] of the T newest tokens, and the same sums over |v|.  sel [B, T, Hkv, n]: listed blocks only,
    and of a list no more entries than the token sees blocks."""
    q, k, v = f64(q), f64(k), f64(v)
    B, T, H, d = q.shape
    n_pages, Hkv, P, _ = k.shape
    o, mag = np.zeros((B, T, H, d)), np.zeros((B, T, H, d))
    for b in range(B):
        if past[b] < 0:
            continue
        for t in range(T):
            last = int(past[b]) + t
            for hk in range(Hkv):
                blocks = range(min(table.shape[1], last // P + 1)) if sel is None else \
                    [j for j in sel[b, t, hk][:last // P + 1] if 0 <= j < table.shape[1]]
                rows = [(int(table[b, j]), r) for j in blocks if 0 <= table[b, j] < n_pages
                        for r in range(P) if j * P + r <= last]
                pg, r = np.array([x[0] for x in rows], int), np.array([x[1] for x in rows], int)
                keys, values = k[pg, hk, r].reshape(-1, d), v[pg, hk, r].reshape(-1, d)
                for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
                    o[b, t, h], mag[b, t, h] = _row(q[b, t, h], keys, values, scale)
    return o, mag


def block_scores(q, k_min, k_max):
    """Bound score of each block for one kv head: q [G, d], k_min, k_max [n, d] -> [n]."""
    q, lo, hi = f64(q), f64(k_min), f64(k_max)
    s = np.maximum(q, 0) @ hi.T + np.minimum(q, 0) @ lo.T
    return np.max(s, axis=0)


def select(q, k_min, k_max, table, past, P, n_select, n_first, n_last):
    """sel [B, T, Hkv, n_select]: chosen blocks in ascending order, -1 behind them."""
    q = f64(q)
    B, T, H, d = q.shape
    n_pages, Hkv, _ = k_min.shape
    G = H // Hkv
    out = np.full((B, T, Hkv, n_select), -1, dtype=np.int64)
    for b in range(B):
        if past[b] < 0:
            continue
        for t in range(T):
            nb = min(table.shape[1], (int(past[b]) + t) // P + 1)
            for hk in range(Hkv):
                if nb <= n_select:
                    out[b, t, hk, :nb] = np.arange(nb)
                    continue
                pg = table[b, :nb]
                has = (pg >= 0) & (pg < n_pages)
                s = np.full(nb, -np.inf)
                s[has] = block_scores(q[b, t, hk * G:(hk + 1) * G], k_min[pg[has], hk], k_max[pg[has], hk])
                forced = [j for j in range(nb) if j < n_first or j >= nb - n_last]
                rest = sorted((j for j in range(nb) if j not in forced), key=lambda j: (not np.isnan(s[j]), 0.0 if np.isnan(s[j]) else -s[j], j))
                out[b, t, hk] = sorted(forced + rest[:n_select - len(forced)])
    return out
