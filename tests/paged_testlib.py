"""Plain 64-bit forms of the paged cache's operators (numpy), for its tests."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every non-negative finite E4M3 value in order of its byte
SCALES = np.array([m * 2.0 ** -9 for m in range(8)]
                  + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]


def nearest(x, grid):
    """Index of the nearest grid value, ties to the even index; past the end, the last."""
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)


def quantize(x, exp=0):
    """The stored values (float64) of x [..., D], groups of 16 channels."""
    x = np.asarray(x, np.float64) * 2.0 ** -exp
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    g = np.where(np.isnan(g), 0.0, g)
    top = np.minimum(np.abs(g).max(-1, keepdims=True), 1e30)
    s = SCALES[nearest(top / 6, SCALES)]
    y = np.minimum(np.abs(g), 1e30) / np.where(s > 0, s, 1.0)
    v = np.where(s > 0, LEVELS[nearest(y, LEVELS)] * s, 0.0) * np.where(g < 0, -1.0, 1.0)
    return v.reshape(x.shape) * 2.0 ** exp


def attention(q, k, v, n, scale, window):
    """q [n, Hq, D] the last n of k, v [T, Hkv, D] (float64).  out, lse and what the tolerances
    need: sum p |v| and the largest sum |q k| of a row."""
    T, Hkv, D = k.shape
    Hq = q.shape[1]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    pv, qk = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n):
        p = T - n + i
        lo = max(0, p - window + 1) if window else 0
        if p < 0:
            continue
        for h in range(Hq):
            kk, vv = k[lo:p + 1, h * Hkv // Hq], v[lo:p + 1, h * Hkv // Hq]
            x = kk @ q[i, h] * scale
            m = x.max()
            e = np.exp(x - m)
            lse[i, h] = m + np.log(e.sum())
            w = e / e.sum()
            out[i, h], pv[i, h] = w @ vv, w @ np.abs(vv)
            qk[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, pv, qk


def plan(lens, n_new, table, free, n_free, P, width, capacity):
    """The page plan, request by request.  table is changed in place."""
    cu, slots, pos, out, status = [0], np.full(capacity, -1), np.zeros(capacity, int), [], 0
    left = n_free
    for b, (a, n) in enumerate(zip(lens, n_new)):
        cu.append(cu[-1] + n)
        have, want = -(-a // P), -(-(a + n) // P)
        if want > width or cu[-1] > capacity:
            ok, status = False, status | 2
            if want <= width and want > have:
                left = min(left, 0) if want - have > left else left - (want - have)
        elif want - have > left and want > have:
            ok, status, left = False, status | 64, -1
        else:
            ok = True
            for j in range(have, want):
                left -= 1
                table[b, j] = free[left]
        out.append(a + n if ok else a)
        for i in range(n):
            if cu[b] + i < capacity:
                pos[cu[b] + i] = a + i
                if ok:
                    slots[cu[b] + i] = table[b, (a + i) // P] * P + (a + i) % P
    used = sum(-(-o // P) - -(-a // P) for o, a in zip(out, lens))
    return cu, out, slots, pos, n_free - used, status
