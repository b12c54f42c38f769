"""Float64 definition of the paged cache and the attention over it (oracle).

TEST INFRASTRUCTURE ONLY -- see the package docstring.  A cache is a pool
[pages, page_size, Hkv, d] with a page table and lengths per sequence; an e4m3
pool's vectors stand for value * 2^(byte - 127).  Everything is written token
by token.
"""

from __future__ import annotations

import math

import numpy as np

from .attention import FAST, EXPERT


def e4m3_grid() -> np.ndarray:
    """The non-negative finite e4m3 values, in order of their bit patterns."""
    out = []
    for bits in range(0x7F):                      # 0x7F is NaN
        e, m = bits >> 3, bits & 7
        out.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


def to_e4m3(x: np.ndarray) -> np.ndarray:
    """Each |x| <= 448 rounded to the nearest e4m3 value, ties to the even pattern."""
    grid = e4m3_grid()
    a = np.abs(np.asarray(x, np.float64))
    hi = np.searchsorted(grid, a).clip(max=len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.copysign(grid[np.where(up, hi, lo)], x)


def exponent(vec: np.ndarray) -> int:
    """The smallest e >= -126 with max |vec| <= 448 * 2^e (0 for a zero vector)."""
    top = float(np.max(np.abs(vec))) if len(vec) else 0.0
    if top == 0.0:
        return 0
    e = -126
    while top > math.ldexp(448.0, e):
        e += 1
    return e


def quantise(vec: np.ndarray):
    """(e4m3 values, exponent byte) of one finite vector.  e = 120 is the largest
    that 32-bit floats reach; 256 * 2^120 is out of their range: 240 is taken."""
    e = exponent(vec)
    y = to_e4m3(np.asarray(vec, np.float64) * 2.0 ** -e)
    return np.clip(y, -240, 240) if e == 120 else y, e + 127


def positions(lens, S, mask=None):
    """[B, S] position of every valid new token (-1: not stored)."""
    B = len(lens)
    pos = np.full((B, S), -1, np.int64)
    for b in range(B):
        at = int(lens[b])
        row = None if mask is None else (mask if np.ndim(mask) == 1 else mask[b])
        for t in range(S):
            if row is None or row[t]:
                pos[b, t] = at
                at += 1
    return pos


def slot(table, b, x, page_size):
    return int(table[b][x // page_size]) * page_size + x % page_size


def rows(pool, exps, table, b, n):
    """Sequence b's first n cached vectors, [n, Hkv, d] in float64."""
    ps = pool.shape[1]
    at = np.array([slot(table, b, x, ps) for x in range(n)], np.int64)
    out = pool.reshape(-1, *pool.shape[2:])[at].astype(np.float64)
    if exps is not None:
        byte = exps.reshape(-1, exps.shape[2])[at].astype(np.int64)
        out = out * np.ldexp(1.0, byte - 127)[..., None]
    return out


def visible(n, i, x, codes, window, sinks):
    """Whether new token i sees the key at position x (cached when x < n).
    codes: (block index, segment id) of the new tokens."""
    ci, si = codes[i]
    if si < 0:
        return False
    if x >= n:
        cj, sj = codes[x - n]
        if sj < 0 or cj > ci or (si == EXPERT and sj == FAST):
            return False
    return window <= 0 or (n + i) - x < window or x < sinks


def mask(n, Sq, codes, window, sinks):
    """The [Sq, n + Sq] matrix of ``visible``, by whole rows."""
    cs = np.array([c for c, _ in codes]).reshape(Sq)
    sg = np.array([g for _, g in codes]).reshape(Sq)
    new = cs[None, :] <= cs[:, None]
    new &= ~((sg[:, None] == EXPERT) & (sg[None, :] == FAST)) & (sg[None, :] >= 0)
    see = np.concatenate([np.ones((Sq, n), bool), new], 1)
    see[sg < 0] = False
    if window > 0:
        x = np.arange(n + Sq)
        see &= ((n + np.arange(Sq))[:, None] - x[None, :] < window) | (x < sinks)[None, :]
    return see


def attend(q, k_new, v_new, k_rows, v_rows, ar, seg=None, scale=1.0, window=0, sinks=0):
    """out [B,Sq,Hq,d] and lse [B,Sq,Hq] from per-sequence cached rows (lists of
    [n_b, Hkv, d]); rows without a visible key give 0 and -inf."""
    B, Sq, Hq, d = q.shape
    Hkv = k_new.shape[2]
    out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for b in range(B):
        a = np.asarray(ar if np.ndim(ar) == 1 else ar[b])
        s = np.zeros(Sq, np.int64) if seg is None else np.asarray(seg if np.ndim(seg) == 1 else seg[b])
        codes = list(zip(np.cumsum(a != 0).tolist(), s.tolist()))
        n = k_rows[b].shape[0]
        keys = np.concatenate([k_rows[b], k_new[b]])
        vals = np.concatenate([v_rows[b], v_new[b]])
        sees = mask(n, Sq, codes, window, sinks)
        live = sees.any(1)
        vals = np.where(sees.any(0)[:, None, None], vals, 0)     # stale rows may hold NaN
        for h in range(Hq):
            g = h // (Hq // Hkv)
            with np.errstate(invalid="ignore", over="ignore"):
                x = np.where(sees, scale * (q[b, :, h] @ keys[:, g].T), -np.inf)
            m = np.where(live, x.max(1), 0)
            w = np.exp(x - m[:, None])
            z = np.where(live, w.sum(1), 1)
            out[b, :, h] = (w @ vals[:, g]) / z[:, None]
            lse[b, :, h] = np.where(live, m + np.log(z), -np.inf)
    return out, lse
