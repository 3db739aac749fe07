"""fp64 reference of rotary positions and of the paged bf16 KV cache (numpy; test infrastructure only).

Written from the definitions in include/fa_gb300.h: a cache is read back position by position through its table, trees
are sets of ancestors, and attention is one softmax over the keys that a row may see.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

PER_TURN = Fraction("0.159154943091895335768883763372514362034459645740456448747667344")  # 1 / (2 pi)


def angles(pos, w):
    """pos * w modulo a turn [T, pairs]: the product in integers (2^-96 of a turn), as fp64 loses it at far positions."""
    turns = np.array([round(Fraction(float(x)) * PER_TURN * 2 ** 96) for x in w], dtype=object)
    part = np.asarray(pos).astype(object)[:, None] * turns % 2 ** 96
    return 2 * np.pi * (part >> 32).astype(np.float64) / 2.0 ** 64


def turn(x, pos, w, mscale=1.0, start=0, interleaved=False, back=False):
    """Rows x [T, H, D] at positions pos [T] turned (``back``: the gradient)."""
    x = np.asarray(x, np.float64)
    theta = angles([int(p) for p in pos], w)[:, None]
    z = mscale * np.exp((-1j if back else 1j) * theta)
    c = np.arange(len(w))
    first = start + (2 * c if interleaved else c)
    second = first + (1 if interleaved else len(w))
    y = x.copy()
    z = (x[..., first] + 1j * x[..., second]) * z
    y[..., first], y[..., second] = z.real, z.imag
    return y


def turn_tolerance(x, y, mscale, w_dims, bf16):
    """Bound on the error of a turned row: the angle's part of a turn is rounded to 24 bits (pi 2^-25), sine and cosine
    to 2 steps (2^-23), times m and the two products and the sum to half a step each (2^-24): below 2^-21 of |x1| +
    |x2|, which 2 max|x| of the row bounds; bf16 rounds by half a step, 2^-8 of the value."""
    big = 2 * np.abs(x).max(-1, keepdims=True) * mscale
    return 2.0 ** -21 * big + (2.0 ** -8 * np.abs(y) if bf16 else 0.0) + 2.0 ** -133


def rows(pool, table, slot, n):
    """K and V of the first n positions of a slot, [n, Hkv, D] each; pool [pages, 2, Hkv, P, D] in fp64."""
    P = pool.shape[3]
    p = np.arange(n)
    page = table[slot][p // P]
    return pool[page, 0, :, p % P], pool[page, 1, :, p % P]


def ancestors(parents):
    """Truth values [n, n]: node i sees j (its ancestors and itself)."""
    n = len(parents)
    see = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            see[i] = see[p]
        see[i, i] = True
    return see


def attention(q, k, v, scale, own):
    """q [n, Hq, D] over k, v [L, Hkv, D]; own [n, n]: what the rows see of the last n positions.  Returns O, LSE
    [Hq, n] and sum_j p_ij |v_j| / sum_j p_ij, which the error bound needs.  Keys and values that a row may not see do
    not enter its sums at all."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    o, mag = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse = np.full((Hq, n), -math.inf)
    for i in range(n):
        keys = np.concatenate([np.arange(L - n), L - n + np.nonzero(own[i])[0]])
        if not len(keys):
            continue
        for h in range(H):
            hq = slice(h * Hq // H, (h + 1) * Hq // H)
            s = scale * (q[i, hq] @ k[keys, h].T)
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(-1, keepdims=True)
            o[i, hq] = (p / total) @ v[keys, h]
            mag[i, hq] = (p / total) @ np.abs(v[keys, h])
            lse[hq, i] = (top + np.log(total))[:, 0]
    return o, lse, mag


def attention_tolerance(q, k, scale, o, lse, mag):
    """Bounds on |O - O_ref| and |LSE - LSE_ref| from the kernel's arithmetic.

    A score sums D products, exact in fp32, with at most D truncating additions (2^-23 each): ds = D 2^-23 sum|q||k|
    scale, and the exponent's argument (below 2^8 in log2 units above the reference, any size below, where the
    weight vanishes as fast) loses 2^-23 of min(2^8, 4 |s| + 1) more.  2^x is good to 2^-21 and a sum of L terms to
    L 2^-24.  P is rounded to bf16 by 2^-8 of itself, in the numerator and, unless it is the tile's largest, not in
    the denominator: 2 * 2^-8 of sum p |v|.  O is rounded by 2^-8 of itself."""
    if not len(k):
        return np.zeros_like(o) + 1e-30, 0.0
    qk = (np.abs(q).reshape(-1, q.shape[-1]) @ np.abs(k).reshape(-1, k.shape[-1]).T).max() * scale
    ds = q.shape[-1] * 2.0 ** -23 * qk + min(2.0 ** 8, 4 * qk + 1) * 2.0 ** -23
    rel = ds + len(k) * 2.0 ** -24 + 2.0 ** -21
    fin = np.abs(lse[np.isfinite(lse)])
    tol_lse = rel + 2.0 ** -22 * (fin.max() if len(fin) else 0.0)
    return (2 * 2.0 ** -8 + 2 * rel) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(o) + 1e-30, tol_lse
