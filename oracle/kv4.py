"""fp64 oracle of the paged 4-bit KV cache -- TEST INFRASTRUCTURE.

Only the tests may import this module; nothing here is shared with the CUDA
path.  Plain numpy, one value at a time in meaning: formats are tables of all
their values, rounding is a search for the nearest (ties to the even code),
the page operations are sequential loops over Python lists.

Layout of a unit (16 positions of one KV head, 18 D bytes), as documented in
include/fa_gb300.h: K codes [16][D/2] (low nibble = even dimension), V codes
[2][D/16][4][16] (low nibble = even position of the pair), K scales
[16][D/16], V scales [D/16][16].
"""
from __future__ import annotations

import numpy as np

UNIT = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)) for e in range(16) for f in range(8)][:127])


def nearest(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Index of the value nearest to each x >= 0 (ties to the even index; beyond the last: the last)."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    dlo, dhi = x - values[lo], values[hi] - x
    take_hi = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo)


def quantise(x: np.ndarray, head_scale: np.ndarray):
    """x [T, H, D] fp64 -> (codes uint8 [T, H, D], scale bytes uint8 [T, H, D/16])."""
    T, H, D = x.shape
    x = (x / head_scale[None, :, None]).reshape(T, H, D // 16, 16)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    sb = nearest(np.minimum(np.abs(x).max(-1) / 6, 448.0), E4M3)
    s = E4M3[sb][..., None]
    y = np.where(s > 0, x / np.where(s > 0, s, 1.0), 0.0)
    codes = nearest(np.abs(y), E2M1) + 8 * (y < 0)  # a zero of either sign has code 0
    return codes.reshape(T, H, D).astype(np.uint8), np.where(bad, 0x7f, sb).astype(np.uint8)


def _scale(b: np.ndarray) -> np.ndarray:
    table = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])
    return table[b]


def _value(c: np.ndarray) -> np.ndarray:
    return np.concatenate([E2M1, -E2M1])[c]


def write_row(unit: np.ndarray, key: int, D: int, kc, ks, vc, vs):
    """Stores one position's codes and scales into its unit (uint8 [18 D])."""
    unit[key * (D // 2):(key + 1) * (D // 2)] = kc[0::2] | kc[1::2] << 4
    d = np.arange(D)
    at = 8 * D + key // 8 * 4 * D + d // 16 * 64 + key % 8 // 2 * 16 + d % 16
    unit[at] = (unit[at] & 0x0f | vc << 4) if key % 2 else (unit[at] & 0xf0 | vc)
    unit[16 * D + key * (D // 16):16 * D + (key + 1) * (D // 16)] = ks
    unit[17 * D + np.arange(D // 16) * 16 + key] = vs


def unit_rows(units: np.ndarray, D: int):
    """K and V values [..., 16, D] of units [..., 18 D], without head scales."""
    lead = units.shape[:-1]
    kc = units[..., :8 * D].reshape(*lead, 16, D // 2)
    k = np.empty((*lead, 16, D))
    k[..., 0::2], k[..., 1::2] = _value(kc & 15), _value(kc >> 4)
    k *= np.repeat(_scale(units[..., 16 * D:17 * D]).reshape(*lead, 16, D // 16), 16, -1)
    v = np.empty((*lead, 16, D))
    vc = units[..., 8 * D:16 * D].reshape(*lead, 2, D // 16, 4, 16)
    vs = _scale(units[..., 17 * D:]).reshape(*lead, D // 16, 16)
    for key in range(16):
        byte = vc[..., key // 8, :, key % 8 // 2, :]
        x = _value(byte >> 4 if key % 2 else byte & 15)
        v[..., key, :] = (x * vs[..., key][..., None]).reshape(*lead, D)
    return k, v


def append(pool, table, lens, slots, counts, k, v, k_scale, v_scale):
    """Writes packed rows k, v [T, H, D] as the last counts[i] positions of slots[i] (pool changed in place)."""
    _, H, U, unit = pool.shape
    D, P = unit // 18, U * 16
    kc, ks = quantise(k, k_scale)
    vc, vs = quantise(v, v_scale)
    row = 0
    for s, n in zip(slots, counts):
        for pos in range(lens[s] - n, lens[s]):
            for h in range(H):
                write_row(pool[table[s][pos // P], h, pos % P // 16], pos % 16, D, kc[row, h], ks[row, h], vc[row, h],
                          vs[row, h])
            row += 1


def rows(pool, table, slot, length, k_scale, v_scale):
    """K and V [H, length, D] of one sequence, fp64."""
    _, H, U, unit = pool.shape
    D, P = unit // 18, U * 16
    if length == 0:
        return np.zeros((H, 0, D)), np.zeros((H, 0, D))
    pages = pool[np.asarray(table[slot][:-(-length // P)])]  # [n, H, U, unit]
    k, v = unit_rows(pages.transpose(1, 0, 2, 3), D)
    return (k.reshape(H, -1, D)[:, :length] * k_scale[:, None, None],
            v.reshape(H, -1, D)[:, :length] * v_scale[:, None, None])


def attention(q, k, v, scale, causal):
    """q [Hq, Lq, D], k, v [Hkv, L, D] fp64 -> O [Hq, Lq, D], LSE [Hq, Lq].  Masked keys take no part at all."""
    Hq, Lq, D = q.shape
    Hkv, L, _ = k.shape
    o, lse = np.zeros((Hq, Lq, D)), np.full((Hq, Lq), -np.inf)
    for h in range(Hq):
        kk, vv = k[h // (Hq // Hkv)], v[h // (Hq // Hkv)]
        for i in range(Lq):
            n = min(L, max(0, i + L - Lq + 1)) if causal else L
            if n == 0:
                continue
            s = kk[:n] @ q[h, i] * scale
            m = s.max()
            p = np.exp(s - m)
            lse[h, i] = m + np.log(p.sum())
            o[h, i] = p @ vv[:n] / p.sum()
    return o, lse


class Pages:
    """Sequential model of the page operations."""

    def __init__(self, num_pages, slots, width, page_size):
        self.P, self.width = page_size, width
        self.table = [[-1] * width for _ in range(slots)]
        self.lens = [0] * slots
        self.refs = [0] * num_pages

    def _pages(self, n):
        return -(-n // self.P)

    def _free(self):
        return [i for i, r in enumerate(self.refs) if r == 0]

    def reserve(self, slots, new):
        free = self._free()
        used = [s for s, a in zip(slots, new) if a]  # a slot may be named again with 0 tokens
        if len(set(used)) < len(used) or any(not 0 <= s < len(self.lens) for s in slots):
            return len(free), -1
        for s, a in zip(slots, new):
            end = self.lens[s] + a
            if not 0 <= end <= self.P * self.width:
                return len(free), -1
            # positions taken back: the page that the end comes to lie in must be the sequence's own
            if a < 0 and end % self.P and self.refs[self.table[s][end // self.P]] != 1:
                return len(free), -1
        need = [max(0, self._pages(self.lens[s] + a) - self._pages(self.lens[s])) for s, a in zip(slots, new)]
        if sum(need) > len(free):
            return len(free), sum(need) - len(free)
        for s, a, c in zip(slots, new, need):
            at = self._pages(self.lens[s])
            for j in range(c):
                page = free.pop(0)
                self.table[s][at + j] = page
                self.refs[page] = 1
            for j in range(self._pages(self.lens[s] + a), at):
                self.refs[self.table[s][j]] -= 1
                self.table[s][j] = -1
            self.lens[s] += a
        return len(self._free()), 0

    def fork(self, parents, children, pool=None):
        free = self._free()
        slots = range(len(self.lens))
        if (len(set(children)) < len(children) or set(parents) & set(children)
                or any(c not in slots or self.lens[c] for c in children) or any(s not in slots for s in parents)):
            return len(free), -1
        need = sum(1 for s in parents if self.lens[s] % self.P)
        if need > len(free):
            return len(free), need - len(free)
        for s, c in zip(parents, children):
            full, rest = divmod(self.lens[s], self.P)
            self.table[c] = self.table[s][:full] + [-1] * (self.width - full)
            for page in self.table[s][:full]:
                self.refs[page] += 1
            if rest:
                page = free.pop(0)
                self.table[c][full] = page
                self.refs[page] = 1
                if pool is not None:  # [layers, pages, H, U, unit]
                    pool[:, page, :, :-(-rest // 16)] = pool[:, self.table[s][full], :, :-(-rest // 16)]
            self.lens[c] = self.lens[s]
        return len(free), 0

    def release(self, slots):
        for s in slots:
            for page in self.table[s][:self._pages(self.lens[s])]:
                self.refs[page] -= 1
            if self.lens[s] or s in slots:
                self.table[s] = [-1] * self.width
            self.lens[s] = 0

    def compact(self, pool=None):
        live = [i for i, r in enumerate(self.refs) if r]
        to = dict(zip([i for i in live if i >= len(live)], [i for i in self._free() if i < len(live)]))
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            if pool is not None:
                pool[:, b] = pool[:, a]
        for s, n in enumerate(self.lens):
            for j in range(self._pages(n)):
                self.table[s][j] = to.get(self.table[s][j], self.table[s][j])
        return len(self.refs) - len(live), 0
