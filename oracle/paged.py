"""Rotary positions with several axes, the paged KV cache and attention over
it, in 64 bits on the host (numpy), written from the definitions in
include/dsa_rope.h and include/dsa_paged.h.
"""
from __future__ import annotations

import numpy as np

E_MIN, E_MAX = -72, 120

# The finite E4M3 values 0 .. 448 of the codes 0x00 .. 0x7e.
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(0x7f)])


def e4m3_encode(x):
    """Codes of x: nearest, ties to the even code, beyond 448 saturated, NaN 0x7f with its sign dropped."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 0x7e)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code |= (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7f), code)


def e4m3_decode(c):
    c = np.asarray(c, dtype=np.uint8)
    m = c & 0x7f
    v = np.where(m == 0x7f, np.nan, E4M3[np.minimum(m, 0x7e)])
    return np.where(c & 0x80, -v, v)


def rope(x, pos, pairs, base=10000.0, restart=False, inverse=False):
    """x [tokens, heads, d] turned at pos [tokens, axes]; angles in extended precision."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    y = x.copy()
    two_pi = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))
    j = 0
    for a, n in enumerate(pairs):
        for i in range(n):
            f = np.longdouble(base ** (-i / n) if restart else base ** (-2.0 * j / d))
            angle = np.fmod(np.asarray(pos)[:, a].astype(np.longdouble) * f, two_pi)
            c, s = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
            if inverse:
                s = -s
            u, w = x[..., j], x[..., j + d // 2]
            y[..., j] = u * c - w * s
            y[..., j + d // 2] = u * s + w * c
            j += 1
    return y


def _smallest(a):
    """The smallest e in [E_MIN, E_MAX] with a <= 448 * 2^e."""
    for e in range(E_MIN, E_MAX):
        if a <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def k_reach(k, rotated):
    """Per row the largest norm of a rotated pair or magnitude of another element (finite ones), the
    squared norm rounded to the 24 bits of fp32 (not to its range) as the definition says."""
    k = np.where(np.isfinite(k), k, 0.0).astype(np.float64)
    h = k.shape[-1] // 2
    sq = (k ** 2)
    both = np.concatenate([sq[..., :rotated] + sq[..., h:h + rotated], sq[..., rotated:h], sq[..., h + rotated:]], -1)
    m, e = np.frexp(both.max(-1))
    return np.sqrt(np.ldexp(m.astype(np.float32).astype(np.float64), e))


def v_reach(v):
    return np.abs(np.where(np.isfinite(v), v, 0.0)).max(-1)


class Cache:
    """The pool and what appends do to it.  `pages` holds codes (uint8) where
    `scales` is given, else fp64 values, unrounded where they were appended."""

    def __init__(self, pages, scales=None):
        self.pages = np.array(pages)
        self.scales = None if scales is None else np.array(scales, dtype=np.float64)
        self.page = self.pages.shape[2]

    def append(self, kr, k, v, cu, lens, table, rotated=0):
        """kr: the rotated keys [tokens, kv_heads, d]; k: as given (their norms set the scales).
        Returns the exact values stored ([tokens, kv_heads, 2, d]), for comparison within a rounding."""
        for s in range(len(lens)):
            n, at = cu[s + 1] - cu[s], lens[s] - (cu[s + 1] - cu[s])
            t = cu[s]
            while n > 0:
                pid, slot = table[s][at // self.page], at % self.page
                m = min(n, self.page - slot)
                rows = np.stack([kr[t:t + m], v[t:t + m]], 2).transpose(1, 0, 2, 3)
                if self.scales is None:
                    self.pages[pid, :, slot:slot + m] = rows
                else:
                    for h in range(k.shape[1]):
                        for i, top in ((0, k_reach(k[t:t + m, h], rotated).max()), (1, v_reach(v[t:t + m, h]).max())):
                            new = 2.0 ** _smallest(top)
                            old = self.scales[pid, h, i]
                            if slot > 0 and old >= new:
                                new = old
                            elif slot > 0:
                                held = e4m3_decode(self.pages[pid, h, :slot, i]) * (old / new)
                                self.pages[pid, h, :slot, i] = e4m3_encode(held)
                            self.scales[pid, h, i] = new
                            self.pages[pid, h, slot:slot + m, i] = e4m3_encode(rows[h, :, i] / new)
                t, at, n = t + m, at + m, n - m
        return np.stack([kr, v], 2)

    def values(self):
        if self.scales is None:
            return self.pages
        return e4m3_decode(self.pages) * self.scales[:, :, None, :, None]


def attend(q, values, cu, lens, table):
    """out; per element the weighted mean of |v| (what a relative error of the weights can move); and keys x
    largest weight x largest |v| (what an absolute one, of the largest weight, can)."""
    q = np.asarray(q, dtype=np.float64)
    out, reach, floor = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    Hk, page, d = values.shape[1], values.shape[2], values.shape[4]
    G = q.shape[1] // Hk
    for s in range(len(lens)):
        n, L = cu[s + 1] - cu[s], lens[s]
        if n == 0:
            continue
        ids = np.asarray(table[s][:(L + page - 1) // page])
        kv = values[ids].transpose(3, 1, 0, 2, 4).reshape(2, Hk, -1, d)[:, :, :L]
        for i in range(n):
            top = L - n + i + 1
            x = q[cu[s] + i].reshape(Hk, G, d)
            z = np.einsum("hgd,hjd->hgj", x, kv[0][:, :top]) / np.sqrt(d)
            w = np.exp(z - z.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            out[cu[s] + i] = np.einsum("hgj,hjd->hgd", w, kv[1][:, :top]).reshape(-1, d)
            most = top * w.max(-1) * np.abs(kv[1][:, :top]).max((1, 2))[:, None]
            floor[cu[s] + i] = np.broadcast_to(most.reshape(-1, 1), (Hk * G, d))
            reach[cu[s] + i] = np.einsum("hgj,hjd->hgd", w, np.abs(kv[1][:, :top])).reshape(-1, d)
    return out, reach, floor
