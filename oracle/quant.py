"""The 8-bit cache and the sampled acceptance in float64. TEST INFRASTRUCTURE.

e4m3 (the OCP 8-bit floating point format, "FN" variant): 1 sign, 4 exponent and 3 mantissa bits,
bias 7, no infinities; the largest value is 448, the smallest normal 2^-6, the subnormal step 2^-9.
A block of consecutive slots of a page shares a power-of-two scale s for K and V and each head, the
smallest with amax <= 448 s.
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126


def e4m3(x):
    """The nearest e4m3 value, ties to even; beyond +-448 clamped; NaN -> 0 (what a cache write stores)."""
    x = np.clip(np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=E4M3_MAX, neginf=-E4M3_MAX),
                -E4M3_MAX, E4M3_MAX)
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e, -5).astype(np.float64) - 4)
    return np.rint(x / step) * step


def needed_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = MIN_SCALE
    if amax > E4M3_MAX * s:
        s = max(s, 2.0 ** (math.frexp(amax / E4M3_MAX)[1] - 1))
        while amax > E4M3_MAX * s:
            s *= 2
    return s


def code_values(codes):
    """Values of e4m3 code bytes (uint8)."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * np.exp2(e - 10.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


class QuantPool:
    """One layer: values [page][K|V][head][slot][D] (already e4m3) and scales [page][K|V][head][block]."""

    def __init__(self, n_pages, n_kv_heads, page_size, head_dim, scale_block):
        self.ps, self.sb = page_size, scale_block
        self.val = np.zeros((n_pages, 2, n_kv_heads, page_size, head_dim))
        self.scale = np.zeros((n_pages, 2, n_kv_heads, page_size // scale_block))

    def write(self, pages, base, k, v):
        """Rows k, v [S][heads][D] at positions base.. of the sequence whose page table is `pages`."""
        rows = np.stack([k, v], 1).astype(np.float64)              # [S][2][heads][D]
        S, p = len(rows), base
        while p < base + S:
            stop = min(base + S, (p // self.sb + 1) * self.sb)
            page, a, blk = pages[p // self.ps], p % self.ps, p % self.ps // self.sb
            for kv in range(2):
                for h in range(rows.shape[2]):
                    x = rows[p - base:stop - base, kv, h]
                    fin = np.abs(x[np.isfinite(x)])
                    s = needed_scale(float(fin.max()) if fin.size else 0.0)
                    if p % self.sb:
                        old = self.scale[page, kv, h, blk]
                        s = max(s, old)
                        low = self.val[page, kv, h, blk * self.sb:a]
                        self.val[page, kv, h, blk * self.sb:a] = e4m3(low * (old / s))
                    self.scale[page, kv, h, blk] = s
                    self.val[page, kv, h, a:a + stop - p] = e4m3(x / s)
            p = stop

    def rows(self, pages, lo, hi):
        """(K, V) of positions lo..hi-1, [n][heads][D] each."""
        out = []
        for p in range(lo, hi):
            page, slot = pages[p // self.ps], p % self.ps
            out.append(self.val[page, :, :, slot] * self.scale[page, :, :, slot // self.sb][..., None])
        x = np.array(out)
        return x[:, 0], x[:, 1]

    def attention(self, pages, base, q, window=0):
        """(o, sum_t p_t |v_t|, max_t sum_d |q_d k_td| / sqrt(D)) of rows q [S][nq][D] at positions base..:
        the result, and the magnitudes that rounding errors scale with."""
        S, nq, D = q.shape
        k, v = self.rows(pages, 0, base + S)
        grp = nq // k.shape[1]
        o, mag, top = (np.zeros((S, nq, D)) for _ in range(3))
        for i in range(S):
            lo = max(0, base + i - window + 1) if window else 0
            for h in range(nq):
                kk, vv = k[lo:base + i + 1, h // grp], v[lo:base + i + 1, h // grp]
                z = kk @ q[i, h].astype(np.float64) / math.sqrt(D)
                p = np.exp(z - z.max())
                p /= p.sum()
                o[i, h], mag[i, h] = p @ vv, p @ np.abs(vv)
                top[i, h] = (np.abs(kk) @ np.abs(q[i, h].astype(np.float64))).max() / math.sqrt(D)
        return o, mag, top


def accept_sampled(span, logits, temperature, uniform, noise, probs=None):
    """(m, committed tokens) of one sequence: span = [current, d_1..d_k], logits [S][V], uniform [S],
    noise [V], probs [S][V] or None (every draft certain)."""
    S, V = logits.shape
    for i in range(S):
        x = np.where(np.isnan(logits[i]), -np.inf, logits[i].astype(np.float64))
        if not (x > -np.inf).any():
            return i, list(span[1:1 + i]) + [0]
        top = x.max()
        if temperature > 0:
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.where(x == top, 1.0, np.exp((x - top) / float(temperature)))
            p[np.isneginf(x)] = 0.0
            p /= p.sum()
        else:
            p = np.zeros(V)
            p[int(np.argmax(x))] = 1.0
        if i < S - 1:
            d = int(span[1 + i])
            usable = 0 <= d < V
            if probs is not None:
                q = probs[i].astype(np.float64)
            else:
                q = np.zeros(V)
                if usable:
                    q[d] = 1.0
            if usable and float(uniform[i]) * q[d] < p[d]:
                continue
            left = np.maximum(p - q, 0)
            w = left if left.sum() > 0 else p
        else:
            w = p
        with np.errstate(divide="ignore"):
            race = np.where(w > 0, w / noise.astype(np.float64), -1.0)
        return i, list(span[1:1 + i]) + [int(np.argmax(race))]
    raise AssertionError("an empty span commits nothing")
