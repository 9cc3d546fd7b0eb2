"""Oracle for the norm before the block-scaled FP8 linears, rotary positions, and
the 8-bit key and value cache with its attention.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``).

  D1  norm: h = X + residual, y = h / sqrt(mean h^2 + eps) * w, float64 throughout;
      the sum is also given as fp32 rounded once more to bf16;
  D2  rotary positions: the angle of pair j is positions[axis of j] * freqs[j];
      (a, b) -> (a cos - b sin, a sin + b cos), float64;
  D3  append: per page of 64 tokens and head, keys and values apart, the least
      power of two s with max |x| <= 448 s over the new tokens (2^-100 at the
      least; not over values that are not finite), at least the page's scale where
      earlier tokens are kept; codes E4M3(x / s); earlier codes become
      E4M3(code * old / s); NaN and infinities become NaN;
  D4  attention: softmax(scale q k^T) v over what a query sees, float64, 0 and
      -infinity where it sees nothing. `mag` is sum p |v|, `square` sum p^2 v^2 and
      `score` the largest sum of scale |q| |k|: what rounded sums may be off by.

Parity status: pinned by tests/test_oracle_decoder.py.
"""

from __future__ import annotations

import numpy as np

from .fp8 import BLOCK, E4M3_MAX, TINY, blocks, e4m3_decode, e4m3_encode
from .svdquant import bf16_round, rn32

F64 = np.float64
PAGE = 64
NAN_CODE = 0x7F


def norm(X, residual, w, eps):
    """D1: {"h", "sum" (bf16 values), "y"}, float64."""
    h = np.asarray(X, F64) + (0.0 if residual is None else np.asarray(residual, F64))
    with np.errstate(invalid="ignore", over="ignore"):
        y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(w, F64)
    return {"h": h, "sum": bf16_round(rn32(h)), "y": y}


def block_tops(y):
    """max(max |y|, 2^-100) of each token's blocks of 128 features, [blocks, M]."""
    return np.stack([np.maximum(np.max(np.abs(y[:, g * BLOCK: (g + 1) * BLOCK]), axis=1), TINY)
                     for g in range(blocks(y.shape[1]))])


def rope(X, positions, freqs, sections, interleaved):
    """D2: X [T, H, D] turned, float64."""
    X = np.asarray(X, F64)
    out = X.copy()
    pairs, j = int(sum(sections)), 0
    for axis, n in enumerate(sections):
        for _ in range(n):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
            angle = positions[:, axis].astype(F64) * freqs[j]
            c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
            out[:, :, a] = X[:, :, a] * c - X[:, :, b] * s
            out[:, :, b] = X[:, :, a] * s + X[:, :, b] * c
            j += 1
    return out


def page_scale(top):
    """The least power of two s with top <= 448 s."""
    s = 2.0 ** np.floor(np.log2(top / E4M3_MAX))
    while s * E4M3_MAX < top:
        s *= 2.0
    while s * E4M3_MAX / 2 >= top:
        s /= 2.0
    return s


def encode(v):
    """E4M3 bytes; NaN where v is not finite."""
    v = np.asarray(v, F64)
    ok = np.isfinite(v)
    return np.where(ok, e4m3_encode(np.where(ok, v, 0.0)), NAN_CODE).astype(np.uint8)


class Cache:
    """Pages as the library lays them out: kc [P, Hk, 64, D], vc [P, Hk, D, 64]
    (bytes), ks, vs [P, Hk] fp32."""

    def __init__(self, kc, ks, vc, vs):
        self.kc, self.ks, self.vc, self.vs = kc.copy(), ks.copy(), vc.copy(), vs.copy()

    def append(self, K, V, starts, lengths, table):
        """D3, in place; K, V [T, Hk, D] float64 values of bf16 numbers."""
        P = self.kc.shape[0]
        for b, length in enumerate(lengths):
            n = starts[b + 1] - starts[b]
            for pos in sorted({max(0, length - n + i) // PAGE for i in range(n) if length - n + i >= 0}):
                page = table[b][pos]
                if not 0 <= page < P:
                    continue
                low, high = max(length - n - pos * PAGE, 0), min(length - pos * PAGE, PAGE)
                row = starts[b] + n - length + pos * PAGE
                for x, codes, scales, across in ((K, self.kc, self.ks, False), (V, self.vc, self.vs, True)):
                    for h in range(codes.shape[1]):
                        self._page(x[row + low: row + high, h], codes[page, h].T if across else codes[page, h],
                                   scales[page], h, low, high)

    @staticmethod
    def _page(x, codes, scales, h, low, high):
        finite = np.abs(x[np.isfinite(x)])
        s = page_scale(max(finite.max() if finite.size else 0.0, TINY))
        if low > 0:
            old = F64(scales[h])
            s = max(s, old)
            if s != old:
                codes[:low] = encode(rn32(e4m3_decode(codes[:low]) * (old / s)))
        with np.errstate(invalid="ignore"):
            codes[low:high] = encode(rn32(x / s))
        scales[h] = s

    def sequence(self, pages, length):
        """Keys and values [length, Hk, D] float64, and which tokens have a page."""
        P, Hk, _, D = self.kc.shape
        k, v, there = np.zeros((length, Hk, D)), np.zeros((length, Hk, D)), np.zeros(length, bool)
        for t in range(0, length, PAGE):
            page, n = pages[t // PAGE], min(PAGE, length - t)
            if 0 <= page < P:
                k[t: t + n] = (e4m3_decode(self.kc[page, :, :n]) * self.ks[page].astype(F64)[:, None, None]).transpose(1, 0, 2)
                v[t: t + n] = (e4m3_decode(self.vc[page, :, :, :n]) * self.vs[page].astype(F64)[:, None, None]).transpose(2, 0, 1)
                there[t: t + n] = True
        return k, v, there


def attention(Q, cache, starts, lengths, table, scale, causal=True, window=0):
    """D4 for the rows starts[0] .. starts[B] - 1 of Q [T, Hq, D]; the others are NaN."""
    Q = np.asarray(Q, F64)
    T, Hq, D = Q.shape
    Hk = cache.kc.shape[1]
    out = {n: np.full((T, Hq, D), np.nan) for n in ("o", "mag", "square")}
    out["lse"], out["score"] = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for b, length in enumerate(lengths):
        k, v, there = cache.sequence(table[b], length)
        n = starts[b + 1] - starts[b]
        for i in range(n):
            pos = length - n + i
            t = np.arange(length)
            see = there & ((t <= pos) if causal else True)
            if window:
                see = see & (t > pos - window)
            for h in range(Hq):
                r, g = starts[b] + i, h // (Hq // Hk)
                q, ks, vs = Q[r, h], k[see, g], v[see, g]
                if not see.any():
                    out["o"][r, h] = out["mag"][r, h] = out["square"][r, h] = 0.0
                    out["lse"][r, h] = -np.inf
                    continue
                with np.errstate(invalid="ignore"):
                    s = scale * (ks @ q)
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    out["o"][r, h], out["mag"][r, h] = p @ vs, p @ np.abs(vs)
                    out["square"][r, h] = (p * p) @ (vs * vs)
                    out["lse"][r, h] = s.max() + np.log(e.sum())
                    out["score"][r, h] = scale * np.max(np.abs(ks) @ np.abs(q))
    return out
