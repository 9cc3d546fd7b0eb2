"""Oracle for the block-scaled FP8 linear and the mixture-of-experts layer on
block-scaled FP8 weights.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``).

  F1  a block (128 x 128 of a weight, one token's 128 features of X; the last
      block of a row or column holds what is left) has A = max(max |v|,
      2^-100), scale RN32(A / 448) and codes E4M3(RN32(v RN32(448 / A)));
  F2  E4M3 (OCP, no infinities): 1 sign, 4 exponent (bias 7), 3 mantissa bits,
      steps of 2^-9 below 2^-6, largest 448; nearest, ties to even;
  F3  linear: y = sum_g sx[g, m] sw[n / 128, g] sum_{k in g} qx qw + bias,
      evaluated in float64 and rounded once;
  F4  experts: logits X Wr^T, the top_k largest with ties to the lowest
      expert, softmax over all or over the chosen ones, silu(X Wg) (X Wu) Wd
      of each choice on the dequantized weights, weighted sum, float64;
  F5  what the FP8 matrix core keeps of F3's products, for bf16 outputs: in each
      run of 8 features every product is cut, toward zero, to a multiple of
      2^(e - 13), e the largest sum of the two codes' exponents among the
      products that are not 0 (codes below 2^-6 have the exponent -6).

Parity status: pinned by tests/test_oracle_fp8.py (the list of all E4M3
values, hand-computed blocks, brute-force loops).
"""

from __future__ import annotations

import numpy as np

from .svdquant import rn32

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100
F64 = np.float64


def _value(b):
    ex, man = (b >> 3) & 15, b & 7
    if ex == 15 and man == 7:
        return np.nan
    mag = man * 2.0 ** -9 if ex == 0 else (1 + man / 8.0) * 2.0 ** (ex - 7)
    return -mag if b & 0x80 else mag


_BYTES = np.array([_value(b) for b in range(256)])


def e4m3_decode(b):
    """Values of E4M3 bytes (NaN for 0x7F and 0xFF)."""
    return _BYTES[np.asarray(b, dtype=np.uint8)]


_VALUES = e4m3_decode(np.arange(127))  # ascending magnitudes of codes 0 .. 126


def e4m3_encode(v):
    """E4M3 bytes nearest to v (|v| < 464), ties to the even code."""
    v = np.asarray(v, dtype=F64)
    m = np.abs(v)
    hi = np.clip(np.searchsorted(_VALUES, m), 1, 126)
    lo = hi - 1
    down, up = m - _VALUES[lo], _VALUES[hi] - m
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return (np.where(take_hi, hi, lo) | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def _scale(amax):
    a = np.maximum(amax, TINY)
    return rn32(a / E4M3_MAX).astype(np.float32), rn32(E4M3_MAX / a).astype(F64)


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def prepare_weights(W):
    """W [K, N] -> codes [N, K] (bytes) and scales [blocks(N), blocks(K)] fp32."""
    W = np.asarray(W, dtype=F64)
    K, N = W.shape
    q = np.zeros((N, K), np.uint8)
    s = np.zeros((blocks(N), blocks(K)), np.float32)
    for b in range(blocks(N)):
        for g in range(blocks(K)):
            n, k = slice(b * BLOCK, (b + 1) * BLOCK), slice(g * BLOCK, (g + 1) * BLOCK)
            s[b, g], r = _scale(np.max(np.abs(W[k, n])))
            q[n, k] = e4m3_encode(rn32(W[k, n].T * r))
    return q, s


def dequantize(q, s):
    """float64 weight [N, K] of codes and block scales."""
    N, K = q.shape
    return e4m3_decode(q) * s.astype(F64)[np.arange(N) // BLOCK][:, np.arange(K) // BLOCK]


def quantize_activations(X):
    """X [M, K] -> codes [M, K] (bytes) and scales [blocks(K), M] fp32."""
    X = np.asarray(X, dtype=F64)
    M, K = X.shape
    q = np.zeros((M, K), np.uint8)
    s = np.zeros((blocks(K), M), np.float32)
    for g in range(blocks(K)):
        k = slice(g * BLOCK, (g + 1) * BLOCK)
        s[g], r = _scale(np.max(np.abs(X[:, k]), axis=1))
        q[:, k] = e4m3_encode(rn32(X[:, k] * r[:, None]))
    return q, s


def dequantize_activations(q, s):
    return e4m3_decode(q) * s.astype(F64).T[:, np.arange(q.shape[1]) // BLOCK]


def forward(X, qw, sw, bias=None):
    """The linear: dict with qx, sx, y (float64), mag = sum |terms| and peaks =
    the sum over runs of 8 features of the largest |x| times the largest |w|."""
    qx, sx = quantize_activations(X)
    x, w = dequantize_activations(qx, sx), dequantize(qw, sw)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        b = np.asarray(bias, dtype=F64)[None, :]
        y, mag = y + b, mag + np.abs(b)
    top = lambda v: np.abs(v).reshape(v.shape[0], -1, 8).max(2)  # noqa: E731
    return {"qx": qx, "sx": sx, "y": y, "mag": mag, "peaks": top(x) @ top(w).T}


def cut_sums(qx, qw):
    """Sums of F5's products in each block of features, [blocks(K), M, N] float64 of codes [M, K] and [N, K]."""
    M, K = qx.shape
    N = qw.shape[0]
    x, w = e4m3_decode(qx), e4m3_decode(qw)
    ex, ew = (np.maximum(q >> 3 & 15, 1).astype(np.int64) - 7 for q in (qx, qw))
    out = np.zeros((blocks(K), M, N))
    for k in range(0, K, 8):
        p = x[:, None, k: k + 8] * w[None, :, k: k + 8]
        e = np.where(p == 0, -40, ex[:, None, k: k + 8] + ew[None, :, k: k + 8]).max(2, keepdims=True)
        unit = np.exp2((e - 13).astype(F64))
        out[k // BLOCK] += (np.trunc(p / unit) * unit).sum(2)
    return out


def forward_cut(qx, sx, qw, sw, bias=None):
    """y (float64) of the linear with F5's sums."""
    y = np.zeros((qx.shape[0], qw.shape[0]))
    for g, s in enumerate(cut_sums(qx, qw)):
        y += s * sx[g].astype(F64)[:, None] * sw[np.arange(qw.shape[0]) // BLOCK, g].astype(F64)[None, :]
    return y if bias is None else y + np.asarray(bias, dtype=F64)[None, :]


def choose(logits, top_k):
    """[T, top_k] experts: largest first, ties to the lowest, NaN and -inf last."""
    key = np.where(logits > -np.inf, logits, -np.inf)
    key = np.where(np.isnan(logits), -np.inf, key)
    return np.argsort(-key, axis=1, kind="stable")[:, :top_k]


def moe(X, wr, w13, s13, w2, s2, top_k, renormalize):
    """The layer on codes w13 [E, 2, I, H], w2 [E, H, I]: dict with idx, gate,
    y (float64) and bound, the rounding error that fp32 sums of the layer's
    products, the 16-bit h and fp32 gates may make before the last rounding."""
    X = np.asarray(X, dtype=F64)
    T, H = X.shape
    E, _, I, _ = w13.shape  # noqa: E741
    logits = X @ np.asarray(wr, dtype=F64).T
    idx = choose(logits, top_k)
    top = np.take_along_axis(logits, idx[:, :1], 1)
    e = np.exp(logits - top)
    chosen = np.take_along_axis(e, idx, 1)
    gate = chosen / (chosen if renormalize else e).sum(1, keepdims=True)
    u32 = 2.0 ** -24
    # gates: the exponent's argument and exp to fp32, a sum of up to E terms, a division
    far = np.max(np.where(np.isfinite(logits - top), np.abs(logits - top), 0.0), axis=1)
    dgate = gate * ((E + 2 * far + 8) * u32)[:, None]
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    n_up, n_down = BLOCK + blocks(H) + 16, BLOCK + blocks(I) + 16  # additions on a term's way
    for x in np.unique(idx):
        t, j = np.nonzero(idx == x)
        wg, wu = dequantize(w13[x, 0], s13[x, 0]), dequantize(w13[x, 1], s13[x, 1])
        wd = dequantize(w2[x], s2[x])
        g, u = X[t] @ wg.T, X[t] @ wu.T
        dg = 2 * n_up * u32 * (np.abs(X[t]) @ np.abs(wg).T)
        du = 2 * n_up * u32 * (np.abs(X[t]) @ np.abs(wu).T)
        silu = g / (1 + np.exp(-g))
        h = silu * u
        # |silu'| <= 1.1; exp, division and product to a few fp32 roundings;
        # h = hi + lo, each of 8 bits: 2^-8 2^-8 of h
        dh = 1.1 * dg * np.abs(u) + (np.abs(silu) + 1.1 * dg) * du + np.abs(h) * (2.0 ** -16 + 8 * u32)
        o, mag = h @ wd.T, np.abs(h) @ np.abs(wd).T
        do = dh @ np.abs(wd).T + 2 * n_down * u32 * mag
        y[t] += gate[t, j][:, None] * o
        bound[t] += gate[t, j][:, None] * (do + (top_k + 2) * u32 * np.abs(o)) + dgate[t, j][:, None] * np.abs(o)
    return {"idx": idx, "gate": gate, "dgate": dgate, "y": y, "bound": bound}
