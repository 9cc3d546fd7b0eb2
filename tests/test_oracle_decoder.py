"""Pins of oracle/decoder.py: hand-computed values and plain loops. No GPU."""

import math

import numpy as np
import pytest

from oracle import decoder as od
from oracle.fp8 import e4m3_decode


def test_norm_by_hand():
    out = od.norm([[3.0, -4.0]], [[0.0, 0.0]], [1.0, 2.0], 0.0)
    r = math.sqrt(12.5)
    assert np.allclose(out["y"], [[3 / r, -8 / r]], rtol=1e-15) and np.array_equal(out["sum"], [[3.0, -4.0]])
    assert np.array_equal(od.norm([[1.0, 2.0]], [[2.0, 2.0]], [1.0, 1.0], 3.5)["h"], [[3.0, 4.0]])
    assert np.allclose(od.norm([[3.0, 4.0]], None, [1.0, 1.0], 3.5)["y"], [[0.75, 1.0]], rtol=1e-15)


def test_block_tops_of_a_short_last_block():
    y = np.zeros((2, 144))
    y[0, 5], y[1, 140] = -3.0, 7.0
    assert np.array_equal(od.block_tops(y), [[3.0, 2.0 ** -100], [2.0 ** -100, 7.0]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_in_the_pair_plane(interleaved):
    rng = np.random.default_rng(1)
    X = rng.standard_normal((3, 2, 40))
    pos = np.array([[0, 5], [7, 1], [1000, 31]])
    freqs = np.concatenate([10000.0 ** (-np.arange(10) / 10), 100.0 ** (-np.arange(6) / 6)])
    Y = od.rope(X, pos, freqs, [10, 6], interleaved)
    assert np.array_equal(Y[:, :, 32:], X[:, :, 32:])
    for j in range(16):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + 16)
        turn = np.exp(1j * pos[:, 0 if j < 10 else 1] * freqs[j])[:, None]
        assert np.allclose(Y[:, :, a] + 1j * Y[:, :, b], (X[:, :, a] + 1j * X[:, :, b]) * turn, atol=1e-12)
    back = od.rope(Y, pos, -freqs, [10, 6], interleaved)
    assert np.allclose(back, X, atol=1e-12)


@pytest.mark.parametrize("top,scale", [(448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (225.0, 1.0), (1.75, 2.0 ** -8),
                                       (1.0, 2.0 ** -8), (2.0 ** -100, 2.0 ** -108), (3.3e38, 2.0 ** 120)])
def test_page_scale(top, scale):
    assert od.page_scale(top) == scale


def _cache(P=3, Hk=2, D=4, fill=0x38):
    return od.Cache(np.full((P, Hk, 64, D), fill, np.uint8), np.ones((P, Hk), np.float32),
                    np.full((P, Hk, D, 64), fill, np.uint8), np.ones((P, Hk), np.float32))


def test_append_places_tokens_and_rescales_the_page():
    c = _cache()
    K = np.zeros((3, 2, 4))
    K[0], K[1], K[2] = 0.5, 2.0, 1000.0
    c.append(K, -K, [0, 3], [66], [[2, 0]])  # tokens 63, 64, 65
    # token 63 joins page 2 (scale 1 is enough), 64 and 65 begin page 0 (scale 4 for 1000)
    assert np.all(c.ks[2] == 1) and np.all(c.ks[0] == 4) and np.all(c.ks[1] == 1)
    assert np.all(e4m3_decode(c.kc[2, :, 63]) == 0.5) and np.all(c.kc[2, :, :63] == 0x38)
    assert np.all(e4m3_decode(c.kc[0, :, 0]) == 0.5) and np.all(e4m3_decode(c.kc[0, :, 1]) == 256.0)
    assert np.all(e4m3_decode(c.vc[0, :, :, 1]) == -256.0) and np.all(c.vc[0, :, :, 2:] == 0x38)
    assert np.all(c.kc[1] == 0x38)
    more = np.full((1, 2, 4), 896.0)
    c.append(more, more, [0, 1], [65], [[1, 2]])  # token 64 again, now in page 2: its first
    assert np.all(c.ks[2] == 2) and np.all(e4m3_decode(c.kc[2, :, 0]) == 448)
    c.append(more * 4, more, [0, 1], [66], [[1, 2]])  # the next: codes of scale 2 become codes of scale 8
    assert np.all(c.ks[2] == 8) and np.all(e4m3_decode(c.kc[2, :, 0]) == 112) and np.all(c.vs[2] == 2)


def test_append_not_finite_and_outside():
    c = _cache()
    x = np.ones((2, 2, 4))
    x[0, 0, 1], x[1, 1, 2] = np.nan, -np.inf
    c.append(x, x, [0, 2], [2], [[1]])
    assert c.kc[1, 0, 0, 1] == 0x7F and c.kc[1, 1, 1, 2] == 0x7F and c.vc[1, 0, 1, 0] == 0x7F
    assert np.all(c.ks[1] == 2.0 ** -8)
    before = c.kc.copy()
    c.append(x, x, [0, 2], [1], [[7]])  # no such page
    assert np.array_equal(c.kc, before)
    c.append(x * 2, x * 2, [0, 2], [1], [[0]])  # one token more than the sequence has: the first is left out
    assert np.all(e4m3_decode(c.kc[0, 0, 0]) * c.ks[0, 0] == 2.0)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 3)])
def test_attention_by_loops(causal, window):
    rng = np.random.default_rng(5)
    Hq, Hk, D = 4, 2, 8
    codes = rng.integers(0, 0x78, (4, Hk, 64, D)).astype(np.uint8)
    c = od.Cache(codes, np.full((4, Hk), 2.0 ** -6, np.float32), codes.transpose(0, 1, 3, 2).copy(),
                 np.full((4, Hk), 2.0 ** -5, np.float32))
    Q = rng.standard_normal((5, Hq, D)) * 0.1
    out = od.attention(Q, c, [0, 2, 5], [70, 3], [[3, 1], [0, -1]], 0.5, causal, window)
    pages = [[3, 1], [0]]
    for r, (b, pos) in enumerate([(0, 68), (0, 69), (1, 0), (1, 1), (1, 2)]):
        for h in range(Hq):
            num, den, total = np.zeros(D), 0.0, [70, 3][b]
            for t in range(total):
                if causal and t > pos or window and t <= pos - window:
                    continue
                page, g = pages[b][t // 64], h // 2
                k = e4m3_decode(c.kc[page, g, t % 64]) * 2.0 ** -6
                v = e4m3_decode(c.vc[page, g, :, t % 64]) * 2.0 ** -5
                w = math.exp(0.5 * float(k @ Q[r, h]))
                num, den = num + w * v, den + w
            assert np.allclose(out["o"][r, h], num / den, rtol=1e-10)
            assert math.isclose(out["lse"][r, h], math.log(den), rel_tol=1e-10, abs_tol=1e-10)


def test_attention_of_nothing():
    c = _cache(D=8)
    out = od.attention(np.ones((3, 2, 8)), c, [0, 2, 3], [1, 0], [[0], [0]], 1.0)
    assert np.all(out["o"][0] == 0) and np.all(np.isneginf(out["lse"][[0, 2]])) and np.all(out["o"][1] == 1.0)
