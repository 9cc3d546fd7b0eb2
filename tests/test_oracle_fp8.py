"""Pins of the block-scaled FP8 oracle (oracle/fp8.py) and of the library's
host preparation against it."""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import workloads as wl
from oracle import fp8 as o8


def test_e4m3_list():
    v = o8.e4m3_decode(np.arange(256))
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7E] == 448.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and np.signbit(v[0x80])
    assert np.all(np.diff(v[:127]) > 0) and np.array_equal(v[128:255], -v[:127])


def test_e4m3_encode_is_nearest_even():
    v = o8.e4m3_decode(np.arange(127))
    assert np.array_equal(o8.e4m3_encode(v), np.arange(127))
    assert np.array_equal(o8.e4m3_encode(-v), np.arange(127) + 128)
    mid = (v[:-1] + v[1:]) / 2
    assert np.array_equal(o8.e4m3_encode(mid), np.arange(126) + (np.arange(126) % 2))  # the even neighbour
    assert np.array_equal(o8.e4m3_encode(np.nextafter(mid, 1e9)), np.arange(126) + 1)
    assert np.array_equal(o8.e4m3_encode(np.nextafter(mid, 0)), np.arange(126))
    assert o8.e4m3_encode(np.float64(463.0)) == 126


def test_blocks_by_hand():
    # a block whose largest is 448 has scale 1: codes are the values' own
    X = np.zeros((1, 144))
    X[0, :3] = [448.0, -1.0, 2.0 ** -9]
    X[0, 128] = -7.0  # the second block, 16 features: scale 7 / 448 = 2^-6
    q, s = o8.quantize_activations(X)
    assert s.shape == (2, 1) and s[0, 0] == 1.0 and s[1, 0] == 2.0 ** -6
    assert list(q[0, :4]) == [0x7E, 0xB8, 1, 0] and q[0, 128] == 0xFE
    # nothing but zeros: codes 0, the least scale
    q, s = o8.quantize_activations(np.zeros((2, 16)))
    assert not q.any() and np.all(s == np.float32(2.0 ** -100 / 448))


def test_forward_and_moe_by_loops():
    rng = np.random.default_rng(3)
    T, H, I, E, k = 5, 32, 16, 6, 2  # noqa: E741
    X, wr = rng.standard_normal((T, H)), rng.standard_normal((E, H))
    w13 = o8.e4m3_encode(rng.standard_normal((E, 2, I, H)))
    w2 = o8.e4m3_encode(rng.standard_normal((E, H, I)))
    s13 = rng.uniform(0.1, 1, (E, 2, 1, 1)).astype(np.float32)
    s2 = rng.uniform(0.1, 1, (E, 1, 1)).astype(np.float32)
    for renorm in (True, False):
        r = o8.moe(X, wr, w13, s13, w2, s2, k, renorm)
        for t in range(T):
            l = [sum(X[t, h] * wr[e, h] for h in range(H)) for e in range(E)]
            order = sorted(range(E), key=lambda e: (-l[e], e))[:k]
            assert list(r["idx"][t]) == order
            den = sum(np.exp(l[e]) for e in (order if renorm else range(E)))
            y = np.zeros(H)
            for e in order:
                g = X[t] @ (o8.e4m3_decode(w13[e, 0]) * s13[e, 0, 0, 0]).T
                u = X[t] @ (o8.e4m3_decode(w13[e, 1]) * s13[e, 1, 0, 0]).T
                y += np.exp(l[e]) / den * ((g / (1 + np.exp(-g)) * u) @ (o8.e4m3_decode(w2[e]) * s2[e, 0, 0]).T)
            assert np.allclose(r["y"][t], y, rtol=1e-12, atol=1e-12)
        assert np.all(r["bound"] > 0) and np.all(r["bound"] < 0.01 * np.abs(r["y"]).max())


def test_choose_ties_and_nan():
    l = np.array([[1.0, 3.0, 3.0, 2.0], [np.nan, -np.inf, 0.0, np.nan], [np.inf, 5.0, np.inf, 1.0]])
    assert o8.choose(l, 3).tolist() == [[1, 2, 3], [2, 0, 1], [0, 2, 1]]


@pytest.mark.parametrize("K,N", [(16, 8), (128, 128), (144, 136), (400, 264)])
def test_prepare_weights_matches_the_oracle(K, N):
    W = wl.random_bf16(K + N, (K, N), 0.02)
    bits = W["bits"].copy()
    bits[0, :] = 0
    bits[1, 0], bits[2, 0] = 0x0001, 0x8000  # the least subnormal, -0
    if K >= 144:
        bits[128:144, :] = 0  # a block row's tail of zeros
    v = wl.f32_from_bf16_bits(bits)
    q, s = b.svdq_fp8_prepare_weights(bits)
    oq, os_ = o8.prepare_weights(v)
    assert np.array_equal(s, os_) and np.array_equal(q, oq)


def test_prepare_weights_zero_and_refusals():
    q, s = b.svdq_fp8_prepare_weights(np.zeros((32, 16), np.uint16))
    assert not q.any() and np.all(s > 0)
    for shape, status in (((24, 16), b.SVDQ_ERR_UNSUPPORTED_SHAPE), ((32, 12), b.SVDQ_ERR_UNSUPPORTED_SHAPE)):
        with pytest.raises(b.SvdqError) as e:
            b.svdq_fp8_prepare_weights(np.zeros(shape, np.uint16))
        assert e.value.status == status
    bad = np.zeros((32, 16), np.uint16)
    bad[3, 3] = 0x7F80  # infinity
    with pytest.raises(b.SvdqError) as e:
        b.svdq_fp8_prepare_weights(bad)
    assert e.value.status == b.SVDQ_ERR_NUMERICAL


def test_cut_sums_by_hand_and_by_loops():
    x, w = np.zeros((1, 144)), np.zeros((2, 144))
    x[0, :3], w[0, :3] = [256.0, 2.0, 2.5], [256.0, 4.0, 3.0]  # 2^16, 8 and 7.5 in one run: 7.5 goes
    x[0, 130:132], w[1, 130:132] = [2.0 ** -9, 2.0 ** -9], [256.0, 2.0 ** -3]  # a subnormal counts as 2^-6
    s = o8.cut_sums(o8.e4m3_encode(x), o8.e4m3_encode(w))
    assert s.shape == (2, 1, 2) and s[0, 0, 0] == 2.0 ** 16 + 8 and s[0, 0, 1] == 0
    assert s[1, 0, 1] == 0.5 and s[1, 0, 0] == 0
    rng = np.random.default_rng(5)
    qx, qw = (rng.integers(0, 127, (n, 32)).astype(np.uint8) | (rng.integers(0, 2, (n, 32)) << 7).astype(np.uint8)
              for n in (3, 4))
    s, vx, vw = o8.cut_sums(qx, qw), o8.e4m3_decode(qx), o8.e4m3_decode(qw)
    expo = lambda v: max(int(np.floor(np.log2(abs(v)))), -6)  # noqa: E731
    for m in range(3):
        for n in range(4):
            total = 0.0
            for k in range(0, 32, 8):
                pairs = [(a, c) for a, c in zip(vx[m, k: k + 8], vw[n, k: k + 8]) if a * c]
                unit = 2.0 ** (max(expo(a) + expo(c) for a, c in pairs) - 13)
                total += sum(np.sign(a * c) * np.floor(abs(a * c) / unit) * unit for a, c in pairs)
            assert s[0, m, n] == total
    sx, sw = np.full((1, 3), 2.0, np.float32), np.full((1, 1), 0.5, np.float32)
    assert np.array_equal(o8.forward_cut(qx, sx, qw, sw, [1.0, 2.0, 3.0, 4.0]), s[0] + [[1.0, 2.0, 3.0, 4.0]])
