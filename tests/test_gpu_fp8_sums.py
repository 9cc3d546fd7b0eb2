"""What the block-scaled FP8 product keeps of a sum (needs an MI355X): for bf16
outputs the oracle's rule F5 (in each run of 8 features the products cut,
toward zero, to multiples of 2^(e - 13)), for fp32 outputs all 24 bits."""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import workloads as wl
from oracle import fp8 as o8
from oracle import svdquant as sq
from tests import gpu_harness as H
from tests.test_gpu_fp8 import _gpu, activations, run_linear, weight, y_of  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens and columns of each kernel of a bf16 product with one group of K: few tokens, tiles of 32 x 32, 64 x 32, 64 x
# 64, 64 x 128, 128 x 128 (three stages, two) and 256 x 256 (whole tiles, and with a divided last round)
SIZES = [(1, 8), (7, 520), (40, 64), (100, 2056), (400, 2056), (500, 2056), (900, 2056), (2100, 2056), (3000, 4104),
         (4200, 4104)]


def product(qx, qw, out):
    """Y [M, N] of codes with scales of 1."""
    t = H.torch()
    M, K = qx.shape
    N, G = qw.shape[0], o8.blocks(K)
    Y = t.empty((M, N), dtype=t.bfloat16 if out == "bf16" else t.float32, device="cuda")
    b.svdq_fp8_gemm(H.dev(qx), t.ones((G, M), device="cuda"), H.dev(qw), t.ones((o8.blocks(N), G), device="cuda"), None,
                    Y)
    return Y.double().cpu().numpy()


# {feature: (x, w)} of one token and column, and what comes out in bf16; in fp32 the sum itself does
TOP, BACK, SMALL = (256.0, 256.0), (256.0, -256.0), (2.5, 3.0)
SUMS = [
    ("2^16 + 2^3", {0: TOP, 1: (2.0, 4.0), 8: BACK}, 8.0),
    ("2^16 + 7.5", {0: TOP, 1: SMALL, 8: BACK}, 0.0),
    ("2^16 - 7.5", {0: TOP, 1: (2.5, -3.0), 8: BACK}, 0.0),
    ("2^16 - 15", {0: TOP, 1: (7.5, -2.0), 8: BACK}, -8.0),
    ("2^16 + 7 x 7.5", {0: TOP, **{k: SMALL for k in range(1, 8)}, 8: BACK}, 0.0),
    ("448^2 + 15: the exponents count", {0: (448.0, 448.0), 1: (7.5, 2.0), 8: (448.0, -448.0)}, 8.0),
    ("448^2 + 7 x 15 - 448^2 + 7 x 15", {0: (448.0, 448.0), **{k: (7.5, 2.0) for k in range(1, 8)},
                                         8: (448.0, -448.0), **{k: (7.5, 2.0) for k in range(9, 16)}}, 112.0),
    ("another run", {7: TOP, 8: SMALL, 16: BACK}, 7.5),
    ("the last of a run", {8: TOP, 15: SMALL, 16: BACK}, 0.0),
    ("another chunk", {15: TOP, 16: SMALL, 64: BACK}, 7.5),
    ("subnormals count as 2^-6", {0: (2.0 ** -9, 256.0), 1: (2.0 ** -9, 2.0 ** -3), 8: (-(2.0 ** -9), 256.0)}, 0.0),
    ("zeros do not count", {0: (0.0, 448.0), 1: (2.0 ** -9, 2.0 ** -9)}, 2.0 ** -18),
]


@pytest.mark.parametrize("M", [1, 40, 700])
@pytest.mark.parametrize("name,pairs,bf16", SUMS, ids=[s[0] for s in SUMS])
def test_single_sums(name, pairs, bf16, M):
    x, w = np.zeros((M, 128)), np.zeros((8, 128))
    for k, (a, c) in pairs.items():
        x[:, k], w[:, k] = a, c
    qx, qw = o8.e4m3_encode(x), o8.e4m3_encode(w)
    assert np.all(o8.cut_sums(qx[:1], qw)[0] == bf16)
    assert np.all(product(qx, qw, "bf16") == bf16)
    assert np.all(product(qx, qw, "f32") == sum(a * c for a, c in pairs.values()))


def cancelling_codes(M, N, seed):
    """Codes of M tokens and N columns, K = 128, whose products cancel: the second
    half holds the first one's pairs, negated and in other runs. The first
    pair of each run has exponents of 13 and more together and no code is below
    2^3, so that every cut and every sum is a whole number below 2^24: exact
    in fp32 in any order."""
    rng = np.random.default_rng(seed)
    def codes(rows, first):
        c = rng.integers(10 << 3, 127, (rows, 64))
        c[:, ::8] = rng.integers(first << 3, 127, (rows, 8))
        return c.astype(np.uint8) | (rng.integers(0, 2, (rows, 64)) << 7).astype(np.uint8)
    x, w = codes(M, 15), codes(N, 12)
    at = np.arange(64)
    at[::8] = rng.permutation(at[::8])
    rest = at % 8 != 0
    at[rest] = rng.permutation(at[rest])
    return np.concatenate([x, x[:, at]], 1), np.concatenate([w, w[:, at] ^ 0x80], 1)


@pytest.mark.parametrize("M,N", SIZES)
def test_sums_that_cancel_bit_for_bit(M, N):
    m, n = min(M, 37), min(N, 72)  # few rows and columns, repeated
    qx, qw = cancelling_codes(m, n, M + N)
    sums = o8.cut_sums(qx, qw)[0]
    assert np.max(np.abs(o8.e4m3_decode(qx)) @ np.abs(o8.e4m3_decode(qw)).T) < 2.0 ** 24
    assert np.array_equal(sums, np.rint(sums)) and np.abs(sums).max() > 0
    rows, cols = np.arange(M) % m, np.arange(N) % n
    want = sq.bf16_from_bits(wl.bf16_bits_from_f32(sums.astype(np.float32)))[rows][:, cols]
    assert np.array_equal(product(qx[rows], qw[cols], "bf16"), want)
    assert not product(qx[rows], qw[cols], "f32").any()


@pytest.mark.parametrize("M,K,N", [(5, 1040, 520), (40, 656, 264), (130, 1152, 136), (260, 528, 264)])
def test_random_sums_lose_no_more_than_the_rule(M, K, N):
    # Against the rule's own sums only fp32 additions differ. Each is off by at
    # most 2^-23 of a running sum of about y; blocks(K) + 32 of them (blocks, the
    # matrix core's runs, waves) by their root times that, twice it to be safe:
    # d. A shift by d turns a value over to its neighbour, a step of at most
    # 2^-7 y, with a probability of d over that step: sqrt(2^-7 y d) in the mean
    # square. One bit less in the cut would differ by about 3e-4.
    bits = activations(M, K, M)
    qw, sw = weight(K, N, N)
    y = y_of(run_linear(bits, qw, sw, None, "bf16"), M, "bf16")
    qx, sx = o8.quantize_activations(wl.f32_from_bf16_bits(bits))
    cut = o8.forward_cut(qx, sx, qw, sw)
    want = sq.bf16_from_bits(wl.bf16_bits_from_f32(cut.astype(np.float32)))
    d = 2 * 2.0 ** -23 * np.sqrt(o8.blocks(K) + 32)
    off = np.linalg.norm(y - want) / np.linalg.norm(cut)
    assert off <= np.sqrt(2.0 ** -7 * d), off
