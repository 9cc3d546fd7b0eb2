"""The block-scaled FP8 kernels at the shapes of theirs that test_gpu_fp8.py does
not reach (needs an MI355X): divided tiles and further rounds of the 256-wide
kernel, the turned start of each kernel for few tokens, every variant of the
expert layer's two big kernels. test_fp8_dispatch.py holds the two lists
against the library's rules."""

import numpy as np
import pytest

from bit_quantized_linear_amd import workloads as wl
from oracle import fp8 as o8
from tests import gpu_harness as H
from tests import test_gpu_fp8 as g
from tests.test_gpu_fp8 import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# few tokens, K in rows 4 KB apart: 16 and 32 columns per block, one launch and two
TURNED = [(2, 4096, 264), (1, 8192, 1032), (16, 4096, 520), (5, 8192, 264), (1, 4096, 5128), (8, 4096, 5128),
          (4, 8192, 5128)]
# the 256-wide kernel, bf16: 8 x 16 tiles, all of them divided (without and with halves past M), a second round with
# divided tiles (17 x 17, a half past M; 24 x 13) and one without (24 x 17)
LARGE = [(2040, 144, 4096), (1900, 144, 4096), (4200, 144, 4104), (6140, 272, 3080), (6100, 144, 4104)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", TURNED)
def test_linear_of_few_tokens_with_a_turned_start(M, K, N, out):
    g.test_linear(M, K, N, out)


@pytest.mark.parametrize("M,K,N", LARGE)
def test_linear_of_divided_tiles(M, K, N):
    g.test_linear(M, K, N, "bf16")


# tokens, H, I, experts, choices; behind them what of the library's rules each is for
EXPERTS = [
    (3, 272, 48, 100, 2),       # 4 tokens in one slot, the choice by itself
    (3, 4096, 48, 100, 2),      # and a turned start
    (5, 4096, 48, 20, 2),       # straight loads, the choice in the up kernel, turned
    (9, 4096, 48, 29, 4),       # 8 tokens in two slots, turned
    (2, 8192, 32, 6, 2),        # two turns of the groups
    (64, 144, 656, 16, 3),      # 16 columns, 4 slots, batches (4 and 2 groups); an expert's tokens in parts
    (64, 144, 656, 20, 8),      # 16 columns, 2 slots, batches
    (64, 2064, 656, 60, 7),     # the same with few tokens per expert
    (8, 2064, 1424, 17, 2),     # 16 columns, 4 slots, batches of 4, 4 and 4 groups
    (64, 144, 1168, 104, 13),   # 8 columns, 2 slots, batches
    (64, 272, 1424, 64, 2),     # 8 columns, 4 slots, batches, an even and an odd number of groups
    (64, 272, 1168, 64, 6),
    (1, 144, 16400, 2, 1),      # 16 shares of I, batches in each
    (1, 144, 16400, 1, 1),
]


def experts(E, H_, I, seed):  # noqa: E741
    """As g.experts, from random bytes: codes of all magnitudes, none a NaN."""
    rng = np.random.default_rng(seed)
    def codes(*shape):
        c = rng.integers(0, 256, shape, np.uint8)
        return np.where(c & 0x7F == 0x7F, np.uint8(0x38), c)
    w13, w2 = codes(E, 2, I, H_), codes(E, H_, I)
    s13 = (rng.uniform(0.5, 1.5, (E, 2, o8.blocks(I), o8.blocks(H_))) * 0.01 / np.sqrt(H_)).astype(np.float32)
    s2 = (rng.uniform(0.5, 1.5, (E, o8.blocks(H_), o8.blocks(I))) * 0.01 / np.sqrt(I)).astype(np.float32)
    return wl.random_bf16(seed, (E, H_), 2.0 / np.sqrt(H_)), w13, s13, w2, s2


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,H_,I,E,k", EXPERTS)
def test_experts(T, H_, I, E, k, renorm):  # noqa: E741
    bits = wl.random_bf16(T + H_ + I, (T, H_))["bits"]
    wr, *w = experts(E, H_, I, T + E + I)
    Y, idx, gate = g.run_moe(bits, wr["bits"], w, k, renorm)
    ref = o8.moe(wl.f32_from_bf16_bits(bits), wr["values"], *w, k, renorm)
    g.check_moe(g.y_of(Y, T, "bf16"), idx, gate, ref)
    again = g.run_moe(bits, wr["bits"], w, k, renorm)[0]
    assert np.array_equal(H.host(Y), H.host(again))


# experts of 1, 4, 5, 8, 9, 16 and 17 tokens: as many as the kernels take at a time, and one more
@pytest.mark.parametrize("I", [48, 1168])
@pytest.mark.parametrize("E", [7, 70])
def test_experts_of_chosen_numbers_of_tokens(E, I):  # noqa: E741
    H_, counts = 272, [1, 4, 5, 8, 9, 16, 17]
    T = sum(counts)
    owner = np.repeat(np.arange(7), counts)
    x = wl.random_bf16(E + I, (T, H_))["values"].copy()
    x[:, :E] = 0.0
    x[np.arange(T), owner] = 8.0  # the router's row e picks feature e
    bits = wl.bf16_bits_from_f32(x)
    wr = np.zeros((E, H_), np.float32)
    wr[np.arange(E), np.arange(E)] = 1.0
    _, *w = experts(E, H_, I, E + I)
    Y, idx, gate = g.run_moe(bits, wl.bf16_bits_from_f32(wr), w, 1)
    assert np.array_equal(idx[:, 0], owner)
    g.check_moe(g.y_of(Y, T, "bf16"), idx, gate, o8.moe(wl.f32_from_bf16_bits(bits), wr, *w, 1, True))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_finite_intermediate_value_next_to_the_largest_number_stays_finite(sign):
    # h = 2^64 (2 - 2^-10) 2^63 is finite in fp32 and past every bf16 number
    H_, I = 32, 16  # noqa: E741
    x = np.zeros((1, H_), np.float32)
    x[0, 0] = 2.0 ** 60
    w13, w2 = np.zeros((1, 2, I, H_), np.uint8), np.zeros((1, H_, I), np.uint8)
    w13[0, :, 3, 0], w2[0, :, 3] = 0x38, 0x38  # 1.0
    s13 = np.array([2.0 ** 4, sign * (2 - 2.0 ** -10) * 2.0 ** 3], np.float32).reshape(1, 2, 1, 1)
    s2 = np.full((1, 1, 1), 2.0 ** -100, np.float32)
    wr = np.zeros((1, H_), np.float32)
    Y, idx, gate = g.run_moe(wl.bf16_bits_from_f32(x), wl.bf16_bits_from_f32(wr), (w13, s13, w2, s2), 1)
    y = g.y_of(Y, 1, "bf16")
    assert np.all(y == sign * 2.0 ** 28), y[0, :4]  # (2 - 2^-10) 2^27, rounded to bf16
