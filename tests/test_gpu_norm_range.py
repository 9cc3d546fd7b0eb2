"""The norm before the block-scaled FP8 linears at the ends of bf16's range: every finite
token has finite outputs, for eps = 0 as well, as long as its own formula has (needs an
MI355X). Tolerances as in tests/test_gpu_norm_rope.py."""

import numpy as np
import pytest

from bit_quantized_linear_amd import workloads as wl
from oracle import decoder as od
from tests import gpu_harness as H
from tests.test_gpu_norm_rope import _gpu, bf16, norm_call, norm_check, values  # noqa: F401

pytestmark = pytest.mark.gpu
LEAST, MOST = 2.0 ** -133, 2.0 ** 127 * (2 - 2.0 ** -7)  # of bf16: the smallest, subnormal; the largest


def rows(K):
    """Tokens of bf16 values (float64), one kind each."""
    rng = np.random.default_rng(K)
    x = np.zeros((10, K))
    x[0, K // 3] = 2.0 ** -126
    x[1, K - 1] = LEAST
    x[2] = LEAST * rng.integers(-5, 6, K)  # subnormal throughout
    x[2, 0] = LEAST
    x[3] = 2.0 ** -120 * rng.standard_normal(K)
    x[4] = rng.choice([-MOST, MOST], K)
    x[5, 1] = -MOST
    x[6] = 2.0 ** 126 * np.clip(rng.standard_normal(K), -1.9, 1.9)
    x[7] = rng.standard_normal(K)
    x[8] = rng.standard_normal(K) * np.exp2(rng.integers(-126, 126, K))
    x[9] = LEAST
    bits = wl.bf16_bits_from_f32(x.astype(np.float32))
    return wl.f32_from_bf16_bits(bits).astype(np.float64), H.dev(bits).view(H.torch().bfloat16)


@pytest.mark.parametrize("K", [16, 96, 256, 400, 1024, 2048, 4096, 5120, 8192, 20000])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-6])
def test_finite_tokens_stay_finite(K, eps):
    xv, x = rows(K)
    wv, w = bf16(K, (K,), 0.5)
    got = norm_call(x, None, w, eps)
    ref = od.norm(xv, None, wv, np.float64(np.float32(eps)))
    assert np.isfinite(ref["y"]).all() and np.isfinite(values(got["Y"])).all() and np.isfinite(H.host(got["sx"])).all()
    norm_check(got, ref)


@pytest.mark.parametrize("M", [10, 1030])
def test_with_a_residual_and_the_sum(M):
    """h near the largest and below the smallest normal number, as a sum of two."""
    K = 512
    rng = np.random.default_rng(5)
    a, b = (np.zeros((M, K), np.float32) for _ in range(2))
    a[::2] = 0.49 * MOST * rng.choice([-1, 1], (len(a[::2]), K))
    b[::2] = a[::2]
    a[1::2] = LEAST * rng.integers(-9, 10, (len(a[1::2]), K))
    b[1::2] = LEAST * 3
    a, b = (wl.bf16_bits_from_f32(v) for v in (a, b))
    wv, w = bf16(6, (K,))
    dev = lambda v: H.dev(v).view(H.torch().bfloat16)  # noqa: E731
    got = norm_call(dev(a), dev(b), w, 0.0)
    norm_check(got, od.norm(wl.f32_from_bf16_bits(a), wl.f32_from_bf16_bits(b), wv, 0.0))


def test_a_token_of_zeros_without_eps_is_nan_and_leaves_the_others():
    xv, x = rows(256)
    x[7] = 0.0
    wv, w = bf16(7, (256,))
    got = norm_call(x, None, w, 0.0)
    assert np.isnan(values(got["Y"])[7]).all() and np.isnan(H.host(got["sx"])[:, 7]).all()
    rest = [i for i in range(len(xv)) if i != 7]
    ref = od.norm(xv[rest], None, wv, 0.0)
    norm_check({"Y": got["Y"][rest], "sum": got["sum"][rest], "qx": got["qx"][rest], "sx": got["sx"][:, rest]}, ref)
