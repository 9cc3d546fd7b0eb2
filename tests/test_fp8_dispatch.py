"""The shapes of the block-scaled FP8 GPU tests against the library's rules: each
kernel and variant that a call can reach is reached by one of them. No GPU."""

import random

import pytest

from tests import fp8_dispatch as d
from tests import test_gpu_fp8 as g
from tests import test_gpu_fp8_paths as paths

MANY = [(4100, 400, 2056, "bf16"), (2300, 1936, 4360, "f32"), (6000, 128, 2048, "bf16"), (1700, 400, 2056, "bf16"),
        (1700, 400, 2056, "f32"), (2100, 272, 2056, "f32"), (2100, 272, 2056, "bf16"), (900, 1040, 1544, "bf16"),
        (900, 1040, 1544, "f32")]  # of test_linear_many_tokens


def _sizes(rng, *ranges):
    return [max(lo, min(hi, round(lo * (hi / lo) ** rng.random() / step) * step)) for lo, hi, step in ranges]


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_every_linear_kernel_has_a_test(out):
    rng = random.Random(1)
    both = g.SHAPES + g.WIDE + paths.TURNED + (paths.LARGE if out == "bf16" else [])
    tested = {d.linear(*s, out) for s in both} | {d.product(*s, out) for s in both}
    tested |= {d.linear(*s) for s in MANY if s[3] == out}
    reached = set()
    for _ in range(40000):
        M, K, N = _sizes(rng, (1, 32768, 1), (16, 16384, 16), (8, 32768, 8))
        K = rng.choice([K, K, 4096, 8192])
        reached |= {d.linear(M, K, N, out), d.product(M, K, N, out)}
    assert len(reached) > 10 and reached <= tested, sorted(map(str, reached - tested))


def test_every_expert_kernel_has_a_test():
    rng = random.Random(2)
    shapes = g.MOE + paths.EXPERTS
    up, down = {d.experts(*s)[0] for s in shapes}, {d.experts(*s)[1] for s in shapes}
    for _ in range(40000):
        T, H, I, E = _sizes(rng, (1, 64, 1), (16, 8192, 16), (16, 20000, 16), (1, 256, 1))  # noqa: E741
        H = rng.choice([H, H, 4096, 8192])
        u, v = d.experts(T, H, I, E, rng.randint(1, min(E, 16)))
        assert u in up and v in down, (T, H, I, E, u, v)
