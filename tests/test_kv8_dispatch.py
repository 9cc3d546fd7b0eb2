"""The rules of tests/kv8_dispatch.py against the library's own, and what the batches of
tests/kv8_batch.py reach by them. No GPU."""

import random

import pytest

from bit_quantized_linear_amd import binding as b
from tests import kv8_dispatch as d


def test_parts_are_the_workspaces():
    """The workspace holds each part of each query: its size tells how many there are."""
    rng = random.Random(1)
    size = lambda low, high: round(low * (high / low) ** rng.random())  # noqa: E731
    for _ in range(20000):
        Hk, B, T, pages, D = size(1, 64), size(1, 300), size(1, 20000), size(1, 2048), rng.choice([64, 128])
        Hq = Hk * size(1, 32)
        assert b.svdq_kv8_attention_workspace_bytes(T, B, pages, Hq, Hk, D) == d.workspace(T, B, pages, Hq, Hk, D)


def test_the_batches_reach_the_kernels_that_they_name():
    pytest.importorskip("torch")
    from tests.kv8_batch import KERNELS

    assert {c[:2] for c in KERNELS} == {(r, p) for r in (16, 32, 64, 128, 256) for p in (False, True)}
    for rows, parts, *sizes in KERNELS:
        plan = d.of(*sizes)
        assert plan.rows == rows and (plan.splits > 1) == parts, (sizes, plan)


def test_the_cases_of_long_prompts_reach_blocks_of_256():
    pytest.importorskip("torch")
    from tests import test_gpu_kv8_blocks as blocks

    plans = [d.of(*case) for case in blocks.EVERY]
    assert all(p.rows == 256 for p in plans)
    assert {(p.splits > 1, p.sorted) for p in plans} == {(False, True), (False, False), (True, False)}
    assert len(blocks.MANY[0]) > 64 and max(blocks.LONG[0]) > 512 * 64
    cuts = [d.attention(T, 2, width, Hq, Hk) for T, Hq, Hk, width in blocks.NONSENSE]
    assert [(p.rows, p.splits > 1) for p in cuts] == [(256, False), (128, True), (128, True), (128, False), (16, True), (64, True)]
    assert cuts[0].sorted
