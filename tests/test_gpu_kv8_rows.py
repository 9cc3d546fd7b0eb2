"""The 8-bit cache's attention where a sequence has 17 to 64 queries of a key head: a
few drafted tokens, or one of many heads (needs an MI355X).

Tolerances as in tests/test_gpu_kv8.py and tests/test_gpu_kv8_paths.py.
"""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from oracle import decoder as od
from tests import gpu_harness as H
from tests.test_gpu_kv8 import PAGE, attend, attention_case, bf16_values, check, plan, poison, random_cache
from tests.test_gpu_kv8_paths import run
from tests.test_gpu_norm_rope import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,new,Hq,Hk", [
    ([17], [17], 1, 1), ([64], [4], 16, 2), ([65], [33], 1, 1), ([130], [64], 1, 1), ([300, 2, 66], [8, 2, 3], 16, 2),
    ([333, 50, 700], [3, 20, 60], 2, 2), ([700, 64, 0, 5], [9, 1, 0, 5], 10, 2), ([200], [1], 40, 1), ([129, 400], [1, 1], 64, 1),
    ([100, 100, 100], [90, 1, 1], 1, 1), ([100, 500], [90, 3], 1, 1)])
def test_rows(lengths, new, Hq, Hk, D):
    assert 16 * len(new) < sum(new) * (Hq // Hk) <= 64 * len(new)
    attention_case(sum(lengths) + D, lengths, new, Hq, Hk, D)


@pytest.mark.parametrize("lengths,new,Hq,Hk,causal,window", [
    ([300, 70], [20, 9], 4, 2, False, 0), ([300, 70], [9, 10], 4, 2, True, 100), ([300], [12], 4, 2, True, 1),
    ([300, 64], [16, 64], 1, 1, True, 64), ([400], [60], 1, 1, True, 5), ([500], [20], 2, 1, True, 129)])
def test_masks(lengths, new, Hq, Hk, causal, window):
    for D in (64, 128):
        attention_case(window + D, lengths, new, Hq, Hk, D, causal, window)


@pytest.mark.parametrize("new", [[12, 8, 9], [30, 3, 20]])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_that_see_nothing(new, causal):
    attention_case(31, [10, 0, 0], new, 4, 2, 64, causal=causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,new,Hq,Hk,parts", [
    ([20001], [5], 8, 2, (9, 64)), ([20001, 70], [32, 10], 4, 2, (9, 64)), ([3000] * 40, [2] * 40, 80, 8, (1, 1)),
    ([18000] + [100] * 35, [8] * 36, 32, 8, (2, 8)), ([2000] * 3, [60] * 3, 1, 1, (2, 64))])
def test_long_contexts(lengths, new, Hq, Hk, parts, D):
    run(sum(lengths) + D, lengths, new, Hq, Hk, D, parts)


@pytest.mark.parametrize("kw", [{"causal": False}, {"window": 1000}, {"window": 257}])
def test_masks_over_many_pages(kw):
    for new in (20, 60):
        run(7 + new, [6000], [new], 1, 1, 128, **kw)


def test_scales_that_are_no_powers_of_two():
    for D in (64, 128):
        run(9 + D, [3000, 100], [20, 50], 2, 2, D, scales="any")


@pytest.mark.parametrize("new", [20, 50])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_reaches_the_queries_that_see_it(new, D):
    rng = np.random.default_rng(14)
    lengths, Hq, Hk = [200], 2, 2
    starts, table, P = plan(rng, lengths, [new])
    Q = bf16_values(rng, (new, Hq, D))
    for what, token, window in (("v", 199 - new // 2, 0), ("k", 199 - new // 2, 0), ("v", 150, 60), ("k", 150, 60), ("v", 3, 0)):
        cache = random_cache(rng, P, Hk, D)
        poison(cache, lengths, table)
        page, at = table[0, token // PAGE], token % PAGE
        if what == "v":
            cache.vc[page, 0, 5, at] = 0x7F
        else:
            cache.kc[page, 1, at, 9] = 0xFF
        got = attend(Q, cache, starts, lengths, table, 0.125, window=window)
        ref = od.attention(Q, cache, starts, lengths, table, 0.125, True, window)
        assert np.isnan(ref["o"]).any()
        check(got, ref, lengths, D)


@pytest.mark.parametrize("new", [20, 50])
def test_pages_that_are_not_there(new):
    rng = np.random.default_rng(15)
    for D in (64, 128):
        lengths = [700, 90]
        starts, table, P = plan(rng, lengths, [new, 3])
        cache = random_cache(rng, P, 2, D)
        table[0, 0], table[0, 5], table[0, 10], table[1, 0] = -1, P, -9, P + 4
        poison(cache, lengths, table)
        Q = bf16_values(rng, (new + 3, 2, D))
        ref = od.attention(Q, cache, starts, lengths, table, 0.125)
        check(attend(Q, cache, starts, lengths, table, 0.125), ref, lengths, D)


@pytest.mark.parametrize("new,window", [(1, 100), (1, 2000), (20, 64), (60, 700), (200, 300), (300, 64)])
def test_windows_much_shorter_than_the_context(new, window):
    """As many parts as the window's pages ask for, fewer than the workspace holds."""
    for D in (64, 128):
        run(new + D, [20000, 300], [new, 1], 4, 2, D, window=window)


@pytest.mark.parametrize("lengths,new,Hq,Hk,kw", [
    ([300], [300], 8, 2, {}), ([700, 40], [600, 40], 8, 8, {}), ([5000], [300], 16, 2, {}), ([5000], [300], 16, 2, {"window": 700}),
    ([3000, 200], [1000, 200], 4, 1, {"causal": False}), ([1400], [1400], 32, 8, {}), ([4000], [1100], 8, 8, {"window": 100})])
def test_prompts_that_leave_units_idle(lengths, new, Hq, Hk, kw):
    """More than 128 queries of a key head, in blocks of 128."""
    for D in (64, 128):
        run(sum(lengths) + D, lengths, new, Hq, Hk, D, **kw)


@pytest.mark.parametrize("lengths,new,Hq,Hk,kw", [
    ([700] + [300] * 15, [200] + [1] * 15, 4, 1, {}), ([300] * 7 + [500], [1] * 7 + [100], 8, 2, {}),
    ([200, 1, 900, 64, 65], [1, 0, 90, 2, 33], 4, 2, {}), ([3000] * 70, [1] * 40 + [33] + [2] * 29, 16, 2, {}),
    ([4000, 100, 100, 100], [150, 1, 1, 1], 1, 1, {"window": 300}), ([4000, 100, 100, 100], [150, 1, 1, 1], 1, 1, {"causal": False})])
def test_a_prompt_among_decoded_tokens(lengths, new, Hq, Hk, kw):
    """Sequences with more queries than a block of the kernel for few takes."""
    assert max(new) * (Hq // Hk) > 64 and sum(new) * (Hq // Hk) <= 64 * len(new)
    for D in (64, 128):
        run(sum(lengths) + D, lengths, new, Hq, Hk, D, **kw)


def test_more_blocks_than_a_grid_dimension_has():
    """50000 sequences of two pages' halves: every other one has two new tokens of 16
    heads, two blocks, and the others have none."""
    t, B, D, heads = H.torch(), 50000, 64, 16
    gen = t.Generator(device="cuda").manual_seed(3)
    codes = lambda *s: t.randn(s, generator=gen, device="cuda").mul_(64).to(t.float8_e4m3fn)  # noqa: E731
    kc, vc = t.full((B, 1, 64, D), 0x7F, dtype=t.uint8, device="cuda"), t.full((B, 1, D, 64), 0xFF, dtype=t.uint8, device="cuda")
    k, v = codes(B, 2, D), codes(B, 2, D)
    kc[:, 0, :2], vc[:, 0, :, :2] = k.view(t.uint8), v.view(t.uint8).transpose(1, 2)
    scale = t.full((B, 1), 2.0 ** -6, device="cuda")
    new = t.tensor([2, 0], device="cuda").repeat(B // 2)
    starts = t.cat([t.zeros(1, dtype=t.long, device="cuda"), new.cumsum(0)]).int()
    q = t.randn((B, heads, D), generator=gen, device="cuda").bfloat16()
    O = t.zeros((B, heads, D), dtype=t.bfloat16, device="cuda")  # noqa: E741
    table = t.arange(B, dtype=t.int32, device="cuda")[:, None].contiguous()
    assert b.svdq_kv8_attention_workspace_bytes(B, B, 1, heads, 1, D) == 0
    b.svdq_kv8_attention(q, kc, scale, vc, scale, starts, new.int(), table, 0.125, O)
    k, v = (x.float()[::2].double() / 64 for x in (k, v))
    s = 0.125 * t.einsum("bthd,bud->bthu", q.double().view(B // 2, 2, heads, D), k)
    s[:, 0, :, 1] = -float("inf")
    p = t.softmax(s, -1)
    want = (p[..., None] * v[:, None, None]).sum(-2).reshape(B, heads, D)
    mag = (p[..., None] * v[:, None, None].abs()).sum(-2).reshape(B, heads, D)
    off = (O.double() - want).abs()
    # half steps of bf16 of the output and of each weight; scores of up to 128 terms, fp32
    assert (off <= 2.0 ** -8 * want.abs() + mag * (2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -12)).all()
