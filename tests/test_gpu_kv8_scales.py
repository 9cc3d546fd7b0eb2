"""Page scales of the 8-bit cache that are not finite, and factors of scores (scale times
a page's key scale) far below 1, in every kernel of the attention (needs an MI355X).

A page whose key scale is not finite has NaN for its scores: the queries that see one of
its tokens have NaN for output and logarithm. One whose value scale is not finite has NaN
for its values: NaN outputs, the same logarithms. Queries that see none of its tokens, and
other heads, are not touched. Tolerances as in tests/test_gpu_kv8.py.
"""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from oracle import decoder as od
from oracle.fp8 import e4m3_decode
from tests import gpu_harness as H
from tests.kv8_batch import KERNELS, PAGE, batch, kernel_id
from tests.test_gpu_kv8 import bf16_dev, bf16_values, random_cache, upload
from tests.test_gpu_norm_rope import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
SPOILED = ["ks", "vs"]


def spoil(x, what, value, page, head=0):
    getattr(x, what)[x.pages[0][page], head] = value


@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("what", SPOILED)
@pytest.mark.parametrize("case", KERNELS, ids=kernel_id)
def test_a_scale_that_is_not_finite(case, what, value):
    """Of the first sequence's last page, which its last two tokens alone see."""
    for D in (64, 128):
        x = batch(D, case, D)
        spoil(x, what, value, len(x.pages[0]) - 1)
        O, L = x.attend()
        new, group = x.new[0], x.Hq // x.Hk
        assert O[new - 2: new, :group].isnan().all() and not O[: new - 2].isnan().any() and not O[new:].isnan().any()
        assert not O[:, group:].isnan().any()
        x.check(O, L)


@pytest.mark.parametrize("what", SPOILED)
@pytest.mark.parametrize("case", KERNELS, ids=kernel_id)
def test_a_scale_that_is_not_finite_behind_a_window(case, what):
    """A page that leaves the window within the call, and one that nobody sees."""
    far = case[2][0] > 2000
    window = 2000 + PAGE * 2 if far else 65
    if case[:2] == (256, True):
        window = 4000  # as many parts as leave it its blocks of 256
    x = batch(3, case, 128, window)
    # the first query sees its page, the last does not
    first = max(0, x.lengths[0] - x.new[0] + 1 - window) // PAGE
    spoil(x, what, NAN, first)
    if first > 0:
        spoil(x, what, NAN, first - 1)
    O, L = x.attend(window=window)
    x.check(O, L, window=window)


@pytest.mark.parametrize("what", SPOILED)
@pytest.mark.parametrize("case", KERNELS, ids=kernel_id)
def test_a_scale_that_is_not_finite_and_seen_by_all(case, what):
    x = batch(4, case, 64)
    spoil(x, what, INF, 1, head=1)
    O, L = x.attend(causal=False)
    group = x.Hq // x.Hk
    assert O[: x.new[0], group: 2 * group].isnan().all() and not O[x.new[0]:].isnan().any()
    x.check(O, L, causal=False)


@pytest.mark.parametrize("case", KERNELS, ids=kernel_id)
def test_a_scale_of_no_power_of_two_beside_one_that_is_not_finite(case):
    x = batch(5, case, 128, scales="any")
    spoil(x, "vs", NAN, len(x.pages[0]) - 1)
    O, L = x.attend()
    x.check(O, L, values_rounded=case[0] > 64)


@pytest.mark.parametrize("case", KERNELS, ids=kernel_id)
def test_factors_below_the_smallest_normal_number(case):
    """Queries near 2^112, scale 2^-112, key scales of 2^-20 to 2^-14: scores are ordinary,
    their factors lie on both sides of 2^-126."""
    x = batch(6, case, 64, spread=2.0 ** 112)
    x.scale = 2.0 ** -112
    x.ks.copy_(x.t.exp2(x.t.randint(-20, -13, x.ks.shape, generator=x.gen, device="cuda").float()))
    assert x.t.isfinite(x.q).all()
    O, L = x.attend()
    x.check(O, L)
    x.ks.mul_(2.0 ** -10)  # no score matters any more: the values' mean
    O, L = x.attend()
    x.check(O, L)


@pytest.mark.parametrize("power", [-110, 90])
@pytest.mark.parametrize("case", KERNELS, ids=kernel_id)
def test_values_near_the_ends_of_the_range(case, power):
    """Values near 2^-108 (weights times their scale are subnormal) and near 2^92, whose
    sums are numbers: 64 times 6018 tokens leave 2^18."""
    for spread in (0.2, 3.0):
        x = batch(7, case, 64, spread=spread)
        x.vs.mul_(2.0 ** power)
        O, L = x.attend()
        assert x.t.isfinite(O).all() and (O != 0).any()
        x.check(O, L)


@pytest.mark.parametrize("old", [0.0, 0.0131, 2.0 ** -20, 2.0 ** 20, INF, NAN])
@pytest.mark.parametrize("D", [64, 128])
def test_append_behind_tokens_of_another_programs_scale(old, D):
    """s = max(need, old), codes E4M3(fp32(x fp32(1 / s))), earlier ones E4M3(fp32(code
    fp32(old / s))), byte for byte; where the scale is no number, the earlier tokens are
    NaN, by their codes or by the scale that stays."""
    t = H.torch()
    rng = np.random.default_rng(D)
    Hk, length, new, low = 2, 45, 7, 38
    cache = random_cache(rng, 3, Hk, D)
    cache.ks[1], cache.vs[1] = old, old
    rows = bf16_values(rng, (new, 2 * Hk, D), 3.0)
    dev, tensors = bf16_dev(rows), upload(cache)
    whole = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    b.svdq_kv8_append(dev[:, :Hk], dev[:, Hk:], whole([0, new]), whole([length]), whole([[1]]), *tensors)
    kc, ks, vc, vs = (H.host(x) for x in tensors)
    f32 = np.float32
    for codes, scales, was, x in ((kc, ks, cache.kc, rows[:, :Hk]), (vc.transpose(0, 1, 3, 2), vs, cache.vc.transpose(0, 1, 3, 2),
                                                                  rows[:, Hk:])):
        assert np.array_equal(codes[[0, 2]], was[[0, 2]]) and np.array_equal(codes[1, :, length:], was[1, :, length:])
        for h in range(Hk):
            need = od.page_scale(np.abs(x[:, h].astype(np.float64)).max())
            s = f32(need if np.isnan(old) else max(need, old))
            assert scales[1, h] == s
            with np.errstate(invalid="ignore"):
                fresh, ratio = od.encode(x[:, h].astype(f32) * (f32(1) / s)), f32(old) / s
                kept = was[1, h, :low] if s == f32(old) else od.encode(e4m3_decode(was[1, h, :low]).astype(f32) * ratio)
            for got, want in ((codes[1, h, low:length], fresh), (codes[1, h, :low], kept)):
                got, want = (np.where((c & 0x7F) == 0, 0, np.where((c & 0x7F) == 0x7F, 0x7F, c)) for c in (got, want))
                assert np.array_equal(got, want)  # the signs of 0 and NaN are open
    if not np.isfinite(old):
        earlier = e4m3_decode(kc[1, :, :low]) * ks[1][:, None, None]
        assert not np.isfinite(ks[1]).all() or np.isnan(earlier).all()
