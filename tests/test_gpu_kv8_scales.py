"""Page scales of the 8-bit cache that are not finite, and factors of scores (scale times
a page's key scale) far below 1, in every kernel of the attention (needs an MI355X).

A page whose key scale is not finite has NaN for its scores: the queries that see one of
its tokens have NaN for output and logarithm. One whose value scale is not finite has NaN
for its values: NaN outputs, the same logarithms. Queries that see none of its tokens, and
other heads, are not touched. Tolerances as in tests/test_gpu_kv8.py.
"""

import pytest

from tests.kv8_batch import KERNELS, PAGE, batch, kernel_id
from tests.test_gpu_norm_rope import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
SPOILED = ["ks", "vs"]


def spoil(x, what, value, page, head=0):
    getattr(x, what)[x.pages[0][page], head] = value


@pytest.mark.parametrize("value", [NAN, INF])
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
