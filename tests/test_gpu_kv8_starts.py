"""Row starts of the 8-bit cache's attention that fall: a sequence whose next start is not
above its own has no new tokens, and the others keep theirs, however a call is cut
(needs an MI355X). Tolerances as in tests/test_gpu_kv8.py."""

import pytest

from bit_quantized_linear_amd import binding as b
from tests import gpu_harness as H
from tests.kv8_batch import Batch64
from tests.test_gpu_norm_rope import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,new,Hq,Hk,parts", [
    ([3000, 200], [1, 1], 8, 2, (9, 64)), ([1100, 1050], [2, 1], 8, 8, (2, 8)), ([200, 100], [2, 1], 4, 2, (1, 1)),
    ([6000], [300], 2, 2, (2, 64)), ([2500, 100], [120, 100], 2, 1, (2, 64)), ([300, 200], [100, 30], 4, 4, (1, 1))])
@pytest.mark.parametrize("fill", [0, -1, 1])
def test_starts_that_fall_behind_the_last_sequence(lengths, new, Hq, Hk, parts, fill):
    """A batch of fixed size whose unused entries hold 0, or what was there before."""
    t = H.torch()
    for D in (64, 128):
        x = Batch64(D, lengths, new, Hq, Hk, D)
        O, L = x.attend()
        x.check(O, L)
        # three sequences more, without new tokens
        whole = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
        y = Batch64(D, lengths, new, Hq, Hk, D)
        y.starts = t.cat([x.starts, whole([fill] * 3)])
        y.dev_lengths = t.cat([x.dev_lengths, whole([0, 70, 0])])
        y.table = t.cat([x.table, x.table.new_full((3, x.table.shape[1]), -1)])
        y.new, count = new + [0] * 3, y.T
        assert parts[0] <= y.parts() <= parts[1], y.parts()
        O2, L2, ws = y.buffers()
        O2.fill_(7.0)
        L2.fill_(7.0)
        y.call(O2, L2, ws)
        assert count == x.T and t.count_nonzero(L2 == 7.0).item() == 0
        x.check(O2, L2)


@pytest.mark.parametrize("parts", [1, 12])
def test_rows_of_no_sequence_between_starts_that_fall(parts):
    """Rows 2 .. 4 belong to nobody: they keep what they hold."""
    t = H.torch()
    n = 3000 if parts > 1 else 200
    x = Batch64(1, [n, n - 30], [2, 2], 4, 2, 64)
    whole = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    y = Batch64(1, [n, n - 30], [2, 2], 4, 2, 64)
    # sequence 0 has rows 5 and 6, the next none, the third rows 0 and 1
    y.T, y.new = 7, [2, 0, 2]
    y.starts, y.dev_lengths = whole([5, 7, 0, 2]), whole([n, 0, n - 30])
    y.table = t.stack([x.table[0], t.full_like(x.table[0], -1), x.table[1]])
    y.q = t.zeros((7, 4, 64), dtype=t.bfloat16, device="cuda")
    y.q[5:7], y.q[0:2] = x.q[:2], x.q[2:]
    assert y.parts() == parts if parts == 1 else y.parts() > 1
    O, L, ws = y.buffers()  # noqa: E741
    O.fill_(7.0)
    L.fill_(7.0)
    y.call(O, L, ws)
    assert (O[2:5] == 7.0).all() and (L[2:5] == 7.0).all()
    x.check(t.cat([O[5:7], O[0:2]]), t.cat([L[5:7], L[0:2]]))


@pytest.mark.parametrize("fill", [0, -1, 1])
def test_append_of_a_batch_whose_last_starts_fall(fill):
    t = H.torch()
    for D in (64, 128):
        x = Batch64(D, [130, 200], [70, 3], 2, 2, D)
        k, v = (t.randn((x.T, 2, D), generator=x.gen, device="cuda").bfloat16() for _ in range(2))
        whole = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
        caches = [[c.clone() for c in (x.kc, x.ks, x.vc, x.vs)] for _ in range(2)]
        b.svdq_kv8_append(k, v, x.starts, x.dev_lengths, x.table, *caches[0])
        b.svdq_kv8_append(k, v, t.cat([x.starts, whole([fill] * 3)]), t.cat([x.dev_lengths, whole([0, 70, 64])]),
                          t.cat([x.table, x.table.new_full((3, x.table.shape[1]), 1)]), *caches[1])
        for a, c in zip(*caches):
            assert t.equal(a.view(t.uint8), c.view(t.uint8))
        assert not t.equal(caches[0][0], x.kc)
