"""The 8-bit cache's attention in blocks of 256 queries, which long prompts and a video's
frames take: masks, windows, queries that see nothing, NaN, pages that are not there,
scales of other programs, graphs, arrays of nonsense (needs an MI355X). Which kernel a
case takes is held against the library's rules (tests/kv8_dispatch.py).

Tolerances as in tests/test_gpu_kv8.py; a scale that is no power of two costs values one
more rounding (2^-8 of each |v|).
"""

import pytest

from bit_quantized_linear_amd import binding as b
from tests import gpu_harness as H
from tests import kv8_dispatch as d
from tests.kv8_batch import PAGE, Batch64
from tests.test_gpu_norm_rope import _gpu, guarded, untouched  # noqa: F401

pytestmark = pytest.mark.gpu
NAN = float("nan")

# lengths, new, Hq, Hk
SORTED = ([706] + [700] * 29, [300] * 30, 8, 8)  # tiles in the order of all sequences' pages
ONE = ([706], [700], 100, 100)
MANY = ([200 + 37 * i % 500 for i in range(70)], [200 - i for i in range(70)], 4, 2)  # more than a wave looks at
SHARED = ([600, 80, 333, 1], [600, 77, 200, 1], 160, 32)  # heads of one key head among a block's queries
PARTS = ([4994], [300], 16, 2)
LONG = ([40000] * 3, [700] * 3, 32, 32)  # runs of more pages than are looked up at a time
SHORT = [SORTED, ONE, MANY, SHARED]
EVERY = SHORT + [PARTS, LONG]


def blocks(seed, case, D, window=0, **kw):
    x = Batch64(seed, *case, D, **kw)
    p = x.plan(window)
    assert p.rows == 256 and p.splits == d.of(*case, window=window).splits, p
    return x


def both(seed, case, window=0, **kw):
    return [blocks(seed + D, case, D, window, **kw) for D in (64, 128)]


@pytest.mark.parametrize("case", range(len(EVERY)))
def test_causal(case):
    for x in both(1, EVERY[case]):
        x.check(*x.attend())


@pytest.mark.parametrize("case", range(len(EVERY)))
def test_all_seen(case):
    for x in both(2, EVERY[case]):
        x.check(*x.attend(causal=False), causal=False)


@pytest.mark.parametrize("case,window", [(c, w) for c in range(len(SHORT)) for w in (1, 17, 64, 65, 200, 333, 5000)]
                         + [(4, 4000), (5, 100), (5, 33000)])
def test_windows(case, window):
    """Inside a page, across pages, past everything."""
    for x in both(3, EVERY[case], window):
        x.check(*x.attend(window=window), window=window)


@pytest.mark.parametrize("kw", [{}, {"causal": False}, {"window": 90}])
def test_queries_that_see_nothing(kw):
    """More new tokens than a sequence has, and sequences of no token."""
    lengths, new = [100, 0, 300, 1] * 8, [300] * 32
    for x in both(4, (lengths, new, 8, 8), kw.get("window", 0)):
        O, L = x.attend(**kw)
        assert (L.isneginf().sum() > 0) and (O[300:600] == 0).all()
        x.check(O, L, **kw)


@pytest.mark.parametrize("kw", [{}, {"causal": False}, {"window": 130}, {"window": 300}])
@pytest.mark.parametrize("case", [0, 2, 3])
def test_nan_reaches_the_queries_that_see_it(case, kw):
    """In keys and values of tokens in pages that all see, that some see, and whose other
    half is behind the window."""
    for x in both(5, EVERY[case], kw.get("window", 0)):
        n, new = x.lengths[0], x.new[0]
        for token, of, head in ((n - 1, "v", 0), (n - new // 2, "k", 1), (n - new // 3, "v", 1), (max(0, n - new - 70), "v", 0),
                                (n - min(n, new) // 4, "k", 0), (3, "k", 1)):
            page = x.pages[0][token // PAGE]
            if of == "k":
                x.kc[page, head, token % PAGE, 9] = 0xFF
            else:
                x.vc[page, head, 5 + token % 50, token % PAGE] = 0x7F
        O, L = x.attend(**kw)
        assert O.isnan().any() and not O.isnan().all()
        x.check(O, L, **kw)


@pytest.mark.parametrize("kw", [{}, {"causal": False}, {"window": 200}])
@pytest.mark.parametrize("case", [0, 2, 4])
def test_pages_that_are_not_there(case, kw):
    """The first, the last, several in a row, and the cache's first page, whose scales
    stand for those of a page that is not there: all NaN."""
    if case == 4 and "window" in kw:
        kw = {"window": 4000}
    for x in both(6, EVERY[case], kw.get("window", 0)):
        P = x.kc.shape[0]
        for s in range(0, len(x.new), 3):
            for i, number in ((0, -1), (3, P), (4, 1 << 30), (5, -(1 << 31)), (len(x.pages[s]) - 1, -1)):
                if i < len(x.pages[s]):
                    x.remove(s, i, number)
        for s, pages in enumerate(x.pages):
            if 0 in pages:
                x.remove(s, pages.index(0))
        x.ks[0], x.vs[0] = NAN, NAN
        O, L = x.attend(**kw)
        assert not O.isnan().any()
        x.check(O, L, **kw)


@pytest.mark.parametrize("case", [0, 2, 4])
def test_scales_that_are_no_powers_of_two(case):
    for kw in ({}, {"causal": False}):
        for x in both(7, EVERY[case], scales="any"):
            x.check(*x.attend(**kw), values_rounded=True, **kw)


@pytest.mark.parametrize("what", ["ks", "vs"])
def test_scales_of_0_and_far_apart(what):
    for x in both(8, SORTED):
        for i, scale in ((0, 0.0), (2, 2.0 ** -60), (3, 2.0 ** -100), (5, 0.0), (10, 0.0), (11, 0.0)):
            getattr(x, what)[x.pages[i % 3][i % len(x.pages[i % 3])]] = scale
        if what == "vs":
            x.vs[x.pages[4][4]] = 2.0 ** 60
        x.check(*x.attend())
        x.check(*x.attend(causal=False), causal=False)


def test_rising_scores():
    for x in both(9, PARTS) + both(10, SORTED):
        for pages in x.pages:
            for i, p in enumerate(pages):
                x.ks[p] = 2.0 ** (-12 + (i * 7 % 13) if i > 5 else -14 + 2 * i)
        x.check(*x.attend())


@pytest.mark.parametrize("case", range(5))
def test_the_same_bits_again(case):
    for x in both(11, EVERY[case]):
        (a, la), (c, lc) = x.attend(), x.attend()
        assert x.t.equal(a.view(x.t.int16), c.view(x.t.int16)) and x.t.equal(la, lc)


def test_without_lse_and_queries_in_wider_rows():
    t = H.torch()
    for x in both(12, SORTED):
        O, L = x.attend()
        wide = t.full((x.T, 3 * x.Hq, x.D), NAN, dtype=t.bfloat16, device="cuda")
        wide[:, x.Hq: 2 * x.Hq] = x.q
        x.q = wide[:, x.Hq: 2 * x.Hq]
        O2 = t.empty_like(O)
        x.call(O2, None, None)
        assert t.equal(O, O2)


@pytest.mark.parametrize("case", [0, 4])
def test_rows_outside_the_sequences_are_left_alone(case):
    t = H.torch()
    for x in both(13, EVERY[case]):
        O, L = x.attend()
        starts = x.starts + 5
        q = t.cat([x.q[:5], x.q, x.q[:7]])
        T = x.T + 12
        assert d.attention(T, len(x.new), x.table.shape[1], x.Hq, x.Hk).rows == 256
        O2 = t.full((T, x.Hq, x.D), 7.0, dtype=t.bfloat16, device="cuda")
        L2 = t.full((T, x.Hq), 7.0, device="cuda")
        n = b.svdq_kv8_attention_workspace_bytes(T, len(x.new), x.table.shape[1], x.Hq, x.Hk, x.D)
        ws = t.full((n,), 0xFF, dtype=t.uint8, device="cuda")
        b.svdq_kv8_attention(q, x.kc, x.ks, x.vc, x.vs, starts, x.dev_lengths, x.table, x.scale, O2, L2, ws)
        for y in (O2, L2):
            assert (y[:5] == 7.0).all() and (y[5 + x.T:] == 7.0).all()
        x.check(O2[5: 5 + x.T], L2[5: 5 + x.T])


def test_a_captured_graph_follows_the_batch():
    """Captured once, replayed while lengths and pages change, eager calls in between."""
    t = H.torch()
    for x in both(14, SORTED):
        O, L, ws = x.buffers()
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(side):
            x.call(O, L, ws)
        t.cuda.current_stream().wait_stream(side)
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            x.call(O, L, ws)
        for lengths in ([700] * 30, [300 + 13 * i for i in range(30)], [10, 0] * 15, [706] + [700 - i for i in range(29)]):
            x.dev_lengths.copy_(t.tensor(lengths, dtype=t.int32))
            x.q.copy_(t.randn(x.q.shape, generator=x.gen, device="cuda"))
            O.fill_(7.0)
            g.replay()
            t.cuda.synchronize()
            got = O.clone(), L.clone()
            x.call(O, L, ws)
            t.cuda.synchronize()
            assert t.equal(got[0].view(t.int16), O.view(t.int16)) and t.equal(got[1], L)
            x.lengths = lengths
            _cut(x).check(O, L)


def _cut(x):
    """Pages of a sequence as far as its length reaches."""
    out = object.__new__(Batch64)
    out.__dict__.update(x.__dict__)
    out.pages = [p[: -(-n // PAGE)] for p, n in zip(x.pages, x.lengths)]
    return out


def test_streams_at_the_same_time():
    t = H.torch()
    x = [blocks(15 + i, c, 128) for i, c in enumerate((SORTED, PARTS, MANY))]
    out = [y.buffers() for y in x]
    streams = [t.cuda.Stream() for _ in x]
    t.cuda.synchronize()
    for _ in range(3):
        for y, o, s in zip(x, out, streams):
            y.call(*o, stream=s)
    t.cuda.synchronize()
    for y, o in zip(x, out):
        y.check(o[0], o[1])


# T, Hq, Hk, width of the table: blocks of 256 queries in order and in parts, of 128 in
# parts and in one, and few in parts
NONSENSE = [(700, 100, 100, 2), (700, 4, 2, 70), (300, 4, 2, 40), (300, 2, 2, 2), (3, 4, 2, 40), (30, 8, 2, 300)]


@pytest.mark.parametrize("starts,lengths", [
    ([0, 50, 7], [100, 90]), ([-5, 4, 90], [100, 5000]), ([3, 3, 2147483647], [-4, 100]),
    ([-2147483648, 2, 40], [2147483647, -2147483648]), ([0, 2147483647, 0], [2147483647, 2147483647]),
    ([600, 10, 650], [70, 2147483647]), ([2147483647, 0, 700], [5, 64])])
@pytest.mark.parametrize("case", range(len(NONSENSE)))
def test_arrays_of_nonsense_stay_inside_the_buffers(case, starts, lengths):
    """Held to the buffers: nothing outside them is written, whatever they say."""
    t = H.torch()
    T, Hq, Hk, width = NONSENSE[case]
    gen = t.Generator(device="cuda").manual_seed(case)
    P, D = 9, 64
    table = t.randint(-3, P + 3, (2, width), generator=gen, device="cuda", dtype=t.int32)
    table[1, width // 2], table[0, 1] = 1 << 30, -2147483648
    codes = lambda *s: t.randint(0, 0x7E, s, generator=gen, device="cuda", dtype=t.uint8)  # noqa: E731
    whole = [guarded(s, t.uint8) for s in ((P, Hk, PAGE, D), (P, Hk, D, PAGE))]
    for view, _ in whole:
        view.copy_(codes(*view.shape))
    scale = t.full((P, Hk), 2.0 ** -6, device="cuda")
    q = t.randn((T, Hq, D), generator=gen, device="cuda").bfloat16()
    O, o_all = guarded((T, Hq, D), t.bfloat16)  # noqa: E741
    L, l_all = guarded((T, Hq), t.float32)
    n = b.svdq_kv8_attention_workspace_bytes(T, 2, width, Hq, Hk, D)
    ws = t.full((n + 64,), 0xA5, dtype=t.uint8, device="cuda")
    whole32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
    for kw in ({}, {"causal": False}, {"window": 70}):
        b.svdq_kv8_attention(q, whole[0][0], scale, whole[1][0], scale, whole32(starts), whole32(lengths), table, 0.125, O, L,
                             ws, **kw)
    t.cuda.synchronize()
    for w in (o_all, l_all, ws, whole[0][1], whole[1][1]):
        untouched(w)
