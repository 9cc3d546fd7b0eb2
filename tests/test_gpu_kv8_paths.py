"""Every way in which the 8-bit cache's attention is cut, on sizes where its loops
run long, against float64 products on the GPU; captured and replayed graphs, other
streams, calls at the same time; scales that the library does not write itself
(needs an MI355X).

Tolerances as in tests/test_gpu_kv8.py. A scale that is no power of two costs values
one more rounding to bf16 where many queries share a page (2^-8 of each |v|).
"""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from oracle.fp8 import _BYTES
from tests import gpu_harness as H
from tests.test_gpu_norm_rope import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu
PAGE = 64


class Batch:
    """A random cache and queries on the GPU; NaN codes where no query looks."""

    def __init__(self, seed, lengths, new, Hq, Hk, D, scales="powers", spread=1.5, width=None):
        t = self.t = H.torch()
        gen = self.gen = t.Generator(device="cuda").manual_seed(seed)
        self.lengths, self.new, self.Hq, self.Hk, self.D = lengths, new, Hq, Hk, D
        used = [-(-n // PAGE) for n in lengths]
        P = sum(used) + 2
        order = t.randperm(P, generator=gen, device="cuda").tolist()
        width = width or max(1, max(used))
        self.pages, at = [], 0
        for n in used:
            self.pages.append(order[at: at + n])
            at += n
        codes = lambda *s: t.randn(s, generator=gen, device="cuda").mul_(64).clamp_(-448, 448).to(t.float8_e4m3fn)  # noqa: E731
        self.kc, self.vc = codes(P, Hk, PAGE, D).view(t.uint8), codes(P, Hk, D, PAGE).view(t.uint8)
        if scales == "powers":
            scale = lambda: t.exp2(t.randint(-8, -4, (P, Hk), generator=gen, device="cuda").float())  # noqa: E731
        else:
            scale = lambda: t.rand((P, Hk), generator=gen, device="cuda") * 0.02 + 0.003  # noqa: E731
        self.ks, self.vs = scale(), scale()
        seen = t.zeros((P, PAGE), dtype=t.bool, device="cuda")
        for n, pages in zip(lengths, self.pages):
            for i, p in enumerate(pages):
                seen[p, : min(PAGE, n - PAGE * i)] = True
        self.kc.masked_fill_(~seen[:, None, :, None], 0x7F)
        self.vc.masked_fill_(~seen[:, None, None, :], 0xFF)
        whole = lambda v: t.tensor(v, dtype=t.int32, device="cuda")  # noqa: E731
        self.starts = whole(np.concatenate([[0], np.cumsum(new)]).tolist())
        self.dev_lengths = whole(lengths)
        self.table = whole([p + [-1] * (width - len(p)) for p in self.pages])
        self.T = sum(new)
        self.q = t.randn((self.T, Hq, D), generator=gen, device="cuda").mul_(spread).bfloat16()
        self.scale = float(np.float32(1 / np.sqrt(D)))

    def parts(self):
        n = b.svdq_kv8_attention_workspace_bytes(self.T, len(self.new), self.table.shape[1], self.Hq, self.Hk, self.D)
        per = 4 * self.T * self.Hq * (self.D + 2)
        assert n % per == 0
        return max(1, n // per)

    def buffers(self):
        t = self.t
        n = b.svdq_kv8_attention_workspace_bytes(self.T, len(self.new), self.table.shape[1], self.Hq, self.Hk, self.D)
        return (t.empty((self.T, self.Hq, self.D), dtype=t.bfloat16, device="cuda"), t.empty((self.T, self.Hq), device="cuda"),
                t.full((n,), 0xFF, dtype=t.uint8, device="cuda"))

    def call(self, O, L, ws, **kw):  # noqa: E741
        b.svdq_kv8_attention(self.q, self.kc, self.ks, self.vc, self.vs, self.starts, self.dev_lengths, self.table, self.scale,
                             O, L, ws, **kw)

    def reference(self, causal=True, window=0):
        """o, lse, sum p |v|, sum p^2 v^2 and the largest sum of |products|, float64."""
        t = self.t
        table = t.tensor(_BYTES, device="cuda")
        out = [t.zeros((self.T, self.Hq, self.D), dtype=t.float64, device="cuda") for _ in range(3)]
        lse, score = (t.zeros((self.T, self.Hq), dtype=t.float64, device="cuda") for _ in range(2))
        row = 0
        for n, new, pages in zip(self.lengths, self.new, self.pages):
            p = t.tensor(pages, dtype=t.long, device="cuda")
            pos = t.arange(n - new, n, device="cuda")[:, None]
            at = t.arange(n, device="cuda")
            hidden = (at > pos) if causal else t.zeros((new, n), dtype=t.bool, device="cuda")
            if window:
                hidden = hidden | (at <= pos - window)
            for g in range(self.Hk):
                k = (table[self.kc[p, g].long()] * self.ks[p, g].double()[:, None, None]).flatten(0, 1)[:n]
                v = (table[self.vc[p, g].long()] * self.vs[p, g].double()[:, None, None]).transpose(1, 2).flatten(0, 1)[:n]
                for h in range(g * self.Hq // self.Hk, (g + 1) * self.Hq // self.Hk):
                    q = self.q[row: row + new, h].double()
                    s = (q @ k.t().contiguous() * self.scale).masked_fill_(hidden, -float("inf"))
                    lse[row: row + new, h] = t.logsumexp(s, 1)
                    w = t.softmax(s, 1)
                    out[0][row: row + new, h], out[1][row: row + new, h] = w @ v, w @ v.abs()
                    out[2][row: row + new, h] = (w * w) @ (v * v)
                    score[row: row + new, h] = self.scale * (q.abs() @ k.abs().t().contiguous()).masked_fill_(hidden, 0).amax(1)
            row += new
        return out, lse, score

    def check(self, O, L, values_rounded=False, **kw):  # noqa: E741
        t = self.t
        (o, mag, square), lse, score = self.reference(**kw)
        delta = (self.D + 8) * 2.0 ** -23 * score + 2.0 ** -22
        sums = (max(self.lengths) + 64) * 2.0 ** -23
        off = (O.double() - o).abs()
        tol = 2.0 ** -8 * o.abs() + mag * (2.0 ** -8 * (1 + 2.0 ** -7) * (2 if values_rounded else 1)
                                           + 2 * delta[..., None] + sums)
        assert t.isfinite(O).all() and (off <= tol).all(), (off / tol).max().item()
        most = 2 * 2.0 ** -8 / 3 ** 0.5 * (o.square().sum() + square.sum() * (2 if values_rounded else 1)).sqrt()
        assert off.square().sum().sqrt() <= most
        assert ((L.double() - lse).abs() <= delta + sums + 2.0 ** -22 * lse.abs()).all()


def run(seed, lengths, new, Hq, Hk, D, parts=None, scales="powers", **kw):
    x = Batch(seed, lengths, new, Hq, Hk, D, scales)
    if parts is not None:
        low, high = parts
        assert low <= x.parts() <= high, x.parts()
    O, L, ws = x.buffers()  # noqa: E741
    x.call(O, L, ws, **kw)
    many = sum(new) * (Hq // Hk) > 16 * len(new)
    x.check(O, L, values_rounded=scales != "powers" and many, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,new,Hq,Hk,parts", [
    ([1000], [1], 4, 2, (1, 1)), ([1100], [1], 4, 2, (2, 8)), ([20001, 70], [1, 1], 4, 2, (9, 64)),
    ([3000] * 40, [1] * 40, 8, 8, (1, 1)), ([18000] + [100] * 35, [1] * 36, 8, 8, (2, 8)), ([70000], [2], 8, 1, (9, 64)),
    ([40000], [1], 17, 1, (2, 64)),
    ([900], [100], 1, 1, (2, 64)), ([130], [100], 1, 1, (1, 1)), ([8000], [90], 1, 1, (9, 64)), ([2500, 100], [120, 100], 2, 1, (2, 64)),
    ([2000], [2000], 2, 2, (2, 64)), ([700] * 30, [300] * 30, 8, 8, (1, 1)), ([33000], [260], 1, 1, (9, 64)),
    ([40000] * 3, [700] * 3, 32, 32, (1, 1))])
def test_every_cut(lengths, new, Hq, Hk, parts, D):
    if len(lengths) == 3:  # runs of more pages than are looked up at a time, on as many blocks as there are units
        lengths, new, Hq, Hk = [34000], [130], 260, 260
        parts = (1, 1)
    run(sum(lengths) + D, lengths, new, Hq, Hk, D, parts)


@pytest.mark.parametrize("lengths,new,Hq,Hk,kw", [
    ([6000], [300], 2, 2, {"causal": False}), ([6000], [300], 2, 2, {"window": 1000}), ([6000, 500], [700, 500], 4, 2, {"window": 257}),
    ([6000], [1], 4, 2, {"window": 4097}), ([5000], [3], 4, 1, {"causal": False}), ([3000], [2900], 1, 1, {"window": 64})])
def test_masks_over_many_pages(lengths, new, Hq, Hk, kw):
    for D in (64, 128):
        run(7 + D, lengths, new, Hq, Hk, D, **kw)


@pytest.mark.parametrize("new", [5, 60])
def test_a_window_past_everything(new):
    """The widest window, and more new tokens than the sequence has."""
    t = H.torch()
    x = Batch(17, [40], [40], 2, 1, 64)
    O, L = (t.zeros((new, 2, 64), dtype=t.bfloat16, device="cuda"), t.zeros((new, 2), device="cuda"))  # noqa: E741
    args = (t.cat([x.q, x.q])[:new], x.kc, x.ks, x.vc, x.vs, t.tensor([0, new], dtype=t.int32, device="cuda"))
    out = []
    for window in (0, 2147483647):
        for length in (40, 3):
            b.svdq_kv8_attention(*args, t.tensor([length], dtype=t.int32, device="cuda"), x.table, 0.125, O, L, window=window)
            out.append((O.clone(), L.clone()))
    for a, c in zip(out[:2], out[2:]):
        assert t.equal(a[0], c[0]) and t.equal(a[1], c[1])
    assert (out[1][0][: new - 3] == 0).all() and t.isneginf(out[1][1][: new - 3]).all() and (out[1][0][-3:] != 0).any()


@pytest.mark.parametrize("lengths,new", [([3000], [1]), ([3000], [300]), ([200], [150])])
def test_scales_that_are_no_powers_of_two(lengths, new):
    for D in (64, 128):
        run(9 + D, lengths, new, 2, 1, D, scales="any")


@pytest.mark.parametrize("new", [1, 300])
@pytest.mark.parametrize("what", ["ks", "vs"])
def test_scales_of_0(new, what):
    """Pages of zeros, as another program may write them, the last among them."""
    x = Batch(11, [2000], [new], 2, 1, 64)
    for i in (3, 4, 17, 30, 31):
        getattr(x, what)[x.pages[0][i]] = 0.0
    O, L, ws = x.buffers()  # noqa: E741
    x.call(O, L, ws)
    x.check(O, L)


@pytest.mark.parametrize("new", [1, 300])
def test_value_scales_far_apart(new):
    x = Batch(12, [2000], [new], 2, 1, 64)
    for i, e in ((3, -60), (4, 60), (17, -100), (20, 30)):
        x.vs[x.pages[0][i]] = 2.0 ** e
    O, L, ws = x.buffers()  # noqa: E741
    x.call(O, L, ws)
    x.check(O, L)


@pytest.mark.parametrize("new", [1, 300])
def test_pages_that_are_not_there_among_others(new):
    x = Batch(13, [3000], [new], 2, 1, 64)
    t = x.t
    gone = [5, 6, 20, 31]
    for i in gone:
        x.table[0, i] = -1 if i % 2 else x.kc.shape[0]
        x.kc[x.pages[0][i]] = 0x7F
        x.vc[x.pages[0][i]] = 0x7F
    O, L, ws = x.buffers()  # noqa: E741
    x.call(O, L, ws, causal=False)
    # the same sequence without these tokens
    y = Batch(13, [3000 - 64 * len(gone)], [new], 2, 1, 64)
    y.kc, y.ks, y.vc, y.vs, y.q = x.kc, x.ks, x.vc, x.vs, x.q
    y.pages = [[p for i, p in enumerate(x.pages[0]) if i not in gone]]
    y.check(O, L, causal=False)
    assert t.isfinite(L).all()


def test_rising_scores():
    """Scores that rise from page to page, by little and by much, and fall again."""
    for new in (1, 300):
        x = Batch(14, [4000], [new], 2, 1, 64)
        for i, p in enumerate(x.pages[0]):
            x.ks[p] = 2.0 ** (-12 + (i * 7 % 13) if i > 5 else -14 + 2 * i)
        O, L, ws = x.buffers()  # noqa: E741
        x.call(O, L, ws)
        x.check(O, L)


def test_the_same_bits_again():
    for new in (1, 40, 400):
        x = Batch(15, [3000], [new], 4, 2, 128)
        a, c = x.buffers(), x.buffers()
        x.call(*a)
        x.call(*c)
        assert x.t.equal(a[0].view(x.t.int16), c[0].view(x.t.int16)) and x.t.equal(a[1], c[1])


@pytest.mark.parametrize("new", [1, 200])
def test_a_captured_graph_follows_the_batch(new):
    """Append and attention captured once, replayed while the sequences grow; eager
    calls and a second graph on the same buffers in between."""
    t = H.torch()
    lengths = [700, 130]
    x = Batch(16, lengths, [new, new], 4, 2, 64, width=40)
    grown = [3, 70, 500]
    free = [p for p in range(x.kc.shape[0]) if all(p not in u for u in x.pages)]
    more = t.zeros((40,) + tuple(x.kc.shape[1:]), dtype=t.uint8, device="cuda")
    first = x.kc.shape[0]
    x.kc = t.cat([x.kc, more])
    x.vc = t.cat([x.vc, more.view(40, 2, 64, 64)])
    x.ks, x.vs = (t.cat([s, t.ones((40, 2), device="cuda")]) for s in (x.ks, x.vs))
    free = list(range(first, first + 40)) + free
    k, v = (t.randn((2 * new, 2, 64), generator=x.gen, device="cuda").bfloat16() for _ in range(2))
    O, L, ws = x.buffers()  # noqa: E741

    def both():
        b.svdq_kv8_append(k, v, x.starts, x.dev_lengths, x.table, x.kc, x.ks, x.vc, x.vs)
        x.call(O, L, ws)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        both()
    t.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            both()
        graphs.append(g)
    for i, more in enumerate(grown):
        for s in range(2):
            x.lengths[s] += more // (s + 1)
            while len(x.pages[s]) * PAGE < x.lengths[s]:
                x.pages[s].append(free.pop())
            x.table[s, : len(x.pages[s])] = t.tensor(x.pages[s], dtype=t.int32, device="cuda")
        x.dev_lengths.copy_(t.tensor(x.lengths, dtype=t.int32))
        k.copy_(t.randn(k.shape, generator=x.gen, device="cuda"))
        v.copy_(t.randn(k.shape, generator=x.gen, device="cuda"))
        x.q.copy_(t.randn(x.q.shape, generator=x.gen, device="cuda"))
        start = [a.clone() for a in (x.kc, x.ks, x.vc, x.vs)]
        graphs[i % 2].replay()
        t.cuda.synchronize()
        got = [O.clone(), L.clone()] + [a.clone() for a in (x.kc, x.ks, x.vc, x.vs)]
        for a, c in zip((x.kc, x.ks, x.vc, x.vs), start):
            a.copy_(c)
        O.zero_()
        both()
        t.cuda.synchronize()
        for a, c in zip(got, [O, L, x.kc, x.ks, x.vc, x.vs]):
            assert t.equal(a.view(t.uint8), c.view(t.uint8))


def test_other_streams_and_calls_at_the_same_time():
    t = H.torch()
    x = [Batch(20 + i, [5000, 300], n, 8, 2, 128) for i, n in enumerate(([1, 1], [200, 100], [2, 1]))]
    out = [y.buffers() for y in x]
    streams = [t.cuda.Stream() for _ in x]
    t.cuda.synchronize()
    for _ in range(3):
        for y, o, s in zip(x, out, streams):
            y.call(*o, stream=s)
    t.cuda.synchronize()
    for y, o in zip(x, out):
        y.check(o[0], o[1])


@pytest.mark.parametrize("new", [1, 100])
def test_a_workspace_too_small_is_refused(new):
    x = Batch(23, [5000], [new], 2, 1, 64)
    O, L, ws = x.buffers()  # noqa: E741
    O.fill_(7.0)
    for short in (None, ws[:-16]):
        with pytest.raises(b.SvdqError) as e:
            x.call(O, L, short)
        assert e.value.status == b.SVDQ_ERR_INVALID_ARGUMENT
    x.t.cuda.synchronize()
    assert (O == 7.0).all()
