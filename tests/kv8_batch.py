"""A batch on the 8-bit cache, as tests/test_gpu_kv8_paths.py makes it, whose reference
(float64 products on the GPU) also knows pages that are not there, tokens and pages that
are NaN, and queries that see nothing. A scale that is not finite stands for NaN."""


from oracle.fp8 import _BYTES
from tests import kv8_dispatch as d
from tests.test_gpu_kv8_paths import PAGE, Batch


class Batch64(Batch):
    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.gone = [set() for _ in self.new]  # pages that the table does not have

    def plan(self, window=0):
        return d.attention(self.T, len(self.new), self.table.shape[1], self.Hq, self.Hk, window)

    def remove(self, sequence, page, number=-1):
        """The page is not in the table; what it held is NaN, its scales as well."""
        self.gone[sequence].add(page)
        self.table[sequence, page] = number
        p = self.pages[sequence][page]
        self.kc[p], self.vc[p], self.ks[p], self.vs[p] = 0x7F, 0xFF, float("nan"), float("nan")

    def attend(self, **kw):
        O, L, ws = self.buffers()  # noqa: E741
        self.call(O, L, ws, **kw)
        return O, L

    def reference(self, causal=True, window=0):
        t = self.t
        bytes64 = t.tensor(_BYTES, device="cuda")
        whole = lambda x: t.where(t.isfinite(x), x.double(), float("nan"))  # noqa: E731
        o, mag, square = (t.zeros((self.T, self.Hq, self.D), dtype=t.float64, device="cuda") for _ in range(3))
        lse = t.full((self.T, self.Hq), -float("inf"), dtype=t.float64, device="cuda")
        score = t.zeros((self.T, self.Hq), dtype=t.float64, device="cuda")
        group, row = self.Hq // self.Hk, 0
        for n, new, pages, gone in zip(self.lengths, self.new, self.pages, self.gone):
            rows, row = slice(row, row + new), row + new
            if n == 0 or new == 0:
                continue
            p = t.tensor(pages, dtype=t.long, device="cuda")
            pos = t.arange(n - new, n, device="cuda")[:, None]
            at = t.arange(n, device="cuda")
            there = t.tensor([i not in gone for i in range(len(pages))], device="cuda").repeat_interleave(PAGE)[:n]
            see = there & ((at <= pos) if causal else t.ones((new, n), dtype=t.bool, device="cuda"))
            if window:
                see = see & (at > pos - window)
            for g in range(self.Hk):
                k = (bytes64[self.kc[p, g].long()] * whole(self.ks[p, g])[:, None, None]).flatten(0, 1)[:n]
                v = (bytes64[self.vc[p, g].long()] * whole(self.vs[p, g])[:, None, None]).transpose(1, 2).flatten(0, 1)[:n]
                lost = t.isnan(v)
                v = v.masked_fill(lost, 0.0)
                lost = see.double() @ lost.double() > 0
                kt = k.t().contiguous()
                for h in range(g * group, (g + 1) * group):
                    q = self.q[rows, h].double()
                    s = (q @ kt * self.scale).masked_fill_(~see, -float("inf"))
                    top = s.amax(1, keepdim=True)
                    w = (s - t.where(t.isneginf(top), 0.0, top)).exp_()
                    total = w.sum(1, keepdim=True)
                    lse[rows, h] = (top + total.log())[:, 0]
                    w /= t.where(total == 0, 1.0, total)
                    o[rows, h] = (w @ v).masked_fill_(lost, float("nan"))
                    mag[rows, h] = w @ v.abs()
                    square[rows, h] = (w * w) @ (v * v)
                    score[rows, h] = self.scale * (q.abs() @ kt.abs()).masked_fill_(~see, 0.0).amax(1)
        return (o, mag, square), lse, score

    def check(self, O, L, values_rounded=False, **kw):  # noqa: E741
        t = self.t
        (o, mag, square), lse, score = self.reference(**kw)
        assert t.equal(t.isnan(O), t.isnan(o)) and not t.isinf(O).any()
        assert t.equal(t.isnan(L), t.isnan(lse)) and t.equal(t.isneginf(L), t.isneginf(lse))
        assert (O[t.isneginf(lse)] == 0).all()
        delta = (self.D + 8) * 2.0 ** -23 * score + 2.0 ** -22
        sums = (max(self.lengths) + 64) * 2.0 ** -23
        off = (O.double() - o).abs()
        tol = 2.0 ** -8 * o.abs() + mag * (2.0 ** -8 * (1 + 2.0 ** -7) * (2 if values_rounded else 1)
                                           + 2 * delta[..., None] + sums)
        fine = ~t.isnan(o)
        assert (off <= tol)[fine].all(), (off / tol)[fine].max().item()
        most = 2 * 2.0 ** -8 / 3 ** 0.5 * (o[fine].square().sum() + square[fine].sum() * (2 if values_rounded else 1)).sqrt()
        assert off[fine].square().sum().sqrt() <= most
        fine = t.isfinite(lse)
        assert ((L.double() - lse).abs() <= delta + sums + 2.0 ** -22 * lse.abs())[fine].all()


# Batches for each kernel, in one part and in several: (rows of a block, several parts,
# lengths, new, Hq, Hk). The first sequence's last page is seen by its last two tokens alone.
KERNELS = [
    (16, False, [258, 70], [4, 1], 4, 2), (16, True, [3010, 70], [4, 1], 4, 2),
    (32, False, [258, 70], [12, 8], 4, 2), (32, True, [3010], [12], 4, 2),
    (64, False, [258], [30], 4, 2), (64, True, [3010], [30], 4, 2),
    (128, False, [258, 90], [60, 50], 4, 2), (128, True, [6018], [60], 4, 2),
    (256, False, [706] + [700] * 29, [300] * 30, 8, 8), (256, True, [4994], [300], 16, 2),
]


def kernel_id(case):
    return f"{case[0]}{' in parts' if case[1] else ''}"


def batch(seed, case, D, window=0, **kw):
    """The case's batch, in the kernel and cut that it names."""
    rows, parts, *sizes = case
    x = Batch64(seed, *sizes, D, **kw)
    p = x.plan(window)
    assert p.rows == rows and (p.splits > 1) == parts, p
    return x
