"""The 8-bit key and value cache against oracle/decoder.py, through the binding
(needs an MI355X).

append is the oracle's bit for bit, every byte of the cache. attention: an output is
within half a bf16 step of its value, 2^-8, plus, relative to mag = sum p |v|:
2^-8 for the weights' rounding to bf16; twice what a score may be off by, delta =
(D + 8) 2^-23 sum |scale q k| (fp32 sums of D products, each addition off by at most
2^-23; the scale's and the exponent's own roundings) plus 2^-22; and 2^-23 for each of
the length + 64 additions of a sum. Roundings of different weights are independent:
over many outputs the error's 2-norm is near 2^-8 / sqrt(3) of the 2-norm of o and of
the terms p v together; twice that is asked.
Keys, values, pages and table entries that a call must not look at hold NaN codes.
"""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import workloads as wl
from oracle import decoder as od
from tests import gpu_harness as H
from tests.test_gpu_norm_rope import _gpu, guarded, untouched, values  # noqa: F401

pytestmark = pytest.mark.gpu
PAGE = od.PAGE


def bf16_values(rng, shape, std=1.0):
    return wl.f32_from_bf16_bits(wl.bf16_bits_from_f32((std * rng.standard_normal(shape)).astype(np.float32)))


def bf16_dev(v):
    return H.dev(wl.bf16_bits_from_f32(np.asarray(v, np.float32))).view(H.torch().bfloat16)


def plan(rng, lengths, new, spare=2, width=None):
    """starts, table and page count of sequences in pages of random order; -1 behind."""
    used = [-(-n // PAGE) for n in lengths]
    total = sum(used) + spare
    order = rng.permutation(total)
    table = np.full((len(lengths), width or max(1, max(used))), -1, np.int32)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at: at + n]
        at += n
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32), table, total


def random_cache(rng, P, Hk, D, low=-8, high=-5):
    """Codes of normal numbers, and scales 2^low .. 2^high."""
    from oracle.fp8 import e4m3_encode

    codes = lambda *shape: e4m3_encode(np.clip(64 * rng.standard_normal(shape), -448, 448))  # noqa: E731
    scale = lambda: np.exp2(rng.integers(low, high + 1, (P, Hk))).astype(np.float32)  # noqa: E731
    return od.Cache(codes(P, Hk, PAGE, D), scale(), codes(P, Hk, D, PAGE), scale())


def poison(cache, lengths, table):
    """NaN codes wherever no sequence has a token."""
    seen = np.zeros((cache.kc.shape[0], PAGE), bool)
    for n, pages in zip(lengths, table):
        for t in range(n):
            if 0 <= pages[t // PAGE] < len(seen):
                seen[pages[t // PAGE], t % PAGE] = True
    for p in range(len(seen)):
        cache.kc[p][:, ~seen[p]] = 0x7F
        cache.vc[p][:, :, ~seen[p]] = 0xFF


def upload(cache):
    return [H.dev(a) for a in (cache.kc, cache.ks, cache.vc, cache.vs)]


def attend(Q, cache, starts, lengths, table, scale, causal=True, window=0, lse=True, T=None):
    t = H.torch()
    q = Q if isinstance(Q, t.Tensor) else bf16_dev(Q)
    T, Hq, D = q.shape
    O, o_all = guarded((T, Hq, D), t.bfloat16)  # noqa: E741
    L, l_all = guarded((T, Hq), t.float32)
    n = b.svdq_kv8_attention_workspace_bytes(T, len(lengths), table.shape[1], Hq, cache.kc.shape[1], D)
    ws = t.full((n + 64,), 0xFF, dtype=t.uint8, device="cuda")  # NaN, if read before it is written
    b.svdq_kv8_attention(q, *upload(cache), H.dev(np.asarray(starts, np.int32)), H.dev(np.asarray(lengths, np.int32)),
                         H.dev(table), scale, O, L if lse else None, ws, causal=causal, window=window)
    t.cuda.synchronize()
    untouched(o_all)
    untouched(l_all)
    assert np.all(H.host(ws[n:]) == 0xFF)
    return values(O), H.host(L).astype(np.float64)


def check(got, ref, lengths, D, rows=None):
    o, lse = got
    rows = slice(None) if rows is None else rows
    o, lse = o[rows], lse[rows]
    r = {k: v[rows] for k, v in ref.items()}
    length = max(lengths)
    delta = ((D + 8) * 2.0 ** -23 * r["score"] + 2.0 ** -22)[..., None]
    tol = 2.0 ** -8 * np.abs(r["o"]) + r["mag"] * (2.0 ** -8 * (1 + 2.0 ** -7) + 2 * delta + (length + 64) * 2.0 ** -23)
    off = np.abs(o - r["o"])
    assert np.array_equal(np.isnan(o), np.isnan(r["o"]))
    ok = ~np.isnan(off)
    assert np.all(off[ok] <= tol[ok]), np.nanmax(off / np.maximum(tol, 1e-300))
    if ok.sum() > 2000 and np.linalg.norm(r["o"][ok]) > 0:
        most = 2 * 2.0 ** -8 / np.sqrt(3.0) * np.sqrt(np.sum(r["o"][ok] ** 2) + np.sum(r["square"][ok]))
        assert np.linalg.norm(off[ok]) <= most, np.linalg.norm(off[ok]) / most
    empty = np.isneginf(r["lse"])
    assert np.array_equal(np.isneginf(lse), empty) and np.all(o[empty] == 0.0)
    fine = np.isfinite(r["lse"])
    far = np.abs(lse[fine] - r["lse"][fine])
    assert np.all(far <= (delta[..., 0] + (length + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(r["lse"]))[fine])
    assert np.array_equal(np.isnan(lse), np.isnan(r["lse"]))


# ----------------------------------------------------------------- append --

def append_case(seed, lengths, new, Hk, D, std=1.0, width=None, break_page=False, edit=None):
    rng = np.random.default_rng(seed)
    t = H.torch()
    starts, table, P = plan(rng, lengths, new, width=width)
    if break_page:
        table[0, 0] = P + 3
    cache = random_cache(rng, P, Hk, D)
    T = int(starts[-1])
    rows = bf16_values(rng, (T, 3 * Hk, D), std)
    rows[:, :, ::7] *= 16.0
    if edit:
        rows = rows.copy()
        edit(rows)
    dev = bf16_dev(rows)
    ref = od.Cache(cache.kc, cache.ks, cache.vc, cache.vs)
    for _ in range(2):  # the same call again gives the same cache
        tensors = upload(cache)
        args = (dev[:, Hk: 2 * Hk], dev[:, 2 * Hk:], H.dev(starts), H.dev(np.asarray(lengths, np.int32)), H.dev(table))
        b.svdq_kv8_append(*args, *tensors)
        t.cuda.synchronize()
        again = [x.clone() for x in tensors]
        b.svdq_kv8_append(*args, *tensors)
        t.cuda.synchronize()
        for x, y in zip(tensors, again):
            assert t.equal(x, y)
    ref.append(rows[:, Hk: 2 * Hk].astype(np.float64), rows[:, 2 * Hk:].astype(np.float64), starts, lengths, table)
    for x, want in zip(tensors, (ref.kc, ref.ks, ref.vc, ref.vs)):
        got = H.host(x)
        if got.dtype == np.uint8:  # the sign of NaN is open
            got, want = np.where((got & 0x7F) == 0x7F, 0x7F, got), np.where((want & 0x7F) == 0x7F, 0x7F, want)
        assert np.array_equal(got, want), np.argwhere(got != want)[:4]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,new,Hk", [([1], [1], 1), ([64], [64], 2), ([65], [1], 2), ([64], [1], 1), ([200], [130], 3),
                                            ([70, 1, 129, 64], [3, 1, 129, 1], 2), ([300], [5], 2), ([63, 127], [2, 64], 1),
                                            ([130, 0, 5], [65, 0, 0], 2)])
def test_append_is_exact(lengths, new, Hk, D):
    append_case(sum(lengths) + D, lengths, new, Hk, D)


@pytest.mark.parametrize("std", [2.0 ** -60, 2.0 ** -110, 0.01, 300.0, 2.0 ** 100])
def test_append_of_small_and_large_values(std):
    append_case(3, [100, 40], [90, 3], 2, 64, std)


def test_append_more_sequences_than_a_wave_looks_at():
    rng = np.random.default_rng(4)
    new = rng.integers(0, 3, 150).tolist()
    append_case(4, [int(n + rng.integers(0, 140)) for n in new], new, 1, 64)


def test_append_leaves_out_tokens_before_the_first_and_pages_outside():
    append_case(5, [10, 66], [25, 70], 2, 64, break_page=False)
    append_case(6, [130, 66], [130, 3], 2, 64, break_page=True)


def test_append_not_finite():
    def edit(rows):
        rows[0, 2, 3], rows[3, 3, 9], rows[4, 5, 1], rows[5] = np.nan, np.inf, -np.inf, np.inf

    append_case(7, [70], [20], 2, 64, edit=edit)


def test_append_of_a_maximum_on_the_border_of_a_scale():
    for top in (448.0, 450.0, 1.75, 1.7578125, 2.0 ** -100, 0.0):  # 450: the next bf16 number
        def edit(rows):
            rows[:] = 0.0
            rows[1, :, 5] = top

        append_case(8, [4], [4], 1, 64, edit=edit)


# -------------------------------------------------------------- attention --

def attention_case(seed, lengths, new, Hq, Hk, D, causal=True, window=0, std=1.0, width=None, lse=True):
    rng = np.random.default_rng(seed)
    starts, table, P = plan(rng, lengths, new, width=width)
    cache = random_cache(rng, P, Hk, D)
    # tokens at the ends of pages and sequences weigh most
    for n, pages in zip(lengths, table):
        for t in {0, n - 1, n // 2, n - 2} | set(range(63, n, 64)):
            if 0 <= t < n:
                cache.vc[pages[t // PAGE], :, :, t % PAGE] = 0x7E
    poison(cache, lengths, table)
    Q = bf16_values(rng, (int(starts[-1]), Hq, D), std)
    scale = 1.0 / np.sqrt(D)
    got = attend(Q, cache, starts, lengths, table, scale, causal, window, lse)
    ref = od.attention(Q, cache, starts, lengths, table, np.float64(np.float32(scale)), causal, window)
    if not lse:
        got = (got[0], ref["lse"])
    check(got, ref, lengths, D)


FEW = [([1], [1], 1, 1), ([64], [1], 2, 1), ([65], [1], 2, 2), ([130], [1], 8, 2), ([5, 700, 64], [1, 1, 1], 16, 2),
       ([300, 2, 66], [4, 2, 3], 8, 2), ([1000], [1], 5, 1), ([200], [2], 7, 1), ([97, 600], [1, 1], 24, 1),
       ([129, 0, 10], [1, 0, 1], 4, 4), ([333, 50], [3, 20], 2, 2)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,new,Hq,Hk", FEW)
def test_decode(lengths, new, Hq, Hk, D):
    assert sum(new) * (Hq // Hk) <= 16 * len(new) or Hq // Hk > 16
    attention_case(sum(lengths) + D, lengths, new, Hq, Hk, D)


MANY = [([40], [40], 2, 1), ([64], [64], 1, 1), ([65], [65], 1, 1), ([200], [200], 3, 1), ([300], [77], 4, 2),
        ([130, 40, 257], [130, 20, 100], 4, 2), ([500], [33], 7, 1), ([129], [129], 2, 2), ([100, 1, 300], [100, 1, 2], 2, 1),
        ([260], [17], 1, 1), ([70], [70], 40, 8)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,new,Hq,Hk", MANY)
def test_prompt(lengths, new, Hq, Hk, D):
    assert sum(new) * (Hq // Hk) > 16 * len(new)
    attention_case(sum(lengths) + D, lengths, new, Hq, Hk, D)


@pytest.mark.parametrize("lengths,new,Hq,Hk,causal,window", [
    ([300, 70], [1, 1], 4, 2, False, 0), ([300, 70], [1, 1], 4, 2, True, 100), ([300], [4], 4, 2, True, 1),
    ([300, 64], [4, 1], 4, 2, True, 64), ([300, 70], [200, 70], 4, 2, False, 0), ([400, 70], [200, 70], 4, 2, True, 100),
    ([300], [300], 2, 2, True, 1), ([400], [150], 2, 1, True, 64), ([400], [390], 3, 1, True, 63), ([100], [100], 2, 1, True, 5000),
    ([500], [200], 2, 1, True, 129)])
def test_masks(lengths, new, Hq, Hk, causal, window):
    for D in (64, 128):
        attention_case(window + D, lengths, new, Hq, Hk, D, causal, window)


@pytest.mark.parametrize("new", [[30, 3, 1], [3, 2, 1]])
@pytest.mark.parametrize("causal", [True, False])
def test_queries_that_see_nothing(new, causal):
    # more new tokens than a sequence has, and sequences of no token
    attention_case(31, [10 if new[0] > 3 else 1, 0, 0], new, 4, 2, 64, causal=causal)


def test_without_lse():
    attention_case(1, [100], [1], 4, 2, 64, lse=False)
    attention_case(1, [100], [90], 4, 2, 64, lse=False)


@pytest.mark.parametrize("new", [1, 60])
def test_sharp_and_flat_weights(new):
    for std in (0.0, 30.0):
        attention_case(2, [333], [new], 4, 2, 64, std=std)


def test_wide_tables_and_many_sequences():
    attention_case(3, [100, 40], [1, 1], 2, 1, 64, width=300)
    rng = np.random.default_rng(9)
    new = rng.integers(0, 3, 140).tolist()
    attention_case(4, [int(n + rng.integers(0, 100)) for n in new], new, 2, 1, 64)
    new = rng.integers(0, 40, 70).tolist()
    attention_case(5, [int(n + rng.integers(0, 100)) for n in new], new, 2, 1, 64)


@pytest.mark.parametrize("new", [[2, 1], [40, 33]])
def test_rows_and_pages_outside_are_left_alone(new):
    """Rows before the first and behind the last sequence keep their bytes; tokens of
    page numbers outside the cache are not seen."""
    rng = np.random.default_rng(12)
    lengths = [150, 140]
    starts, table, P = plan(rng, lengths, new)
    cache = random_cache(rng, P, 2, 64)
    table[0, 1], table[1, 0] = P, -7
    poison(cache, lengths, table)
    Q = bf16_values(rng, (sum(new) + 9, 4, 64))
    starts = starts + 4
    got = attend(Q, cache, starts, lengths, table, 0.125)
    ref = od.attention(Q, cache, starts, lengths, table, 0.125)
    check(got, ref, lengths, 64, slice(4, 4 + sum(new)))
    o, _ = got
    left = np.concatenate([o[:4], o[4 + sum(new):]])
    assert np.all(left == wl.f32_from_bf16_bits(np.uint16(0xA5A5)))  # as guarded() filled it


@pytest.mark.parametrize("starts,lengths", [([0, 50, 7], [100, 90]), ([-5, 4, 90], [100, 5000]), ([3, 3, 2147483647], [-4, 100]),
                                            ([-2147483648, 2, 40], [2147483647, -2147483648])])
def test_arrays_of_nonsense_stay_inside_the_buffers(starts, lengths):
    """Held to the buffers: nothing outside them is read or written, whatever they say."""
    t = H.torch()
    rng = np.random.default_rng(13)
    _, table, P = plan(rng, [100, 90], [1, 1])
    cache = random_cache(rng, P, 2, 64)
    table[1, 1] = 1 << 30
    for T in (2, 40):
        Q = bf16_values(rng, (T, 4, 64))
        attend(Q, cache, starts, lengths, table, 0.125)
        x = bf16_dev(bf16_values(rng, (T, 2, 64)))
        whole = [guarded(a.shape, t.uint8 if a.dtype == np.uint8 else t.float32) for a in (cache.kc, cache.ks, cache.vc, cache.vs)]
        for (view, _), a in zip(whole, (cache.kc, cache.ks, cache.vc, cache.vs)):
            view.copy_(H.dev(a))
        b.svdq_kv8_append(x, x, H.dev(np.asarray(starts, np.int32)), H.dev(np.asarray(lengths, np.int32)), H.dev(table),
                          *[v for v, _ in whole])
        t.cuda.synchronize()
        for _, w in whole:
            untouched(w)


@pytest.mark.parametrize("new", [3, 50])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_reaches_the_queries_that_see_it(new, D):
    """NaN in a value or key of a token: NaN for later queries, nothing for earlier
    ones, and with a window nothing for those far behind."""
    rng = np.random.default_rng(14)
    lengths, Hq, Hk = [200], 4, 2
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
        got = attend(Q, cache, starts, lengths, table, 0.1, window=window)
        ref = od.attention(Q, cache, starts, lengths, table, np.float64(np.float32(0.1)), window=window)
        assert np.isnan(ref["o"]).any() and (token < 150 or new == 3 or not np.isnan(ref["o"]).all(axis=(1, 2)).all())
        check(got, ref, lengths, D)


def test_queries_in_wider_rows_and_shared_pages():
    t = H.torch()
    rng = np.random.default_rng(15)
    lengths, new = [130, 130], [2, 2]
    starts, table, P = plan(rng, lengths, new)
    table[1, :2] = table[0, :2]  # a shared prefix
    cache = random_cache(rng, P, 2, 64)
    rows = bf16_values(rng, (4, 8, 64))
    wide = bf16_dev(rows)
    for few in (True, False):
        if not few:
            lengths, new = [130, 130], [40, 33]
            starts = np.array([0, 40, 73], np.int32)
            rows = bf16_values(rng, (73, 8, 64))
            wide = bf16_dev(rows)
        got = attend(wide[:, 2:6], cache, starts, lengths, table, 0.125)
        check(got, od.attention(rows[:, 2:6], cache, starts, lengths, table, 0.125), lengths, 64)
    assert t.equal(wide, bf16_dev(rows))


@pytest.mark.parametrize("lengths,new", [([500, 90], [1, 1]), ([300], [70])])
def test_joining_parts_of_a_context(lengths, new):
    """Outputs over two halves of the pages, joined with their lse, are the whole's."""
    rng = np.random.default_rng(16)
    starts, table, P = plan(rng, lengths, new)
    cache = random_cache(rng, P, 1, 64)
    Q = bf16_values(rng, (sum(new), 2, 64))
    ref = od.attention(Q, cache, starts, lengths, table, 0.125, causal=False)
    left, right = table.copy(), table.copy()
    left[:, 1:], right[:, :1] = -1, -1
    (o0, l0), (o1, l1) = (attend(Q, cache, starts, lengths, t, 0.125, causal=False) for t in (left, right))
    top = np.maximum(l0, l1)
    w0, w1 = np.exp(l0 - top)[..., None], np.exp(l1 - top)[..., None]
    check(((o0 * w0 + o1 * w1) / (w0 + w1), top + np.log((w0 + w1)[..., 0])), ref, lengths, 64)


def test_offsets_past_32_bits():
    """Pages whose bytes lie beyond 2^31 and 2^32 of the cache."""
    t = H.torch()
    rng = np.random.default_rng(17)
    Hk, D = 8, 128
    P = (1 << 32) // (Hk * PAGE * D) + 40
    kc = t.zeros((P, Hk, PAGE, D), dtype=t.uint8, device="cuda")
    vc = t.zeros((P, Hk, D, PAGE), dtype=t.uint8, device="cuda")
    ks, vs = (t.ones((P, Hk), device="cuda") for _ in range(2))
    for new in (1, 40):
        lengths = [130]
        table = np.array([[3, P // 2 + 5, P - 1]], np.int32)
        small = od.Cache(*(np.zeros(s, d) for s, d in (((3, Hk, PAGE, D), np.uint8), ((3, Hk), np.float32),
                                                       ((3, Hk, D, PAGE), np.uint8), ((3, Hk), np.float32))))
        K, V = (bf16_values(rng, (130, Hk, D)) for _ in range(2))
        Q = bf16_values(rng, (new, Hk, D))
        small.append(K.astype(np.float64), V.astype(np.float64), [0, 130], lengths, [[0, 1, 2]])
        whole = lambda v: H.dev(np.asarray(v, np.int32))  # noqa: E731
        b.svdq_kv8_append(bf16_dev(K), bf16_dev(V), whole([0, 130]), whole(lengths), H.dev(table), kc, ks, vc, vs)
        for i, p in enumerate(table[0]):
            n = min(PAGE, 130 - 64 * i)
            assert np.array_equal(H.host(kc[p, :, :n]), small.kc[i, :, :n]) and np.array_equal(H.host(ks[p]), small.ks[i])
            assert np.array_equal(H.host(vc[p, :, :, :n]), small.vc[i, :, :, :n])
        O, L = t.empty((new, Hk, D), dtype=t.bfloat16, device="cuda"), t.empty((new, Hk), device="cuda")  # noqa: E741
        ws = t.empty(b.svdq_kv8_attention_workspace_bytes(new, 1, 3, Hk, Hk, D), dtype=t.uint8, device="cuda")
        b.svdq_kv8_attention(bf16_dev(Q), kc, ks, vc, vs, whole([0, new]), whole(lengths), H.dev(table), 0.09, O, L, ws)
        ref = od.attention(Q, small, [0, new], lengths, [[0, 1, 2]], np.float64(np.float32(0.09)))
        check((values(O), H.host(L).astype(np.float64)), ref, lengths, D)
