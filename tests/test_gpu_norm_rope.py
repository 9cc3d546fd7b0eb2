"""The norm before the block-scaled FP8 linears and the rotary positions against
oracle/decoder.py, through the binding (needs an MI355X).

norm: y is fp32 with one rounding each of the sum, 1 / sqrt (of an fp64 mean), and
two products: 2^-24 each, 5 2^-24 of |y| with the fp32 rounding of eps. A scale has
one more for its division. A code stands for a number within half an E4M3 step
(2^-4 of it, 2^-10 below 2^-6) of y 448 / A, whose factors are off by 5, 6 and 1
times 2^-24. rope: sine and cosine are within 2^-22 (the angle's reduced part is
fp32, 2^-25 of half a turn; 2 units of the function), products and sum 2^-24 each:
2^-21 (|a| + |b|). Outputs in bf16 add half a step, 2^-8.
"""

import numpy as np
import pytest

from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import workloads as wl
from oracle import decoder as od
from oracle import svdquant as sq
from oracle.fp8 import e4m3_decode
from tests import gpu_harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert b.svdq_check_device(torch.cuda.current_device()) == b.SVDQ_OK


def bf16(seed, shape, std=1.0):
    """bf16 values (float32) and their tensor."""
    a = wl.random_bf16(seed, shape, std)
    return a["values"], H.dev(a["bits"]).view(H.torch().bfloat16)


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def guarded(shape, dtype):
    """A tensor whose rows behind the first shape[0] must stay as they are."""
    t = H.torch()
    n = int(np.prod(shape[1:]))
    whole = t.full((shape[0] * n * dtype.itemsize + 64,), 0xA5, dtype=t.uint8, device="cuda")
    return whole[:-64].view(dtype).view(shape), whole


def untouched(whole):
    assert np.all(H.host(whole[-64:]) == 0xA5)


def norm_call(X, R, w, eps, total="new", y=True, codes=True):
    t = H.torch()
    M, K = X.shape
    out = {"Y": guarded((M, K), t.bfloat16) if y else None, "sum": None}
    out["qx"] = guarded((M, K), t.uint8) if codes else None
    out["sx"] = guarded((b.fp8_blocks(K), M), t.float32) if codes else None
    dest = None
    if total == "new":
        out["sum"] = guarded((M, K), t.bfloat16)
        dest = out["sum"][0]
    elif total == "residual":
        dest = R
    elif total == "X":
        dest = X
    first = lambda n: out[n][0] if out[n] else None  # noqa: E731
    b.svdq_fp8_norm_quantize(X, R, w, eps, dest, first("Y"), first("qx"), first("sx"))
    t.cuda.synchronize()
    for v in out.values():
        if v is not None:
            untouched(v[1])
    got = {n: v[0] for n, v in out.items() if v is not None}
    if dest is not None:
        got["sum"] = dest
    return got


def norm_check(got, ref):
    y, e = ref["y"], 2.0 ** -24
    if "sum" in got:
        assert np.array_equal(values(got["sum"]), ref["sum"])
    if "Y" in got:
        off = np.abs(values(got["Y"]) - y)
        assert np.all(off <= (2.0 ** -8 + 6 * e) * np.abs(y) + 2.0 ** -134), off.max()
    if "qx" in got:
        A = od.block_tops(y)
        s = H.host(got["sx"]).astype(np.float64)
        assert np.all(np.abs(s - A / 448.0) <= 7 * e * A / 448.0)
        want = y * (448.0 / A).T[:, np.arange(y.shape[1]) // 128]
        code = e4m3_decode(H.host(got["qx"]))
        near = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -20 * np.abs(want)
        assert np.all(np.abs(code - want) <= near), np.max(np.abs(code - want) / near)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (2, 1936), (5, 2048), (17, 5120), (333, 400), (2, 8192),
                                 (3, 8208), (2, 20000), (1030, 1040), (4097, 96), (1, 65552),
                                 (1001, 256), (257, 1024), (256, 1024), (300, 2064), (257, 6144), (300, 6160), (259, 512)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(M, K, residual):
    xv, x = bf16(M + K, (M, K))
    rv, r = bf16(M + K + 1, (M, K), 3.0)
    rv, r = (rv, r) if residual else (None, None)
    wv, w = bf16(K, (K,), 0.5)
    got = norm_call(x, r, w, 1e-5)
    norm_check(got, od.norm(xv, rv, wv, np.float32(1e-5)))


@pytest.mark.parametrize("M,K", [(2, 512), (2, 12288), (1100, 768)])
@pytest.mark.parametrize("where", ["residual", "X"])
def test_the_sum_may_replace_an_input(M, K, where):
    xv, x = bf16(1, (M, K))
    rv, r = bf16(2, (M, K))
    wv, w = bf16(3, (K,))
    got = norm_call(x, r, w, 1e-6, total=where)
    norm_check(got, od.norm(xv, rv, wv, np.float32(1e-6)))


def test_norm_outputs_one_at_a_time():
    xv, x = bf16(1, (9, 272))
    wv, w = bf16(2, (272,))
    ref = od.norm(xv, None, wv, np.float32(0.01))
    both = norm_call(x, None, w, 0.01, total=None)
    for kw in ({"y": False}, {"codes": False}, {"y": False, "total": None}, {"codes": False, "total": None}):
        got = norm_call(x, None, w, 0.01, **kw)
        norm_check(got, ref)
        for n in set(got) & set(both):
            assert np.array_equal(H.host(got[n].view(H.torch().uint8)), H.host(both[n].view(H.torch().uint8)))


def test_norm_of_very_large_and_small_rows_and_zeros():
    xv, _ = bf16(4, (5, 256))
    xv = xv.copy()
    xv[0] *= np.float32(2.0 ** 120)
    xv[1] *= np.float32(2.0 ** -120)
    xv[2] = 0.0
    xv[3, 1:] = 0.0
    bits = wl.bf16_bits_from_f32(xv)
    xv = wl.f32_from_bf16_bits(bits)
    wv, w = bf16(5, (256,))
    x = H.dev(bits).view(H.torch().bfloat16)
    got = norm_call(x, None, w, 1e-30)
    ref = od.norm(xv, None, wv, np.float64(np.float32(1e-30)))
    norm_check(got, ref)
    assert np.all(e4m3_decode(H.host(got["qx"])[2]) == 0.0)


def test_norm_of_rows_that_are_not_finite_leaves_the_others():
    xv, x = bf16(6, (4, 400))
    wv, w = bf16(7, (400,))
    clean = norm_call(x, None, w, 1e-6)
    x[1, 7], x[2, 300] = float("nan"), float("inf")
    got = norm_call(x, None, w, 1e-6)
    for row in (0, 3):
        for n in ("Y", "qx", "sum"):
            assert np.array_equal(H.host(got[n][row].view(H.torch().uint8)), H.host(clean[n][row].view(H.torch().uint8)))
    s = H.host(got["sx"])
    assert np.all(np.isnan(s[:, 1])) and np.all((H.host(got["qx"])[1] & 0x7F) == 0x7F)
    assert np.all(np.isnan(values(got["Y"])[1])) and np.isnan(values(got["Y"])[2, 300]) and np.isnan(s[2, 2])
    assert np.array_equal(s[:, [0, 3]], H.host(clean["sx"])[:, [0, 3]])


# ------------------------------------------------------------------- rope --

def rope_inputs(T, axes, pairs, far, seed):
    rng = np.random.default_rng(seed)
    pos = rng.integers(0, far, (T, axes)).astype(np.int32)
    pos[-1] = far - 1
    freqs = 10000.0 ** (-rng.random(pairs))
    freqs[0] = 1.0
    return pos, freqs


def rope_check(y, x, pos, freqs, sections, interleaved):
    ref = od.rope(x, pos, freqs, sections, interleaved)
    pairs = sum(sections)
    both = np.zeros_like(ref)
    a, c = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    both[..., a] = both[..., c] = np.abs(x[..., a]) + np.abs(x[..., c])
    off = np.abs(y - ref)
    assert np.all(off <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * both * (1 + 2.0 ** -8)), off.max()
    assert np.array_equal(y[..., 2 * pairs:], x[..., 2 * pairs:])


@pytest.mark.parametrize("T,H_,D,sections,far", [(1, 1, 16, (8,), 10), (3, 5, 64, (32,), 1 << 20), (7, 3, 128, (22, 21, 21), 50),
                                                 (2, 40, 128, (16, 24, 24), 1000), (5, 9, 80, (0, 7, 9), 100),
                                                 (33, 2, 96, (4, 8, 12, 16), 77), (2, 3, 512, (100, 156), 3000),
                                                 (4, 80, 128, (64,), 2147483647), (300, 6, 64, (3, 0, 5), 40), (4099, 2, 64, (10, 22), 90),
                                                 (8191, 1, 80, (16,), 1000), (6146, 4, 128, (60, 4), 70)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(T, H_, D, sections, far, interleaved):
    t = H.torch()
    xv, x = bf16(T + D, (T, H_, D))
    pos, freqs = rope_inputs(T, len(sections), sum(sections), far, T)
    y, whole = guarded((T, H_, D), t.bfloat16)
    b.svdq_rope(x, H.dev(pos), H.dev(freqs), sections, y, interleaved=interleaved)
    t.cuda.synchronize()
    untouched(whole)
    rope_check(values(y), xv, pos, freqs, sections, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_a_projections_rows_in_place(interleaved):
    t = H.torch()
    T, Hq, Hk, D = 13, 6, 2, 64
    xv, x = bf16(8, (T, Hq + 2 * Hk, D))
    pos, freqs = rope_inputs(T, 2, 24, 5000, 9)
    heads = x[:, : Hq + Hk]
    apart = t.empty((T, Hq + Hk, D), dtype=t.bfloat16, device="cuda")
    b.svdq_rope(heads, H.dev(pos), H.dev(freqs), (20, 4), apart, interleaved=interleaved)
    b.svdq_rope(heads, H.dev(pos), H.dev(freqs), (20, 4), heads, interleaved=interleaved)
    t.cuda.synchronize()
    rope_check(values(heads), xv[:, : Hq + Hk], pos, freqs, (20, 4), interleaved)
    assert t.equal(apart, heads.contiguous()) and np.array_equal(values(x)[:, Hq + Hk:], xv[:, Hq + Hk:])


def test_rope_turned_back():
    t = H.torch()
    xv, x = bf16(11, (6, 4, 128))
    pos, freqs = rope_inputs(6, 1, 64, 1 << 20, 12)
    y, back = t.empty_like(x), t.empty_like(x)
    b.svdq_rope(x, H.dev(pos), H.dev(freqs), (64,), y)
    b.svdq_rope(y, H.dev(pos), H.dev(-freqs), (64,), back)
    # y's rounding is turned as y is, then the result is rounded
    size = np.abs(xv)[..., :64] + np.abs(xv)[..., 64:]
    size = np.concatenate([size, size], -1)
    assert np.all(np.abs(values(back) - xv) <= 2.0 ** -8 * np.abs(xv) + 2 * 2.0 ** -8 * size)


def test_rope_not_finite_stays_in_its_pair():
    t = H.torch()
    xv, x = bf16(13, (2, 2, 32))
    pos, freqs = rope_inputs(2, 1, 16, 100, 14)
    clean, y = t.empty_like(x), t.empty_like(x)
    b.svdq_rope(x, H.dev(pos), H.dev(freqs), (16,), clean)
    x[1, 0, 3] = float("nan")
    b.svdq_rope(x, H.dev(pos), H.dev(freqs), (16,), y)
    bad = np.isnan(values(y))
    assert bad.sum() == 2 and bad[1, 0, 3] and bad[1, 0, 19]
    assert np.array_equal(values(y)[~bad], values(clean)[~bad])
