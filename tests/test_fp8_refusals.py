"""What the block-scaled FP8 entry points refuse, before anything is launched:
by the library (shapes, null and misaligned pointers, an unsupported device)
and by the binding (tensors that do not cover what a call touches). No GPU."""

import pytest

from bit_quantized_linear_amd import binding as b
from tests.test_binding_checks import Dev, Reached, guarded  # noqa: F401

FAKE = 0x10000
MISALIGNED = 0x10008
INVALID, SHAPE, MIS = b.SVDQ_ERR_INVALID_ARGUMENT, b.SVDQ_ERR_UNSUPPORTED_SHAPE, b.SVDQ_ERR_MISALIGNED


def quantize(X=FAKE, M=16, K=128, qx=FAKE, sx=FAKE):
    return b.lib().svdq_fp8_quantize_act(X, M, K, qx, sx, None)


def gemm(qx=FAKE, sx=FAKE, qw=FAKE, sw=FAKE, bias=None, M=16, N=64, K=128, Y=FAKE, dt=0):
    return b.lib().svdq_fp8_gemm(qx, sx, qw, sw, bias, M, N, K, Y, dt, None)


def linear(X=FAKE, qw=FAKE, sw=FAKE, bias=None, M=16, N=64, K=128, ws=FAKE, wb=1 << 20, Y=FAKE, dt=0):
    return b.lib().svdq_fp8_linear(X, qw, sw, bias, M, N, K, ws, wb, Y, dt, None)


def moe(X=FAKE, wr=FAKE, w13=FAKE, s13=FAKE, w2=FAKE, s2=FAKE, T=2, H=64, I=32, E=4, k=2, idx=None,  # noqa: E741
        gate=None, ws=FAKE, wb=1 << 20, Y=FAKE):
    return b.lib().svdq_fp8_moe_layer(X, wr, w13, s13, w2, s2, T, H, I, E, k, 1, idx, gate, ws, wb, Y, None)


@pytest.mark.parametrize("call,args,status", [
    (quantize, {"M": -1}, INVALID), (quantize, {"K": 0}, INVALID), (quantize, {"K": 120}, SHAPE),
    (quantize, {"K": 1 << 22}, SHAPE), (quantize, {"X": None}, INVALID), (quantize, {"sx": None}, INVALID),
    (quantize, {"qx": MISALIGNED}, MIS),
    (gemm, {"M": -1}, INVALID), (gemm, {"N": 0}, INVALID), (gemm, {"K": 72}, SHAPE), (gemm, {"N": 60}, SHAPE),
    (gemm, {"K": 1 << 22}, SHAPE), (gemm, {"M": 2147483647, "N": 8}, SHAPE), (gemm, {"M": 1, "N": 2147483640}, SHAPE),
    (quantize, {"M": 2147483647}, SHAPE), (quantize, {"M": (1 << 28) - 15}, SHAPE),
    (gemm, {"M": 1, "N": 1 << 27}, SHAPE), (linear, {"M": 1, "N": (1 << 27) - 24, "K": 16}, SHAPE),
    (gemm, {"M": (1 << 28) - 15, "N": 8}, SHAPE), (linear, {"M": (1 << 28) - 15, "N": 8}, SHAPE),
    (gemm, {"M": 2147483647, "N": 2147483640}, SHAPE), (gemm, {"dt": 2}, INVALID),
    (gemm, {"qw": None}, INVALID), (gemm, {"sx": None}, INVALID), (gemm, {"Y": None}, INVALID),
    (gemm, {"bias": MISALIGNED}, MIS), (gemm, {"sw": MISALIGNED}, MIS),
    (linear, {"wb": 16 * 128}, INVALID), (linear, {"ws": None}, INVALID), (linear, {"X": None}, INVALID),
    (linear, {"X": MISALIGNED}, MIS), (linear, {"N": 4}, SHAPE), (linear, {"K": 24}, SHAPE),
    (moe, {"T": -1}, INVALID), (moe, {"T": 65}, SHAPE), (moe, {"H": 72}, SHAPE), (moe, {"I": 40}, SHAPE),
    (moe, {"E": 257}, SHAPE), (moe, {"k": 0}, INVALID), (moe, {"k": 5}, INVALID),
    (moe, {"E": 64, "k": 17}, SHAPE), (moe, {"T": 64, "E": 64, "k": 16, "I": 1 << 20}, SHAPE), (moe, {"wb": 64}, INVALID), (moe, {"ws": None}, INVALID),
    (moe, {"w13": None}, INVALID), (moe, {"s2": None}, INVALID), (moe, {"X": None}, INVALID),
    (moe, {"Y": None}, INVALID), (moe, {"idx": MISALIGNED}, MIS), (moe, {"w2": MISALIGNED}, MIS),
], ids=str)
def test_refused_before_a_launch(call, args, status):
    assert call(**args) == status


@pytest.mark.parametrize("call", [quantize, gemm, linear, moe])
def test_other_devices_fail_closed(call):
    b.svdq_debug_set_arch_override("gfx942")
    try:
        assert call() == b.SVDQ_ERR_UNSUPPORTED_DEVICE
    finally:
        b.svdq_debug_set_arch_override(None)


def test_workspace_bytes():
    assert b.svdq_fp8_workspace_bytes(3, 144) >= 3 * 144 + 4 * 2 * 3
    assert b.svdq_fp8_workspace_bytes(0, 144) == 0 and b.svdq_fp8_workspace_bytes(-1, 144) == 0
    assert b.svdq_fp8_workspace_bytes(3, 100) == 0
    assert b.svdq_fp8_moe_workspace_bytes(2, 32, 4, 2) >= 2 * 2 * 2 * 32 * 2
    for bad in ((-1, 32, 4, 2), (65, 32, 4, 2), (2, 40, 4, 2), (2, 32, 0, 2), (2, 32, 257, 2), (2, 32, 4, 5)):
        assert b.svdq_fp8_moe_workspace_bytes(*bad) == 0


def _case(name):
    M, K, N = 40, 144, 136
    ws = lambda n: Dev((n,), 1)  # noqa: E731
    if name == "quantize":
        return lambda t: b.svdq_fp8_quantize_act(t["X"], t["qx"], t["sx"]), {
            "X": Dev((M, K), 2), "qx": Dev((M, K), 1), "sx": Dev((2, M), 4)}
    if name == "gemm":
        return lambda t: b.svdq_fp8_gemm(t["qx"], t["sx"], t["qw"], t["sw"], t["bias"], t["Y"]), {
            "qx": Dev((M, K), 1), "sx": Dev((2, M), 4), "qw": Dev((N, K), 1), "sw": Dev((2, 2), 4),
            "bias": Dev((N,), 2), "Y": Dev((M, N), 2)}
    if name == "linear":
        return lambda t: b.svdq_fp8_linear(t["X"], t["qw"], t["sw"], t["bias"], t["ws"], t["Y"]), {
            "X": Dev((M, K), 2), "qw": Dev((N, K), 1), "sw": Dev((2, 2), 4), "bias": Dev((N,), 2),
            "ws": ws(b.svdq_fp8_workspace_bytes(M, K)), "Y": Dev((M, N), 4)}
    T, H, I, E, k = 3, 144, 48, 5, 2  # noqa: E741
    return lambda t: b.svdq_fp8_moe_layer(t["X"], t["wr"], t["w13"], t["s13"], t["w2"], t["s2"], t["Y"], t["idx"],
                                          t["gate"], t["ws"]), {
        "X": Dev((T, H), 2), "wr": Dev((E, H), 2), "w13": Dev((E, 2, I, H), 1), "s13": Dev((E, 2, 1, 2), 4),
        "w2": Dev((E, H, I), 1), "s2": Dev((E, 2, 1), 4), "Y": Dev((T, H), 2), "idx": Dev((T, k), 4),
        "gate": Dev((T, k), 4), "ws": ws(b.svdq_fp8_moe_workspace_bytes(T, I, E, k))}


class SizeQueries:
    """The guard of the shared fixture lets the older size queries through;
    the ones here go to the library too."""

    def __init__(self, guard):
        self.guard = guard

    def __getattr__(self, name):
        if name in ("svdq_fp8_workspace_bytes", "svdq_fp8_moe_workspace_bytes"):
            return getattr(self.guard.real, name)
        return getattr(self.guard, name)


@pytest.mark.parametrize("name", ["quantize", "gemm", "linear", "moe"])
def test_the_binding_checks_every_tensor(name, guarded, monkeypatch):  # noqa: F811
    sized = SizeQueries(guarded)
    monkeypatch.setattr(b, "lib", lambda: sized)
    call, tensors = _case(name)
    with pytest.raises(Reached):
        call(tensors)
    for arg, t in tensors.items():
        short = Dev((1,) * len(t.shape), t.element_size())
        if (name, arg) != ("quantize", "X"):  # whose shape is what gives the sizes
            with pytest.raises((ValueError, TypeError)):
                call({**tensors, arg: short})
        with pytest.raises((ValueError, TypeError)):
            call({**tensors, arg: Dev(t.shape, t.element_size(), device=1)})
        if arg != "ws":
            with pytest.raises((ValueError, TypeError)):
                call({**tensors, arg: Dev(t.shape, 8)})


def test_moe_shapes_that_do_not_fit(guarded, monkeypatch):  # noqa: F811
    sized = SizeQueries(guarded)
    monkeypatch.setattr(b, "lib", lambda: sized)
    call, t = _case("moe")
    for arg, shape in (("wr", (5, 128)), ("w13", (5, 2, 48, 128)), ("w13", (4, 2, 48, 144)), ("w2", (5, 48, 144)),
                       ("gate", (3, 3)), ("idx", (2, 2))):
        with pytest.raises(ValueError):
            call({**t, arg: Dev(shape, t[arg].element_size())})
    with pytest.raises(ValueError):
        b.svdq_fp8_moe_layer(t["X"], t["wr"], t["w13"], t["s13"], t["w2"], t["s2"], t["Y"], None, None, t["ws"])


@pytest.mark.parametrize("name", ["gemm", "linear"])
def test_an_output_is_needed_for_its_type(name, guarded, monkeypatch):  # noqa: F811
    sized = SizeQueries(guarded)
    monkeypatch.setattr(b, "lib", lambda: sized)
    call, t = _case(name)
    with pytest.raises(TypeError, match="Y"):
        call({**t, "Y": None})


# of every tensor: the types a call takes (integers of the width hold the bits), and some of the same width that are
# another format or another kind of number
E4M3 = (["float8_e4m3fn", "uint8", "int8"],
        ["float8_e4m3fnuz", "float8_e5m2", "float8_e5m2fnuz", "float8_e8m0fnu", "bool"])
BF16 = (["bfloat16", "int16", "uint16"], ["float16"])
F32 = (["float32"], ["int32"])
I32 = (["int32", "uint32"], ["float32"])
FORMATS = {
    "quantize": {"X": BF16, "qx": E4M3, "sx": F32},
    "gemm": {"qx": E4M3, "sx": F32, "qw": E4M3, "sw": F32, "bias": BF16, "Y": BF16},
    "linear": {"X": BF16, "qw": E4M3, "sw": F32, "bias": BF16, "Y": F32},
    "moe": {"X": BF16, "wr": BF16, "w13": E4M3, "s13": F32, "w2": E4M3, "s2": F32, "Y": BF16, "idx": I32, "gate": F32},
}


@pytest.mark.parametrize("name", list(FORMATS))
def test_tensors_of_another_format_are_refused(name, guarded, monkeypatch):  # noqa: F811
    import torch

    sized = SizeQueries(guarded)
    monkeypatch.setattr(b, "lib", lambda: sized)
    call, tensors = _case(name)
    assert set(FORMATS[name]) == set(tensors) - {"ws"}
    for arg, (taken, refused) in FORMATS[name].items():
        for dtype in taken + refused:
            t = Dev(tensors[arg].shape, tensors[arg].element_size())
            t.dtype, t.get_device = getattr(torch, dtype), lambda: 0
            assert t.dtype.itemsize == t.element_size()
            with pytest.raises(Reached if dtype in taken else TypeError, match=None if dtype in taken else arg):
                call({**tensors, arg: t})


# scales in another order have the same bytes; a flat buffer is taken by its size
@pytest.mark.parametrize("name,arg,wrong,flat", [
    ("quantize", "sx", (40, 2), (2 * 40 + 5,)), ("gemm", "sx", (40, 2), (2 * 40,)), ("gemm", "sw", (1, 4), (4,)),
    ("linear", "sw", (1, 4), (5,)), ("moe", "s13", (5, 2, 2, 1), (20,)), ("moe", "s13", (5, 1, 2, 2), (20,)),
    ("moe", "s2", (5, 1, 2), (10,)),
])
def test_scales_in_another_order_are_refused(name, arg, wrong, flat, guarded, monkeypatch):  # noqa: F811
    sized = SizeQueries(guarded)
    monkeypatch.setattr(b, "lib", lambda: sized)
    call, tensors = _case(name)
    right = tensors[arg].shape
    for shape, what in ((wrong, ValueError), (flat, Reached), ((right[0] + 1,) + right[1:], Reached)):
        with pytest.raises(what, match=arg if what is ValueError else None):
            call({**tensors, arg: Dev(shape, 4)})


def test_workspace_of_shapes_that_no_call_takes():
    # K from 2^22, M past 2^28 - 16, and numbers whose blocks of 128 pass 31 bits
    for M, K in ((1, 1 << 22), (1, 2147483632), (64, 2147483632), ((1 << 28) - 15, 16), (2147483647, 16),
                 (2147483647, 2147483632)):
        assert b.svdq_fp8_workspace_bytes(M, K) == 0
        if M <= (1 << 28) - 16:
            assert linear(M=M, K=K) == SHAPE
    M, K = (1 << 28) - 16, (1 << 22) - 16
    assert b.svdq_fp8_workspace_bytes(M, K) >= M * K + 4 * M * (1 << 15)


def test_typed_tensors_elsewhere_are_refused(guarded, monkeypatch):  # noqa: F811
    import torch

    sized = SizeQueries(guarded)
    monkeypatch.setattr(b, "lib", lambda: sized)
    call, tensors = _case("gemm")
    with pytest.raises(TypeError, match="sx: device entry points take GPU tensors"):
        call({**tensors, "sx": torch.zeros((2, 40))})
    other = Dev((2, 40), 4)
    other.dtype, other.get_device = torch.float32, lambda: 1
    with pytest.raises(TypeError, match="sx is on cuda:1, the current device is cuda:0"):
        call({**tensors, "sx": other})
