"""What the norm, the rotary positions and the 8-bit cache's entry points refuse,
before anything is launched: by the library (shapes, null and misaligned pointers,
an unsupported device) and by the binding (tensors that do not cover what a call
touches, of another type, layout or device). No GPU."""

import types

import numpy as np
import pytest
import torch

from bit_quantized_linear_amd import binding as b
from tests.test_binding_checks import Reached

FAKE = 0x10000
MISALIGNED = 0x10008
INVALID, SHAPE, MIS = b.SVDQ_ERR_INVALID_ARGUMENT, b.SVDQ_ERR_UNSUPPORTED_SHAPE, b.SVDQ_ERR_MISALIGNED
INF, NAN = float("inf"), float("nan")


def norm(X=FAKE, r=FAKE, w=FAKE, eps=1e-6, M=4, K=128, total=FAKE, Y=FAKE, qx=FAKE, sx=FAKE):
    return b.lib().svdq_fp8_norm_quantize(X, r, w, eps, M, K, total, Y, qx, sx, None)


def rope(X=FAKE, xs=256, pos=FAKE, freqs=FAKE, sections=(16, 8, 8), axes=None, T=4, H=4, D=64, Y=FAKE, ys=256):
    held = None if sections is None else (b._i * max(1, len(sections)))(*sections)
    return b.lib().svdq_rope(X, xs, pos, freqs, held, len(sections or ()) if axes is None else axes, 0, T, H, D, Y, ys,
                             None)


def append(K=FAKE, ks=128, V=FAKE, vs=128, starts=FAKE, lengths=FAKE, table=FAKE, T=4, B=2, pages=8, P=16, Hk=2, D=64,
           cache=(FAKE,) * 4):
    return b.lib().svdq_kv8_append(K, ks, V, vs, starts, lengths, table, T, B, pages, P, Hk, D, *cache, None)


def attention(Q=FAKE, qs=256, cache=(FAKE,) * 4, starts=FAKE, lengths=FAKE, table=FAKE, T=4, B=2, pages=8, P=16, Hq=4,
              Hk=2, D=64, scale=0.125, causal=1, window=0, O=FAKE, lse=None, ws=FAKE, wb=1 << 30):  # noqa: E741
    return b.lib().svdq_kv8_attention(Q, qs, *cache, starts, lengths, table, T, B, pages, P, Hq, Hk, D, scale, causal,
                                      window, O, lse, ws, wb, None)


@pytest.mark.parametrize("call,args,status", [
    (norm, {"M": -1}, INVALID), (norm, {"K": 0}, INVALID), (norm, {"eps": -1.0}, INVALID), (norm, {"eps": NAN}, INVALID),
    (norm, {"eps": INF}, INVALID), (norm, {"K": 120}, SHAPE), (norm, {"K": 1 << 22}, SHAPE), (norm, {"M": 1 << 22}, SHAPE),
    (norm, {"X": None}, INVALID), (norm, {"w": None}, INVALID), (norm, {"qx": None}, INVALID), (norm, {"sx": None}, INVALID),
    (norm, {"Y": None, "qx": None, "sx": None}, INVALID), (norm, {"r": MISALIGNED}, MIS), (norm, {"total": MISALIGNED}, MIS),
    (norm, {"Y": MISALIGNED}, MIS), (norm, {"sx": MISALIGNED}, MIS),
    (rope, {"T": -1}, INVALID), (rope, {"H": 0}, INVALID), (rope, {"D": 0}, INVALID), (rope, {"axes": 0}, INVALID),
    (rope, {"sections": (8,) * 5}, SHAPE), (rope, {"sections": (8, -8, 8)}, INVALID), (rope, {"sections": (0,)}, INVALID),
    (rope, {"sections": None, "axes": 1}, INVALID), (rope, {"sections": (12,)}, SHAPE), (rope, {"sections": (40,)}, SHAPE),
    (rope, {"sections": (264,), "D": 1024, "xs": 4096, "ys": 4096}, SHAPE), (rope, {"D": 68, "xs": 1024, "ys": 1024}, SHAPE),
    (rope, {"xs": 248}, INVALID), (rope, {"ys": 255}, INVALID), (rope, {"xs": 260}, SHAPE), (rope, {"T": 1 << 24}, SHAPE),
    (rope, {"H": 1 << 18, "xs": 1 << 24, "ys": 1 << 24}, SHAPE), (rope, {"xs": 512}, INVALID),  # in place: one stride
    (rope, {"X": None}, INVALID), (rope, {"pos": None}, INVALID), (rope, {"freqs": None}, INVALID),
    (rope, {"Y": MISALIGNED}, MIS), (rope, {"pos": MISALIGNED}, MIS),
    (append, {"T": -1}, INVALID), (append, {"B": -1}, INVALID), (append, {"pages": 0}, INVALID), (append, {"P": 0}, INVALID),
    (append, {"Hk": 0}, INVALID), (append, {"D": 96}, SHAPE), (append, {"T": 1 << 24}, SHAPE), (append, {"B": 65536}, SHAPE),
    (append, {"Hk": 1025, "ks": 1 << 20, "vs": 1 << 20}, SHAPE), (append, {"pages": (1 << 24) + 1}, SHAPE),
    (append, {"ks": 120}, INVALID), (append, {"vs": 132}, SHAPE), (append, {"K": None}, INVALID),
    (append, {"starts": None}, INVALID), (append, {"table": None}, INVALID), (append, {"V": MISALIGNED}, MIS),
    (append, {"cache": (FAKE, FAKE, None, FAKE)}, INVALID), (append, {"cache": (FAKE, MISALIGNED, FAKE, FAKE)}, MIS),
    (attention, {"T": -1}, INVALID), (attention, {"D": 32}, SHAPE), (attention, {"Hq": 5, "qs": 512}, SHAPE),
    (attention, {"Hq": 0}, INVALID), (attention, {"qs": 248}, INVALID), (attention, {"scale": 0.0}, INVALID),
    (attention, {"scale": NAN}, INVALID), (attention, {"scale": INF}, INVALID), (attention, {"scale": -1.0}, INVALID),
    (attention, {"window": -1}, INVALID), (attention, {"window": 4, "causal": 0}, INVALID),
    (attention, {"B": 65535, "Hq": 1024, "Hk": 1024, "qs": 1 << 20}, SHAPE),
    (attention, {"T": (1 << 24) - 1, "Hq": 65, "Hk": 65, "qs": 4160}, SHAPE), (attention, {"Q": None}, INVALID),
    (attention, {"O": None}, INVALID), (attention, {"lengths": None}, INVALID), (attention, {"ws": None, "pages": 512}, INVALID),
    (attention, {"wb": 64, "pages": 512}, INVALID), (attention, {"lse": MISALIGNED}, MIS), (attention, {"table": MISALIGNED}, MIS),
], ids=str)
def test_refused_before_a_launch(call, args, status):
    assert call(**args) == status


@pytest.mark.parametrize("call", [norm, rope, append, attention])
def test_other_devices_fail_closed(call):
    b.svdq_debug_set_arch_override("gfx942")
    try:
        assert call() == b.SVDQ_ERR_UNSUPPORTED_DEVICE
    finally:
        b.svdq_debug_set_arch_override(None)


@pytest.mark.parametrize("call,args", [(norm, {"M": 0, "X": None}), (rope, {"T": 0, "X": None}), (append, {"T": 0, "K": None}),
                                       (append, {"B": 0, "table": None}), (attention, {"T": 0, "Q": None, "ws": None}),
                                       (attention, {"B": 0, "ws": None})], ids=str)
def test_empty_calls_launch_nothing(call, args):
    b.svdq_debug_set_arch_override("gfx950")
    try:
        assert call(**args) == b.SVDQ_OK
    finally:
        b.svdq_debug_set_arch_override(None)


def test_workspace_of_what_is_refused_is_0():
    ws = b.svdq_kv8_attention_workspace_bytes
    assert ws(1, 1, 512, 32, 8, 128) > 0
    for args in ((-1, 1, 512, 32, 8, 128), (1, 1, 0, 32, 8, 128), (1, 1, 512, 30, 8, 128), (1, 1, 512, 32, 8, 96),
                 (0, 1, 512, 32, 8, 128), (1, 0, 512, 32, 8, 128), (4096, 1, 512, 32, 8, 128)):
        assert ws(*args) == 0, args


class Dev:
    """Stand-in for a torch tensor on a GPU."""

    def __init__(self, shape, dtype, device=0, stride=None):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, device >= 0
        self.device = types.SimpleNamespace(index=device)
        plain = [int(np.prod(shape[i + 1:])) for i in range(len(shape))]
        self._stride = tuple(plain if stride is None else stride)
        self._plain = self._stride == tuple(plain)

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self._stride

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return self.dtype.itemsize

    @property
    def nbytes(self):
        return self.numel() * self.element_size()

    def is_contiguous(self):
        return self._plain

    def data_ptr(self):
        return FAKE


class Guard:
    """Size queries go to the real library; an entry point raises Reached."""

    def __init__(self, real):
        self.real = real

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def entry(*args):
            raise Reached(name)

        return entry


@pytest.fixture
def guarded(monkeypatch):
    guard = Guard(b.lib())
    monkeypatch.setattr(b, "lib", lambda: guard)
    monkeypatch.setattr(b, "_current_device", lambda: 0)
    monkeypatch.setattr(b, "_stream", lambda s: None)


BF, F32, F64, I32, E4 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.float8_e4m3fn
T, B, PAGES, P, HQ, HK, D, M, K = 6, 3, 40, 50, 4, 2, 64, 5, 144
CALLS = {
    "norm": (lambda t: b.svdq_fp8_norm_quantize(t["X"], t["residual"], t["weight"], 1e-6, t["total"], t["Y"], t["qx"], t["sx"]),
             {"X": ((M, K), BF), "residual": ((M, K), BF), "weight": ((K,), BF), "total": ((M, K), BF), "Y": ((M, K), BF),
              "qx": ((M, K), E4), "sx": ((2, M), F32)}),
    "rope": (lambda t: b.svdq_rope(t["X"], t["positions"], t["freqs"], (10, 6), t["Y"]),
             {"X": ((T, HQ, D), BF), "positions": ((T, 2), I32), "freqs": ((16,), F64), "Y": ((T, HQ, D), BF)}),
    "append": (lambda t: b.svdq_kv8_append(t["K"], t["V"], t["starts"], t["lengths"], t["table"], t["kc"], t["ks"], t["vc"],
                                           t["vs"]),
               {"K": ((T, HK, D), BF), "V": ((T, HK, D), BF), "starts": ((B + 1,), I32), "lengths": ((B,), I32),
                "table": ((B, PAGES), I32), "kc": ((P, HK, 64, D), E4), "ks": ((P, HK), F32), "vc": ((P, HK, D, 64), E4),
                "vs": ((P, HK), F32)}),
    "attention": (lambda t: b.svdq_kv8_attention(t["Q"], t["kc"], t["ks"], t["vc"], t["vs"], t["starts"], t["lengths"],
                                                 t["table"], 0.1, t["O"], t["lse"], t["workspace"]),
                  {"Q": ((T, HQ, D), BF), "starts": ((B + 1,), I32), "lengths": ((B,), I32), "table": ((B, PAGES), I32),
                   "kc": ((P, HK, 64, D), E4), "ks": ((P, HK), F32), "vc": ((P, HK, D, 64), E4), "vs": ((P, HK), F32),
                   "O": ((T, HQ, D), BF), "lse": ((T, HQ), F32), "workspace": (
                       (b.svdq_kv8_attention_workspace_bytes(T, B, PAGES, HQ, HK, D),), torch.uint8)}),
}
EACH = [(c, n) for c, (_, t) in CALLS.items() for n in t]


def tensors(call, **changed):
    return {n: changed[n] if n in changed else Dev(s, d) for n, (s, d) in CALLS[call][1].items()}


@pytest.mark.parametrize("call", CALLS)
def test_well_formed_arguments_reach_the_library(call, guarded):
    with pytest.raises(Reached):
        CALLS[call][0](tensors(call))


@pytest.mark.parametrize("call,name", EACH)
def test_a_tensor_too_small_or_elsewhere_or_of_another_type_is_refused(call, name, guarded):
    shape, dtype = CALLS[call][1][name]
    other = {BF: torch.float16, F32: BF, F64: F32, I32: torch.int64, E4: torch.float8_e5m2, torch.uint8: None}[dtype]
    if name not in ("X", "K", "Q", "table", "workspace"):  # what gives the call its sizes
        with pytest.raises(ValueError):
            CALLS[call][0](tensors(call, **{name: Dev(shape[:-1] + (shape[-1] - 1,), dtype)}))
    with pytest.raises(TypeError):
        CALLS[call][0](tensors(call, **{name: Dev(shape, dtype, device=1)}))
    with pytest.raises(TypeError):
        CALLS[call][0](tensors(call, **{name: Dev(shape, dtype, device=-1)}))
    if other is not None:
        with pytest.raises(TypeError):
            CALLS[call][0](tensors(call, **{name: Dev(shape, other)}))


@pytest.mark.parametrize("call,name", [("rope", "X"), ("rope", "Y"), ("append", "K"), ("append", "V"), ("attention", "Q")])
def test_rows_may_be_parts_of_wider_ones_and_nothing_else(call, name, guarded):
    (n, H, d), dtype = CALLS[call][1][name]
    ok = Dev((n, H, d), dtype, stride=(3 * H * d, d, 1))
    with pytest.raises(Reached):
        CALLS[call][0](tensors(call, **{name: ok}))
    for stride in ((H * d, 1, H), (H * d, 2 * d, 1), (0, d, 1), (d, n * d, 1), (H * d - 8, d, 1)):
        with pytest.raises(TypeError):
            CALLS[call][0](tensors(call, **{name: Dev((n, H, d), dtype, stride=stride)}))


@pytest.mark.parametrize("call,name", [("attention", "O"), ("append", "kc"), ("attention", "vc"), ("rope", "positions"),
                                       ("norm", "X"), ("norm", "total"), ("append", "table")])
def test_other_tensors_are_contiguous(call, name, guarded):
    shape, dtype = CALLS[call][1][name]
    with pytest.raises(TypeError):
        CALLS[call][0](tensors(call, **{name: Dev(shape, dtype, stride=tuple(range(1, len(shape) + 1)))}))


def test_a_missing_workspace_reaches_the_library_which_refuses_it(guarded):
    with pytest.raises(Reached):
        CALLS["attention"][0](tensors("attention", workspace=None))


def test_scales_that_overflow():
    """Scores are base-2 logarithms: the scale times log2 e has to be a number."""
    assert attention(scale=2.0 ** 126.5) == INVALID and attention(scale=3.4e38) == INVALID
    b.svdq_debug_set_arch_override("gfx950")
    try:
        assert attention(T=0, Q=None, ws=None, scale=2.0 ** 126) == b.SVDQ_OK
    finally:
        b.svdq_debug_set_arch_override(None)
