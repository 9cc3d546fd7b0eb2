"""The module with which the binding looks at a call's tensors: on the CPU it refuses
every tensor, and the binding does without it where it was not built."""

import importlib
import sys

import pytest

from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import build


def test_it_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    pointers, heads, e4m3, bf16, f32, i32, f64 = b._quick()
    x = torch.zeros((2, 4, 8), dtype=torch.bfloat16)
    assert pointers(0, x, bf16, 0) is None and heads(0, bf16, x) is None
    assert pointers(0, None, bf16, 0) == (None,) and pointers(0) == ()
    assert len({e4m3, bf16, f32, i32, f64}) == 5 and all(bin(k).count("1") >= 1 for k in (e4m3, bf16, f32, i32, f64))
    assert not any(a & c for i, a in enumerate((e4m3, bf16, f32, i32, f64)) for c in (e4m3, bf16, f32, i32, f64)[:i])
    with pytest.raises(TypeError):
        importlib.import_module("bit_quantized_linear_amd._tensors").kind(3)
    for wrong in ((), (0, x), ("0", x, bf16, 0)):
        with pytest.raises(TypeError):
            pointers(*wrong)


def test_the_binding_does_without_it(monkeypatch):
    monkeypatch.setattr(b, "_quick_calls", None)
    monkeypatch.setitem(sys.modules, "bit_quantized_linear_amd._tensors", None)
    monkeypatch.delattr("bit_quantized_linear_amd._tensors", raising=False)
    assert b._quick() == ()


def test_it_is_built_beside_the_library():
    assert build._tensors_job()[-1] == build.TENSORS + ".tmp"
