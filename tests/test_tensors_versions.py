"""The module with which the binding looks at a call's tensors reads torch's and Python's
own structures: it is used with the torch and Python that it was built for, and with no
other. No GPU."""

import sys

import pytest

from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import build

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _fresh(monkeypatch):
    monkeypatch.setattr(b, "_quick_calls", None)


def test_it_says_what_it_was_built_for():
    from bit_quantized_linear_amd import _tensors

    assert torch.__version__ in _tensors.built_for and torch.version.git_version in _tensors.built_for
    assert sys.implementation.cache_tag in _tensors.built_for
    assert len(b._quick()) == 7


@pytest.mark.parametrize("where,name,value", [(torch, "__version__", "2.0.0"), (torch.version, "git_version", "0" * 40),
                                              (sys.implementation, "cache_tag", "cpython-399")])
def test_another_torch_or_python_does_without_it(monkeypatch, where, name, value):
    monkeypatch.setattr(where, name, value)
    assert b._quick() == ()


def test_one_that_does_not_say_is_not_used(monkeypatch):
    from bit_quantized_linear_amd import _tensors

    monkeypatch.delattr(_tensors, "built_for")
    assert b._quick() == ()


def test_its_file_is_this_pythons_and_a_build_leaves_no_other(monkeypatch, tmp_path):
    import importlib.machinery as machinery

    assert build.TENSORS.endswith(machinery.EXTENSION_SUFFIXES[0])
    old = ["_tensors.so", "_tensors.cpython-39-x86_64-linux-gnu.so"]
    for name in old + ["libsvdq.so", "_other.so"]:
        (tmp_path / name).write_text("")
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    build._remove_tensors()
    assert sorted(p.name for p in tmp_path.iterdir()) == ["_other.so", "libsvdq.so"]
