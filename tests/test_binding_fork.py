"""The binding keeps two of torch's functions for the current device and stream,
which skip torch's own check of the process. A child that is forked from a
process with a GPU in use must get torch's error on its first call, not an
answer that belongs to its parent. No GPU: torch's side is a stand-in."""

import os

import pytest
import torch

from bit_quantized_linear_amd import binding as b


class Refused(RuntimeError):
    pass


def _refuse():
    raise Refused("Cannot re-initialize CUDA in forked subprocess")


def _in_child(call):
    """What `call` does in a forked child: "refused" or what it returned."""
    r, w = os.pipe()
    pid = os.fork()
    if pid == 0:
        try:
            said = str(call())
        except Refused:
            said = "refused"
        except BaseException as e:  # noqa: BLE001
            said = repr(e)
        os.write(w, said.encode())
        os._exit(0)
    os.close(w)
    said = os.read(r, 200).decode()
    os.close(r)
    os.waitpid(pid, 0)
    return said


@pytest.fixture
def started(monkeypatch):
    """The binding after a first call, and torch refusing from now on."""
    monkeypatch.setattr(b, "_device_of", None)
    monkeypatch.setattr(b, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 7, raising=False)
    assert b._current_device() == 0 and b._stream(None) == 7
    monkeypatch.setattr(torch.cuda, "current_device", _refuse)


def test_a_forked_child_is_refused(started):
    assert b._current_device() == 0 and b._stream(None) == 7  # here as before
    assert _in_child(b._current_device) == "refused"
    assert _in_child(lambda: b._stream(None)) == "refused"
    assert b._current_device() == 0 and b._stream(None) == 7


def test_a_child_of_a_process_without_a_call_starts_anew(monkeypatch):
    monkeypatch.setattr(b, "_device_of", None)
    monkeypatch.setattr(b, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert _in_child(b._current_device) == "3"
