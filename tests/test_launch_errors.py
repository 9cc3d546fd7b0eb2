"""A launch that the runtime refuses: the call says so, and leaves no error behind for
whoever asks next (torch looks for one after each of its own launches). In a process of
its own, with the runtime's launch and error calls replaced. No GPU."""

import os
import shutil
import subprocess
import sys

import pytest

from bit_quantized_linear_amd import binding as b

RUNTIME = r"""
struct dim3 { unsigned x, y, z; };
static int last = 0, launches = 0, fail = 0;
extern "C" {
int hipLaunchKernel(const void *, dim3, dim3, void **, unsigned long, void *) { ++launches; return last = fail; }
int hipGetLastError() { const int e = last; last = 0; return e; }
void runtime_fails(int e) { fail = e; }
int runtime_launches() { return launches; }
int runtime_last() { return last; }
}
"""

CALLS = r"""
import ctypes as C, sys
sys.path.insert(0, sys.argv[3])
from bit_quantized_linear_amd import binding as b
runtime = C.CDLL(sys.argv[1], mode=C.RTLD_GLOBAL)
lib = C.CDLL(sys.argv[2])
for name, (res, args) in b.SIGNATURES.items():
    getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
assert lib.svdq_debug_set_arch_override(b"gfx950") == b.SVDQ_OK
A = 0x10000  # never looked at: nothing is launched
two = (C.c_int * 1)(8)
calls = {
    "norm": lambda: lib.svdq_fp8_norm_quantize(A, None, A, 1e-6, 4, 128, None, A, None, None, None),
    "rope": lambda: lib.svdq_rope(A, 64, A, A, two, 1, 0, 4, 1, 64, A, 64, None),
    "append": lambda: lib.svdq_kv8_append(A, 64, A, 64, A, A, A, 4, 1, 2, 4, 1, 64, A, A, A, A, None),
    "few": lambda: lib.svdq_kv8_attention(A, 64, A, A, A, A, A, A, A, 4, 1, 2, 4, 1, 1, 64, 0.1, 1, 0, A, None, None, 0, None),
    "many": lambda: lib.svdq_kv8_attention(A, 64, A, A, A, A, A, A, A, 400, 1, 2, 4, 1, 1, 64, 0.1, 1, 0, A, None, None, 0,
                                           None),
}
for name, call in calls.items():
    for error, status in ((0, b.SVDQ_OK), (1, b.SVDQ_ERR_HIP), (98, b.SVDQ_ERR_HIP), (0, b.SVDQ_OK)):
        runtime.runtime_fails(error)
        before = runtime.runtime_launches()
        got = call()
        assert runtime.runtime_launches() == before + 1, "the call reaches the replaced launch"
        assert (got, runtime.runtime_last()) == (status, 0), (name, error, got, runtime.runtime_last())
print("good")
"""


def test_a_refused_launch_leaves_no_error_behind(tmp_path):
    if os.path.exists("/dev/kfd"):
        pytest.skip("a GPU is present: nothing may be launched here")
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    source, runtime = tmp_path / "runtime.cpp", tmp_path / "runtime.so"
    source.write_text(RUNTIME)
    subprocess.run([cxx, "-shared", "-fPIC", "-o", str(runtime), str(source)], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(b.__file__)))
    p = subprocess.run([sys.executable, "-c", CALLS, str(runtime), b.LIB_PATH, root], stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.endswith("good\n"), p.stdout
