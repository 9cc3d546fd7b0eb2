"""The host preparation shares its work with threads. Where the process may start
no more of them, it does the work itself: a C entry has no one to throw to, so
an exception there would end the process. No GPU; the call runs in a process
of its own, whose address space has no room for another thread's stack."""

import os
import subprocess
import sys

CHILD = """
import resource, sys, threading
import numpy as np
from bit_quantized_linear_amd import binding as b
from bit_quantized_linear_amd import workloads as wl

b.lib()
bits = wl.random_bf16(1, (256, 1024), 0.02)["bits"]
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
if sys.argv[1] == "full":
    resource.setrlimit(resource.RLIMIT_AS, (size + (64 << 20), resource.RLIM_INFINITY))
    try:
        threading.Thread(target=lambda: None).start()
    except RuntimeError:
        pass
    else:
        sys.exit("a thread could start")
q, s = b.svdq_fp8_prepare_weights(bits)
w, ws = b.w8a8_prepare_weights(bits)
sys.stdout.buffer.write(q.tobytes() + s.tobytes() + w.tobytes())
"""


def _run(kind):
    import resource

    def stack():  # what a new thread's stack takes, 4 times the room left
        resource.setrlimit(resource.RLIMIT_STACK, (256 << 20, resource.getrlimit(resource.RLIMIT_STACK)[1]))

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = {**os.environ, "SVDQ_HOST_THREADS": "4", "OMP_NUM_THREADS": "1", "PYTHONPATH": root}
    return subprocess.run([sys.executable, "-c", CHILD, kind], env=env, cwd=root, capture_output=True,
                          preexec_fn=stack, timeout=120)


def test_preparation_without_room_for_threads():
    free, full = _run("free"), _run("full")
    assert free.returncode == 0, free.stderr.decode()[-500:]
    assert full.returncode == 0, full.stderr.decode()[-500:]
    assert full.stdout == free.stdout and len(free.stdout) > 2 * 256 * 1024
