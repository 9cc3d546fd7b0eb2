"""The wait guard of test_lds_stage_waits.py for the tiles of the block-scaled FP8
product, which keep a later stage's direct-to-LDS loads under way while they
read the current one. Compiled as the library is; no GPU. (The experts' kernels
are not held to it: down waits for the slots that it has just filled, and up
mixes in loads to registers, which the guard takes for the end of a stage.)"""

import os
import re
import subprocess

from bit_quantized_linear_amd import build as B
from tests.test_lds_stage_waits import _stalls, pytestmark  # noqa: F401

KERNELS = ["fp8_gemm_kernel", "fp8_gemm256_kernel"]


def _functions(src, tmp_path):
    """{symbol: its lines} of a source's gfx950 assembly."""
    out = tmp_path / (src + ".s")
    subprocess.run([B.HIPCC] + B.HIP_FLAGS + B.HIP_EXTRA.get(src, []) +
                   ["-I", B.CSRC, "-I", B.BUILD, "--cuda-device-only", "-S", os.path.join(B.CSRC, src), "-o", str(out)],
                   check=True, capture_output=True)
    found, name = {}, None
    for line in out.read_text().splitlines():
        m = re.match(r"(_Z\w+):", line)
        if m:
            name = m.group(1)
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name:
            found[name].append(line)
    return found


def test_reads_do_not_wait_for_the_loads_of_later_stages(tmp_path):
    functions = _functions("fp8.hip", tmp_path)
    for kernel in KERNELS:
        bodies = {n: body for n, body in functions.items() if kernel in n}
        assert bodies, kernel
        for name, body in bodies.items():
            assert any(re.match(r"\s*buffer_load\S*\s.*\blds\b", line) for line in body), f"no staged loads in {name}"
            assert not _stalls(body), (name, _stalls(body)[:3])
