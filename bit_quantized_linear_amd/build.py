"""Build libsvdq.so (HIP kernels for gfx950 + host C++) in-tree.

    python -m bit_quantized_linear_amd.build

HIP sources are compiled by hipcc for gfx950 only; host C++ sources by the
ROCm clang++. Objects go to ``_build/`` beside this file and the shared
library to ``libsvdq.so`` in this package directory. The GELU table of the
fused MLP epilogue is generated first (``gelu_table.py`` ->
``_build/gelu_table.h``). Beside the library, ``_tensors.<Python's tag>.so``: a
small module for this Python and torch, which the binding does without where it
is missing or was built for others.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig

if __package__:
    from . import gelu_table
else:  # run as a script
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from bit_quantized_linear_amd import gelu_table

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsvdq.so")
TENSORS = os.path.join(PKG, "_tensors" + importlib.machinery.EXTENSION_SUFFIXES[0])
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
ARCH = "gfx950"

HIPCC = os.path.join(ROCM, "bin", "hipcc")
CLANGXX = os.path.join(ROCM, "lib", "llvm", "bin", "clang++")

COMMON = ["-O3", "-fPIC", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
          "-ffp-contract=off", "-Wall", "-Wno-unused-function"]
# packed fp32 ops are disabled for all device code (v_pk_{add,mul,fma}_f32)
HIP_FLAGS = COMMON + [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang",
                      "-packed-fp32-ops"]
CXX_FLAGS = COMMON + ["-I", os.path.join(ROCM, "include"), "-D__HIP_PLATFORM_AMD__", "-pthread"]
# per-source extras: the W4A16 and block-scaled FP8 kernels feed every MFMA
# result straight into VALU arithmetic, so their MFMAs write VGPRs (no
# accumulation-register copies)
HIP_EXTRA = {src: ["-mllvm", "-amdgpu-mfma-vgpr-form"] for src in ("w4a16.hip", "fp8.hip", "fp8_moe.hip")}


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if p.returncode != 0:
        raise RuntimeError("build step failed:\n" + " ".join(cmd) + "\n" + p.stdout)
    return p.stdout


def _remove_tensors():
    """An earlier build's module may be another Python's or torch's."""
    for path in glob.glob(os.path.join(glob.escape(PKG), "_tensors*.so")):
        os.remove(path)


def _tensors_job():
    """How the module for tensors is built, or None without torch."""
    try:
        import torch
        from bit_quantized_linear_amd.binding import built_for
        from torch.utils.cpp_extension import include_paths
    except ImportError:
        return None
    include = [x for path in [*include_paths(), sysconfig.get_paths()["include"]] for x in ("-isystem", path)]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [CLANGXX, "-O2", "-fPIC", "-shared", "-std=c++17", "-fvisibility=hidden", "-Wall", *include,
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBUILT_FOR="{built_for(torch)}"',
            os.path.join(CSRC, "python", "tensors.cpp"), "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", TENSORS + ".tmp"]


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    _remove_tensors()
    gelu_table.write(os.path.join(BUILD, "gelu_table.h"))
    jobs = []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        jobs.append([HIPCC] + HIP_FLAGS + ["-I", BUILD] + HIP_EXTRA.get(os.path.basename(src), []) +
                    ["-c", src, "-o", obj])
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cpp"))):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        jobs.append([CLANGXX] + CXX_FLAGS + ["-c", src, "-o", obj])
    workers = max(1, min(len(jobs), int(os.environ.get("MAX_JOBS", "8"))))
    with cf.ThreadPoolExecutor(workers) as ex:
        tensors = _tensors_job()
        module = tensors and ex.submit(_run, tensors)
        outs = list(ex.map(_run, jobs))
        if module:
            try:
                outs.append(module.result())
                shutil.move(tensors[-1], TENSORS)
            except RuntimeError as e:
                print(f"{TENSORS} is left out: {e}", file=sys.stderr)
    if verbose:
        for o in outs:
            if o.strip():
                print(o)
    objs = [j[-1] for j in jobs]
    tmp = LIB + ".tmp"
    _run([HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs +
         ["-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-pthread"])
    shutil.move(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
