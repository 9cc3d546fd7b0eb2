"""MI355X (gfx950) quantized linears: SVDQuant W4A4 (INT4 and MXFP4), INT8
tensorwise W8A8, W4A16, block-scaled FP8 with a mixture-of-experts layer.

The compute lives in the HIP/C++ shared library ``libsvdq.so`` built from
``csrc/`` (its C interface is ``include/svdq.h``). ``binding`` is a thin
ctypes layer with the same entry-point names that marshals numpy arrays,
torch tensors and streams into that interface; it never computes anything
itself and raises if the library is missing. ``workloads`` draws the seeded
synthetic inputs.
"""

from . import binding, workloads  # noqa: F401

__all__ = ["binding", "workloads"]
