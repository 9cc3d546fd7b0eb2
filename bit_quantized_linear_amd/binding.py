"""ctypes binding of libsvdq.so (interface: include/svdq.h).

Argument marshalling only: host entry points take numpy arrays, device entry
points take torch tensors resident on the GPU (their data pointers are passed
through) and the current torch stream. Nothing here computes any step of the
linear; if the library is missing every call raises.
"""

from __future__ import annotations

import ctypes as C
import math
import os
import sys

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsvdq.so")

SVDQ_OK = 0
SVDQ_ERR_INVALID_ARGUMENT = 1
SVDQ_ERR_UNSUPPORTED_SHAPE = 2
SVDQ_ERR_UNSUPPORTED_DEVICE = 3
SVDQ_ERR_MISALIGNED = 4
SVDQ_ERR_NUMERICAL = 5
SVDQ_ERR_HIP = 6
SVDQ_BF16 = 0
SVDQ_F32 = 1
QFMT_INT4 = 0
QFMT_FP6 = 1
GROUP = 64
FP8_BLOCK = 128
FP8_MOE_MAX_TOKENS = 64
FP8_MOE_MAX_EXPERTS = 256
FP8_MOE_MAX_TOP_K = 16
ROPE_MAX_AXES = 4
ROPE_MAX_PAIRS = 256
KV8_PAGE = 64

_vp, _i, _f, _sz, _ll = C.c_void_p, C.c_int, C.c_float, C.c_size_t, C.c_int64

# name -> (restype, argtypes), mirroring include/svdq.h
SIGNATURES = {
    "svdq_status_string": (C.c_char_p, [_i]),
    "svdq_version": (_i, []),
    "svdq_qrow_bytes": (_sz, [_i, _i]),
    "svdq_repack_codes": (_i, [_vp, _i, _i, _i, _vp]),
    "svdq_check_device": (_i, [_i]),
    "svdq_prepare_weights": (_i, [_vp, _i, _i, _vp, _f, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]),
    "svdq_prepare_residual": (_i, [_vp, _i, _i, _vp, _vp, _vp, _i, _i, _vp, _vp]),
    "w8a8_prepare_weights": (_i, [_vp, _i, _i, _vp, _vp]),
    "svdq_channel_absmax": (_i, [_vp, _i, _i, _vp, _vp]),
    "svdq_act_workspace_bytes": (_sz, [_i, _i, _i]),
    "svdq_quantize_act": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "svdq_quantize_act_noalloc": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "svdq_w4a4_linear": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _vp]),
    "svdq_mlp_workspace_bytes": (_sz, [_i, _i, _i]),
    "svdq_w4a4_linear_gelu_quantize": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _i,
                                           _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "svdq_debug_gelu_bf16": (_i, [_vp, _vp, _i, _vp]),
    "w8a8_workspace_bytes": (_sz, [_i, _i]),
    "w8a8_linear": (_i, [_vp, _vp, _f, _vp, _i, _i, _i, _vp, _sz, _vp, _vp]),
    "svdq_mx_scale_ld": (_sz, [_i]),
    "svdq_mx_prepare_residual": (_i, [_vp, _i, _i, _vp, _vp, _vp, _i, _vp, _vp]),
    "svdq_mx_quantize_act": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "svdq_mx_linear": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _vp]),
    "w4a16_weight_bytes": (_sz, [_i, _i]),
    "w4a16_prepare_weights": (_i, [_vp, _i, _i, _i, _vp]),
    "w4a16_linear": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "svdq_fp8_prepare_weights": (_i, [_vp, _i, _i, _vp, _vp]),
    "svdq_fp8_quantize_act": (_i, [_vp, _i, _i, _vp, _vp, _vp]),
    "svdq_fp8_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp]),
    "svdq_fp8_workspace_bytes": (_sz, [_i, _i]),
    "svdq_fp8_linear": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _sz, _vp, _i, _vp]),
    "svdq_fp8_moe_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "svdq_fp8_moe_layer": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp, _vp]),
    "svdq_fp8_norm_quantize": (_i, [_vp, _vp, _vp, _f, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "svdq_rope": (_i, [_vp, _ll, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _ll, _vp]),
    "svdq_kv8_append": (_i, [_vp, _ll, _vp, _ll, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "svdq_kv8_attention_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "svdq_kv8_attention": (_i, [_vp, _ll, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _i, _vp,
                                _vp, _vp, _sz, _vp]),
    "svdq_debug_group_partials": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _vp, _vp]),
    "w8a8_debug_acc": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp]),
    "svdq_debug_set_arch_override": (_i, [C.c_char_p]),
    "svdq_debug_mfma_ops": (C.c_int64, [_i, _i, _i]),
    "svdq_debug_mfma_rate": (_i, [_i, _i, _i, _vp, _vp]),
}

_lib = None


class SvdqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")


def lib():
    """The loaded library; raises if it was not built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_quantized_linear_amd.build` (there is no CPU fallback)")
        # one HIP runtime per process: torch (the device memory and stream
        # plumbing) is loaded first, so that this library binds to the HIP
        # runtime torch already uses instead of loading a second one beside it
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        handle = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().svdq_status_string(status).decode()


def _check(fn, status):
    if status != SVDQ_OK:
        raise SvdqError(fn, status)


def _np_ptr(a, dtype):
    if a is None:
        return None
    if a.dtype != np.dtype(dtype) or not a.flags["C_CONTIGUOUS"]:
        raise TypeError(f"expected a C-contiguous {np.dtype(dtype)} array")
    return a.ctypes.data


_device_of = None


def _current_device():
    global _device_of
    if _device_of is None:
        import torch

        device = torch.cuda.current_device()  # starts torch's side of the device, too
        # once that is up, the number without the check for it (0.2 us a call)
        _device_of = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        return device
    return _device_of()


def _dev_ptr(t, itemsize=None, nbytes=0, name="tensor", device=None, formats=None):
    """Device pointer of a torch tensor (None -> NULL).

    The library receives raw pointers and sizes, so the extent a call will
    touch is checked here, before anything is launched: the tensor must be a
    contiguous GPU tensor on the current device (`device`, looked up when not
    given) holding at least `nbytes` bytes, of one of the types `formats` where
    they are given. A violation raises TypeError (kind, layout, element size,
    type, device) or ValueError (too small)."""
    if t is None:
        return None
    dtype = None if formats is None else getattr(t, "dtype", None)
    # a tensor with a type to look at tells its device by number at half the cost
    index = (t.device.index if t.is_cuda else -1) if dtype is None else t.get_device()
    if index < 0:
        raise TypeError(f"{name}: device entry points take GPU tensors")
    if not t.is_contiguous():
        raise TypeError(f"{name}: tensors must be contiguous")
    if dtype is None:
        size = t.element_size()
        if itemsize is not None and size != itemsize:
            raise TypeError(f"{name}: expected {itemsize}-byte elements, got {size}")
    elif dtype in formats:  # each of `itemsize` bytes
        size = itemsize
    else:
        raise TypeError(f"{name}: {dtype}, the call takes {', '.join(sorted(map(str, formats)))}")
    dev = _current_device() if device is None else device
    if index != dev:
        raise TypeError(f"{name} is on cuda:{index}, the current device is cuda:{dev}")
    have = t.numel() * size
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, the call needs at least {nbytes}")
    return t.data_ptr()


def _shape2(t, name):
    if t is None or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D tensor")
    rows, columns = t.shape
    return int(rows), int(columns)


_raw_stream = None


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    global _raw_stream
    if _raw_stream is None:
        import torch

        # the current stream's handle, where torch has it without a Stream
        # object (3 us a call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = (lambda: raw(_current_device())) if raw else (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def _forget_device():
    global _device_of, _raw_stream
    _device_of = _raw_stream = None


# a forked child cannot use its parent's GPU: it asks torch anew, whose own
# check says so
os.register_at_fork(after_in_child=_forget_device)


# ------------------------------------------------------------------ info --

def svdq_version() -> int:
    return lib().svdq_version()


def svdq_qrow_bytes(K: int, qfmt: int) -> int:
    return int(lib().svdq_qrow_bytes(K, qfmt))


def svdq_check_device(device: int = 0) -> int:
    return lib().svdq_check_device(device)


def svdq_debug_set_arch_override(arch):
    return lib().svdq_debug_set_arch_override(None if arch is None else arch.encode())


# ------------------------------------------------------------------ host --

def svdq_prepare_weights(W_bits, act_absmax, rank, alpha=0.5, group=GROUP, want_sigma=False):
    """Host preparation. W_bits: uint16 [K, N] bf16 bits; act_absmax: float32 [K]."""
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    act_absmax = np.ascontiguousarray(act_absmax, dtype=np.float32)
    K, N = W_bits.shape
    out = {
        "s": np.empty(K, np.float32),
        "l1t": np.empty((rank, K), np.uint16),
        "l2t": np.empty((N, rank), np.uint16),
        "qw": np.empty((N, K // 2), np.uint8),
        "sw": np.empty((max(K // group, 0), N), np.float32),
        "sigma": np.empty(rank, np.float64),
    }
    st = lib().svdq_prepare_weights(
        _np_ptr(W_bits, np.uint16), K, N, _np_ptr(act_absmax, np.float32), float(alpha), rank, group,
        out["s"].ctypes.data, out["l1t"].ctypes.data if rank else None,
        out["l2t"].ctypes.data if rank else None, out["qw"].ctypes.data, out["sw"].ctypes.data,
        out["sigma"].ctypes.data if rank else None)
    _check("svdq_prepare_weights", st)
    if not want_sigma:
        out.pop("sigma")
    return out


def svdq_prepare_residual(W_bits, smooth, l1t, l2t, group=GROUP):
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    smooth = np.ascontiguousarray(smooth, dtype=np.float32)
    l1t = np.ascontiguousarray(l1t, dtype=np.uint16)
    l2t = np.ascontiguousarray(l2t, dtype=np.uint16)
    K, N = W_bits.shape
    rank = l1t.shape[0]
    qw = np.empty((N, K // 2), np.uint8)
    sw = np.empty((K // group, N), np.float32)
    st = lib().svdq_prepare_residual(_np_ptr(W_bits, np.uint16), K, N, _np_ptr(smooth, np.float32),
                                     l1t.ctypes.data if rank else None, l2t.ctypes.data if rank else None,
                                     rank, group, qw.ctypes.data, sw.ctypes.data)
    _check("svdq_prepare_residual", st)
    return {"qw": qw, "sw": sw}


def svdq_repack_codes(q, K, qfmt):
    """Canonical INT4 rows [rows, K/2] -> container `qfmt` rows."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    rows = q.shape[0]
    out = np.empty((rows, svdq_qrow_bytes(K, qfmt)), np.uint8)
    st = lib().svdq_repack_codes(q.ctypes.data if rows else None, rows, K, qfmt,
                                 out.ctypes.data if rows else None)
    _check("svdq_repack_codes", st)
    return out


def w8a8_prepare_weights(W_bits):
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    K, N = W_bits.shape
    qw = np.empty((N, K), np.int8)
    sw = np.zeros(1, np.float32)
    st = lib().w8a8_prepare_weights(_np_ptr(W_bits, np.uint16), K, N, qw.ctypes.data, sw.ctypes.data)
    _check("w8a8_prepare_weights", st)
    return qw, float(sw[0])


def svdq_mx_scale_ld(rows) -> int:
    """Row stride (bytes) of an MXFP4 scale matrix [K/32, ld] for `rows` rows."""
    return int(lib().svdq_mx_scale_ld(rows))


def svdq_mx_prepare_residual(W_bits, smooth, l1t, l2t):
    """MXFP4 residual of a bf16 weight W [K, N] given smoothing and factors:
    codes (MX container, N rows of K/2 bytes) and E8M0 scales [K/32, ld(N)]."""
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    smooth = np.ascontiguousarray(smooth, dtype=np.float32)
    l1t = np.ascontiguousarray(l1t, dtype=np.uint16)
    l2t = np.ascontiguousarray(l2t, dtype=np.uint16)
    K, N = W_bits.shape
    rank = l1t.shape[0]
    qw = np.empty((N, K // 2), np.uint8)
    uw = np.zeros((max(K // 32, 0), svdq_mx_scale_ld(N)), np.uint8)
    st = lib().svdq_mx_prepare_residual(_np_ptr(W_bits, np.uint16), K, N, _np_ptr(smooth, np.float32),
                                        l1t.ctypes.data if rank else None, l2t.ctypes.data if rank else None,
                                        rank, qw.ctypes.data, uw.ctypes.data)
    _check("svdq_mx_prepare_residual", st)
    return {"qw": qw, "uw": uw}


def w4a16_weight_bytes(K, N) -> int:
    return int(lib().w4a16_weight_bytes(K, N))


def w4a16_prepare_weights(W_bits, group=GROUP):
    """W4A16 weight container (uint8, w4a16_weight_bytes(K, N) bytes) of a
    bf16 weight W [K, N]."""
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    K, N = W_bits.shape
    nbytes = w4a16_weight_bytes(K, N)
    out = np.empty(max(nbytes, 1), np.uint8)
    st = lib().w4a16_prepare_weights(_np_ptr(W_bits, np.uint16), K, N, group, out.ctypes.data)
    _check("w4a16_prepare_weights", st)
    return out[:nbytes]


def fp8_blocks(n) -> int:
    """Blocks of 128 that cover n features."""
    return -(-n // FP8_BLOCK)


def svdq_fp8_prepare_weights(W_bits):
    """Block-scaled FP8 weight of a bf16 weight W [K, N]: E4M3 codes (uint8,
    [N, K]) and scales (float32, [ceil(N/128), ceil(K/128)])."""
    W_bits = np.ascontiguousarray(W_bits, dtype=np.uint16)
    K, N = W_bits.shape
    qw = np.empty((N, K), np.uint8)
    sw = np.empty((fp8_blocks(N), fp8_blocks(K)), np.float32)
    st = lib().svdq_fp8_prepare_weights(_np_ptr(W_bits, np.uint16), K, N, qw.ctypes.data, sw.ctypes.data)
    _check("svdq_fp8_prepare_weights", st)
    return qw, sw


# ---------------------------------------------------------------- device --
#
# Every wrapper checks, before calling into the library, that each tensor
# covers the extent the call will read or write for the sizes it passes (the
# library sees only pointers and sizes), and that each tensor is on the
# current device.

def svdq_channel_absmax(X, absmax, stream=None):
    M, K = _shape2(X, "X")
    dev = _current_device()
    st = lib().svdq_channel_absmax(_dev_ptr(X, 2, M * K * 2, "X", dev), M, K,
                                   _dev_ptr(absmax, 4, K * 4, "absmax", dev), _stream(stream))
    _check("svdq_channel_absmax", st)


def svdq_act_workspace_bytes(M, K, rank) -> int:
    return int(lib().svdq_act_workspace_bytes(M, K, rank))


def _ws(workspace, dev):
    if workspace is None:
        return None, 0
    return _dev_ptr(workspace, None, 0, "workspace", dev), workspace.numel() * workspace.element_size()


def svdq_quantize_act(X, smooth, l1t, qx, sx, T, rank, group=GROUP, qfmt=QFMT_INT4, workspace=None,
                      stream=None):
    M, K = _shape2(X, "X")
    dev = _current_device()
    G = K // group if group > 0 else 0
    wp, wb = _ws(workspace, dev)
    st = lib().svdq_quantize_act(
        _dev_ptr(X, 2, M * K * 2, "X", dev), _dev_ptr(smooth, 4, K * 4, "smooth", dev),
        _dev_ptr(l1t, 2, rank * K * 2, "l1t", dev), M, K, rank, group, qfmt,
        _dev_ptr(qx, 1, M * svdq_qrow_bytes(K, qfmt), "qx", dev), _dev_ptr(sx, 4, G * M * 4, "sx", dev),
        _dev_ptr(T, 2, M * rank * 2, "T", dev), wp, wb, _stream(stream))
    _check("svdq_quantize_act", st)


def svdq_quantize_act_noalloc(X, smooth, l1t, qx, sx, T, rank, group=GROUP, qfmt=QFMT_INT4, stream=None):
    """svdq_quantize_act with the library's fixed device scratch instead of a
    caller workspace (allocates nothing)."""
    M, K = _shape2(X, "X")
    dev = _current_device()
    G = K // group if group > 0 else 0
    st = lib().svdq_quantize_act_noalloc(
        _dev_ptr(X, 2, M * K * 2, "X", dev), _dev_ptr(smooth, 4, K * 4, "smooth", dev),
        _dev_ptr(l1t, 2, rank * K * 2, "l1t", dev), M, K, rank, group, qfmt,
        _dev_ptr(qx, 1, M * svdq_qrow_bytes(K, qfmt), "qx", dev), _dev_ptr(sx, 4, G * M * 4, "sx", dev),
        _dev_ptr(T, 2, M * rank * 2, "T", dev), _stream(stream))
    _check("svdq_quantize_act_noalloc", st)


def _linear_operands(qx, sx, T, qw, sw, l2t, bias, M, N, K, rank, group, qfmt, dev):
    """Checked pointers of the W4A4 GEMM's inputs (shared by the linear and
    the fused MLP entry point)."""
    R = svdq_qrow_bytes(K, qfmt)
    G = K // group if group > 0 else 0
    return (_dev_ptr(qx, 1, M * R, "qx", dev), _dev_ptr(sx, 4, G * M * 4, "sx", dev),
            _dev_ptr(T, 2, M * rank * 2, "T", dev), _dev_ptr(qw, 1, N * R, "qw", dev),
            _dev_ptr(sw, 4, G * N * 4, "sw", dev), _dev_ptr(l2t, 2, N * rank * 2, "l2t", dev),
            _dev_ptr(bias, 2, N * 2, "bias", dev))


def svdq_w4a4_linear(qx, sx, T, qw, sw, l2t, bias, Y, M, N, K, rank, group=GROUP, qfmt=QFMT_INT4,
                     stream=None):
    dev = _current_device()
    y_dtype = SVDQ_F32 if Y.element_size() == 4 else SVDQ_BF16
    ins = _linear_operands(qx, sx, T, qw, sw, l2t, bias, M, N, K, rank, group, qfmt, dev)
    st = lib().svdq_w4a4_linear(*ins, M, N, K, rank, group, qfmt,
                                _dev_ptr(Y, None, M * N * Y.element_size(), "Y", dev), y_dtype, _stream(stream))
    _check("svdq_w4a4_linear", st)


def svdq_mlp_workspace_bytes(M, N, rank_down) -> int:
    return int(lib().svdq_mlp_workspace_bytes(M, N, rank_down))


def svdq_w4a4_linear_gelu_quantize(qx, sx, T, qw, sw, l2t, bias, M, N, K, rank, smooth_down, l1t_down,
                                   rank_down, qx_down, sx_down, T_down, Y_up=None, workspace=None,
                                   group=GROUP, stream=None):
    dev = _current_device()
    ins = _linear_operands(qx, sx, T, qw, sw, l2t, bias, M, N, K, rank, group, QFMT_FP6, dev)
    Gd = N // group if group > 0 else 0
    ws_need = svdq_mlp_workspace_bytes(M, N, rank_down)
    st = lib().svdq_w4a4_linear_gelu_quantize(
        *ins, M, N, K, rank, group, _dev_ptr(smooth_down, 4, N * 4, "smooth_down", dev),
        _dev_ptr(l1t_down, 2, rank_down * N * 2, "l1t_down", dev), rank_down,
        _dev_ptr(qx_down, 1, M * svdq_qrow_bytes(N, QFMT_FP6), "qx_down", dev),
        _dev_ptr(sx_down, 4, Gd * M * 4, "sx_down", dev), _dev_ptr(T_down, 2, M * rank_down * 2, "T_down", dev),
        _dev_ptr(Y_up, 2, M * N * 2, "Y_up", dev), _dev_ptr(workspace, None, ws_need, "workspace", dev),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(stream))
    _check("svdq_w4a4_linear_gelu_quantize", st)


def svdq_debug_gelu_bf16(y, g, stream=None):
    dev = _current_device()
    n = y.numel()
    st = lib().svdq_debug_gelu_bf16(_dev_ptr(y, 2, n * 2, "y", dev), _dev_ptr(g, 2, n * 2, "g", dev), n,
                                    _stream(stream))
    _check("svdq_debug_gelu_bf16", st)


def w8a8_workspace_bytes(M, K) -> int:
    return int(lib().w8a8_workspace_bytes(M, K))


def w8a8_linear(X, qw, sw, bias, workspace, Y, stream=None):
    M, K = _shape2(X, "X")
    N, Kw = _shape2(qw, "qw")
    if Kw != K:
        raise ValueError(f"qw has {Kw} columns, X has K = {K}")
    dev = _current_device()
    ws_need = w8a8_workspace_bytes(M, K)
    st = lib().w8a8_linear(_dev_ptr(X, 2, M * K * 2, "X", dev), _dev_ptr(qw, 1, N * K, "qw", dev), float(sw),
                           _dev_ptr(bias, 2, N * 2, "bias", dev), M, N, K,
                           _dev_ptr(workspace, None, ws_need, "workspace", dev),
                           workspace.numel() * workspace.element_size(),
                           _dev_ptr(Y, 2, M * N * 2, "Y", dev), _stream(stream))
    _check("w8a8_linear", st)


def svdq_mx_quantize_act(X, smooth, l1t, qx, ux, T, rank, workspace=None, stream=None):
    M, K = _shape2(X, "X")
    dev = _current_device()
    wp, wb = _ws(workspace, dev)
    st = lib().svdq_mx_quantize_act(
        _dev_ptr(X, 2, M * K * 2, "X", dev), _dev_ptr(smooth, 4, K * 4, "smooth", dev),
        _dev_ptr(l1t, 2, rank * K * 2, "l1t", dev), M, K, rank, _dev_ptr(qx, 1, M * (K // 2), "qx", dev),
        _dev_ptr(ux, 1, (K // 32) * svdq_mx_scale_ld(M), "ux", dev), _dev_ptr(T, 2, M * rank * 2, "T", dev),
        wp, wb, _stream(stream))
    _check("svdq_mx_quantize_act", st)


def svdq_mx_linear(qx, ux, T, qw, uw, l2t, bias, Y, M, N, K, rank, stream=None):
    dev = _current_device()
    y_dtype = SVDQ_F32 if Y.element_size() == 4 else SVDQ_BF16
    st = lib().svdq_mx_linear(
        _dev_ptr(qx, 1, M * (K // 2), "qx", dev), _dev_ptr(ux, 1, (K // 32) * svdq_mx_scale_ld(M), "ux", dev),
        _dev_ptr(T, 2, M * rank * 2, "T", dev), _dev_ptr(qw, 1, N * (K // 2), "qw", dev),
        _dev_ptr(uw, 1, (K // 32) * svdq_mx_scale_ld(N), "uw", dev), _dev_ptr(l2t, 2, N * rank * 2, "l2t", dev),
        _dev_ptr(bias, 2, N * 2, "bias", dev), M, N, K, rank,
        _dev_ptr(Y, None, M * N * Y.element_size(), "Y", dev), y_dtype, _stream(stream))
    _check("svdq_mx_linear", st)


def w4a16_linear(X, packed, bias, Y, N, group=GROUP, stream=None):
    """Y [M, N] bf16 = X [M, K] bf16 times the W4A16 container `packed`."""
    M, K = _shape2(X, "X")
    dev = _current_device()
    st = lib().w4a16_linear(_dev_ptr(X, 2, M * K * 2, "X", dev),
                            _dev_ptr(packed, 1, w4a16_weight_bytes(K, N), "packed", dev),
                            _dev_ptr(bias, 2, N * 2, "bias", dev), M, N, K, group,
                            _dev_ptr(Y, 2, M * N * 2, "Y", dev), _stream(stream))
    _check("w4a16_linear", st)


_fp8_types = None


def _fp8_formats():
    """The torch types of E4M3 codes, bf16, fp32 and int32 numbers at the
    block-scaled FP8 entry points. Integers of the width hold the bits, as
    elsewhere; another format of the same width (float16, e4m3fnuz, e5m2) would
    be read as something else."""
    global _fp8_types
    if _fp8_types is None:
        import torch as t

        _fp8_types = (frozenset((t.float8_e4m3fn, t.uint8, t.int8)), frozenset((t.bfloat16, t.int16, t.uint16)),
                      frozenset((t.float32,)), frozenset((t.int32, t.uint32)))
    return _fp8_types


def _fp8_scales(t, shape, name, dev, f32):
    """Pointer of fp32 scales: a tensor with as many dimensions as `shape` has its
    rows, too (the same bytes in another order would pass by their number)."""
    nbytes = 0
    if t is not None and t.shape != shape:
        if t.dim() == len(shape) and tuple(t.shape[1:]) != shape[1:]:
            raise ValueError(f"{name} is {list(t.shape)}, the call takes {list(shape)}")
        nbytes = 4 * math.prod(shape)
    return _dev_ptr(t, 4, nbytes, name, dev, f32)


def svdq_fp8_quantize_act(X, qx, sx, stream=None):
    """E4M3 codes qx [M, K] (1-byte elements) and scales sx [ceil(K/128), M] of X [M, K] bf16."""
    M, K = _shape2(X, "X")
    dev = _current_device()
    e4m3, bf16, f32, _ = _fp8_formats()
    st = lib().svdq_fp8_quantize_act(_dev_ptr(X, 2, M * K * 2, "X", dev, bf16), M, K,
                                     _dev_ptr(qx, 1, M * K, "qx", dev, e4m3),
                                     _fp8_scales(sx, (fp8_blocks(K), M), "sx", dev, f32), _stream(stream))
    _check("svdq_fp8_quantize_act", st)


def _fp8_weight(qw, sw, K, dev, e4m3, f32):
    N, Kw = _shape2(qw, "qw")
    if Kw != K:
        raise ValueError(f"qw has {Kw} columns, X has K = {K}")
    qwp = _dev_ptr(qw, 1, N * K, "qw", dev, e4m3)
    return N, qwp, _fp8_scales(sw, (fp8_blocks(N), fp8_blocks(K)), "sw", dev, f32)


def _fp8_out(Y, M, N, dev, bf16, f32):
    """Pointer and type code of the output Y [M, N], whose element size says which type it is."""
    if Y is None:
        raise TypeError("Y: a tensor is needed, its element size gives the output's type")
    if Y.element_size() == 4:
        return _dev_ptr(Y, 4, M * N * 4, "Y", dev, f32), SVDQ_F32
    return _dev_ptr(Y, 2, M * N * 2, "Y", dev, bf16), SVDQ_BF16


def svdq_fp8_gemm(qx, sx, qw, sw, bias, Y, stream=None):
    """Y [M, N] (bf16 or fp32, by its element size) of quantized activations
    qx [M, K], sx and the block-scaled weight qw [N, K], sw."""
    M, K = _shape2(qx, "qx")
    dev = _current_device()
    e4m3, bf16, f32, _ = _fp8_formats()
    N, qwp, swp = _fp8_weight(qw, sw, K, dev, e4m3, f32)
    Yp, out = _fp8_out(Y, M, N, dev, bf16, f32)
    st = lib().svdq_fp8_gemm(_dev_ptr(qx, 1, M * K, "qx", dev, e4m3),
                             _fp8_scales(sx, (fp8_blocks(K), M), "sx", dev, f32), qwp, swp,
                             _dev_ptr(bias, 2, N * 2, "bias", dev, bf16), M, N, K, Yp, out, _stream(stream))
    _check("svdq_fp8_gemm", st)


def svdq_fp8_workspace_bytes(M, K) -> int:
    return int(lib().svdq_fp8_workspace_bytes(M, K))


def svdq_fp8_linear(X, qw, sw, bias, workspace, Y, stream=None):
    """Y [M, N] (bf16 or fp32, by its element size) = X [M, K] bf16 quantized
    on the way, times the block-scaled weight qw [N, K], sw, plus bias."""
    M, K = _shape2(X, "X")
    dev = _current_device()
    e4m3, bf16, f32, _ = _fp8_formats()
    N, qwp, swp = _fp8_weight(qw, sw, K, dev, e4m3, f32)
    Yp, out = _fp8_out(Y, M, N, dev, bf16, f32)
    ws_need = svdq_fp8_workspace_bytes(M, K)
    st = lib().svdq_fp8_linear(_dev_ptr(X, 2, M * K * 2, "X", dev, bf16), qwp, swp,
                               _dev_ptr(bias, 2, N * 2, "bias", dev, bf16), M, N, K,
                               _dev_ptr(workspace, None, ws_need, "workspace", dev),
                               0 if workspace is None else ws_need, Yp, out, _stream(stream))
    _check("svdq_fp8_linear", st)


def svdq_fp8_moe_workspace_bytes(T, I, E, top_k) -> int:  # noqa: E741
    return int(lib().svdq_fp8_moe_workspace_bytes(T, I, E, top_k))


def svdq_fp8_moe_layer(X, wr, w13, s13, w2, s2, Y, idx, gate, workspace, top_k=None, renormalize=True, stream=None):
    """Mixture-of-experts layer of a few tokens: Y [T, H] bf16 from X [T, H],
    the router wr [E, H] (bf16) and the experts' block-scaled FP8 weights
    w13 [E, 2, I, H], s13 and w2 [E, H, I], s2. idx [T, top_k] int32 and
    gate [T, top_k] fp32 take the choices and their weights; each may be None
    (top_k is given then, if both are)."""
    T, H = _shape2(X, "X")
    E, Hr = _shape2(wr, "wr")
    if w13 is None or w13.dim() != 4 or w2 is None or w2.dim() != 3:
        raise TypeError("w13 must be a 4-D and w2 a 3-D tensor")
    shape13, shape2 = w13.shape, w2.shape
    I = int(shape13[2])  # noqa: E741
    if Hr != H or shape13 != (E, 2, I, H) or shape2 != (E, H, I):
        raise ValueError(f"X [{T}, {H}], wr [{E}, {Hr}], w13 {list(shape13)} and w2 {list(shape2)} do not fit")
    for name, t in (("idx", idx), ("gate", gate)):
        if t is not None:
            rows, k = _shape2(t, name)
            if top_k is None:
                top_k = k
            if rows != T or k != top_k:
                raise ValueError(f"{name} is [{rows}, {k}], the call writes [{T}, {top_k}]")
    if top_k is None:
        raise ValueError("top_k is needed where neither idx nor gate is given")
    dev = _current_device()
    gi, gh = fp8_blocks(I), fp8_blocks(H)
    need = svdq_fp8_moe_workspace_bytes(T, I, E, top_k)
    e4m3, bf16, f32, i32 = _fp8_formats()
    st = lib().svdq_fp8_moe_layer(
        _dev_ptr(X, 2, T * H * 2, "X", dev, bf16), _dev_ptr(wr, 2, E * H * 2, "wr", dev, bf16),
        _dev_ptr(w13, 1, E * 2 * I * H, "w13", dev, e4m3), _fp8_scales(s13, (E, 2, gi, gh), "s13", dev, f32),
        _dev_ptr(w2, 1, E * H * I, "w2", dev, e4m3), _fp8_scales(s2, (E, gh, gi), "s2", dev, f32), T, H, I, E,
        top_k, 1 if renormalize else 0, _dev_ptr(idx, 4, T * top_k * 4, "idx", dev, i32),
        _dev_ptr(gate, 4, T * top_k * 4, "gate", dev, f32), _dev_ptr(workspace, None, need, "workspace", dev),
        0 if workspace is None else need, _dev_ptr(Y, 2, T * H * 2, "Y", dev, bf16), _stream(stream))
    _check("svdq_fp8_moe_layer", st)


_quick_calls = None
_ANY_KIND = 2 ** 64 - 1


def built_for(torch):
    """The Python and torch whose structures `_tensors` reads."""
    return f"{sys.implementation.cache_tag}, torch {torch.__version__} {torch.version.git_version}"


def _quick():
    """pointers and heads of `_tensors`, which look at all tensors of a call at once,
    and its names for E4M3 codes, bf16, fp32, int32 and fp64 numbers; empty where it
    was not built, or not for this Python and torch. What they refuse is looked at
    again below, for the error that fits."""
    global _quick_calls
    if _quick_calls is None:
        _quick_calls = ()
        try:
            import torch as t

            from . import _tensors as m

            if getattr(m, "built_for", None) == built_for(t):
                _quick_calls = (m.pointers, m.heads, *(m.kind(*f) for f in (*_fp8_formats(), (t.float64,))))
        except ImportError:
            pass
    return _quick_calls


def _ptr(t, nbytes, name, dev, formats):
    """As _dev_ptr, for the entry points with many tensors: one look at each of a
    tensor's properties, and the reasons only where one is not as it must be."""
    if t is None:
        return None
    if t.dtype in formats and t.get_device() == dev and t.is_contiguous() and t.nbytes >= nbytes:
        return t.data_ptr()
    return _dev_ptr(t, t.element_size(), nbytes, name, dev, formats)


def _shaped_ptr(t, shape, name, dev, formats):
    """The same for a tensor that has exactly the shape."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} is {list(t.shape)}, the call takes {list(shape)}")
    if t.dtype in formats and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _dev_ptr(t, t.element_size(), 0, name, dev, formats)


def svdq_fp8_norm_quantize(X, residual, weight, eps, total, Y, qx, sx, stream=None):
    """Root-mean-square norm of X [M, K] (+ residual), bf16, with weights [K]:
    total = the sum (bf16; may be residual or X itself), Y = the norm in bf16, qx
    [M, K] and sx [ceil(K/128), M] = its E4M3 codes and scales, as
    svdq_fp8_quantize_act writes them. residual, total, Y, and qx with sx may be
    None, but not both Y and qx."""
    M, K = _shape2(X, "X")
    dev = _current_device()
    n = M * K * 2
    p, quick = None, _quick()
    if quick:
        pointers, _, e4m3, bf16, f32, _, _ = quick
        p = pointers(dev, X, bf16, n, residual, bf16, n, weight, bf16, K * 2, total, bf16, n, Y, bf16, n, qx, e4m3, M * K,
                     sx, f32, (fp8_blocks(K), M))
    if p is None:
        e4m3, bf16, f32, _ = _fp8_formats()
        p = (_ptr(X, n, "X", dev, bf16), _ptr(residual, n, "residual", dev, bf16), _ptr(weight, K * 2, "weight", dev, bf16),
             _ptr(total, n, "total", dev, bf16), _ptr(Y, n, "Y", dev, bf16), _ptr(qx, M * K, "qx", dev, e4m3),
             None if sx is None else _fp8_scales(sx, (fp8_blocks(K), M), "sx", dev, f32))
    st = lib().svdq_fp8_norm_quantize(p[0], p[1], p[2], eps, M, K, p[3], p[4], p[5], p[6], _stream(stream))
    _check("svdq_fp8_norm_quantize", st)


def _dev_heads(t, name, dev):
    """Pointer, stride between tokens and T, H, D of heads [T, H, D] in bf16, whose
    rows may be parts of wider ones (a projection's output)."""
    quick = _quick()
    if quick:
        seen = quick[1](dev, quick[3], t)
        if seen is not None:
            return seen
    bf16 = _fp8_formats()[1]
    if t is None or t.dim() != 3:
        raise TypeError(f"{name} must be a 3-D tensor")
    if t.dtype not in bf16:
        raise TypeError(f"{name}: {t.dtype}, the call takes {', '.join(sorted(map(str, bf16)))}")
    index = t.get_device()
    if index != dev:
        if index < 0:
            raise TypeError(f"{name}: device entry points take GPU tensors")
        raise TypeError(f"{name} is on cuda:{index}, the current device is cuda:{dev}")
    T, H, D = t.shape
    row, head, one = t.stride()
    width = H * D
    if T <= 1 or width == 0:  # there is no next row
        row = -(-width // 8) * 8
    if row < width or (one != 1 and D > 1) or (head != D and H > 1):
        raise TypeError(f"{name}: the heads of a token must be contiguous, and tokens apart")
    return t.data_ptr(), row, T, H, D


_f64_types = None


def _f64_format():
    global _f64_types
    if _f64_types is None:
        import torch as t

        _f64_types = frozenset((t.float64,))
    return _f64_types


def svdq_rope(X, positions, freqs, sections, Y, interleaved=False, stream=None):
    """Y = X [T, H, D] (bf16, rows may be parts of wider ones) turned by rotary
    positions: positions [T, axes] int32, freqs [R / 2] fp64, sections: the pairs of
    each axis, R / 2 in all. Y may be X."""
    dev = _current_device()
    xp, xs, *shape = x = _dev_heads(X, "X", dev)
    yp, ys, *out = x if Y is X else _dev_heads(Y, "Y", dev)
    if out != shape:
        raise ValueError(f"Y is {out}, the call writes {shape}")
    T, H, D = shape
    axes = len(sections)
    if positions is None:
        raise TypeError(f"positions must be a tensor [{T}, {axes}]")
    p, quick = None, _quick()
    if quick:
        pointers, _, _, _, _, i32, f64 = quick
        p = pointers(dev, positions, i32, (T, axes), freqs, f64, 8 * sum(sections))
    if p is None:
        p = (_shaped_ptr(positions, (T, axes), "positions", dev, _fp8_formats()[3]),
             _ptr(freqs, 8 * sum(sections), "freqs", dev, _f64_format()))
    st = lib().svdq_rope(xp, xs, p[0], p[1], (_i * axes)(*sections), axes, 1 if interleaved else 0, T, H, D, yp, ys,
                         _stream(stream))
    _check("svdq_rope", st)


def _kv8_tensors(kc, ks, vc, vs, starts, lengths, table, Hk, D, dev):
    """Checked pointers of the 8-bit cache and of a batch, as the library takes them:
    kc, ks, vc, vs, starts, lengths, table; and the batch's sequences, the table's
    width and the cache's pages."""
    if kc is None or vc is None or ks is None or vs is None or kc.dim() != 4:
        raise TypeError("kc and vc must be 4-D tensors, ks and vs their scales")
    P = kc.shape[0]
    B, max_pages = _shape2(table, "table")
    keys, values, scales = (P, Hk, KV8_PAGE, D), (P, Hk, D, KV8_PAGE), (P, Hk)
    p, quick = None, _quick()
    if quick:
        pointers, _, e4m3, _, f32, i32, _ = quick
        p = pointers(dev, kc, e4m3, keys, ks, f32, scales, vc, e4m3, values, vs, f32, scales, starts, i32, 4 * (B + 1),
                     lengths, i32, 4 * B, table, i32, 0)
    if p is None:
        e4m3, _, f32, i32 = _fp8_formats()
        p = (_shaped_ptr(kc, keys, "kc", dev, e4m3), _shaped_ptr(ks, scales, "ks", dev, f32),
             _shaped_ptr(vc, values, "vc", dev, e4m3), _shaped_ptr(vs, scales, "vs", dev, f32),
             _ptr(starts, 4 * (B + 1), "starts", dev, i32), _ptr(lengths, 4 * B, "lengths", dev, i32),
             _ptr(table, 0, "table", dev, i32))
    return p, B, max_pages, P


def svdq_kv8_append(K, V, starts, lengths, table, kc, ks, vc, vs, stream=None):
    """New keys and values K, V [T, Hk, D] (bf16, rows may be parts of wider ones)
    into the 8-bit cache kc [pages, Hk, 64, D], ks [pages, Hk], vc [pages, Hk, D, 64],
    vs [pages, Hk]; starts [B + 1], lengths [B] and table [B, max_pages] int32 say
    which rows are whose and where they go."""
    dev = _current_device()
    kp, kst, *shape = _dev_heads(K, "K", dev)
    vp, vst, *other = _dev_heads(V, "V", dev)
    if other != shape:
        raise ValueError(f"V is {other}, K {shape}")
    T, Hk, D = shape
    p, B, max_pages, P = _kv8_tensors(kc, ks, vc, vs, starts, lengths, table, Hk, D, dev)
    st = lib().svdq_kv8_append(kp, kst, vp, vst, p[4], p[5], p[6], T, B, max_pages, P, Hk, D, p[0], p[1], p[2], p[3],
                               _stream(stream))
    _check("svdq_kv8_append", st)


def svdq_kv8_attention_workspace_bytes(T, B, max_pages, Hq, Hk, D) -> int:
    return int(lib().svdq_kv8_attention_workspace_bytes(T, B, max_pages, Hq, Hk, D))


def svdq_kv8_attention(Q, kc, ks, vc, vs, starts, lengths, table, scale, O, lse=None, workspace=None,  # noqa: E741
                       causal=True, window=0, stream=None):
    """O [T, Hq, D] bf16 = attention of the newest tokens' queries Q [T, Hq, D] (bf16,
    rows may be parts of wider ones) over the 8-bit cache; lse [T, Hq] fp32 takes
    the logarithms of the weights' sums. The library refuses a workspace (any
    contiguous GPU tensor) of too few bytes. The rest as svdq_kv8_append."""
    dev = _current_device()
    qp, qst, T, Hq, D = _dev_heads(Q, "Q", dev)
    Hk = kc.shape[1] if kc is not None and kc.dim() == 4 else 0
    p, B, max_pages, P = _kv8_tensors(kc, ks, vc, vs, starts, lengths, table, Hk, D, dev)
    out, quick = None, _quick()
    if quick:
        pointers, _, _, bf16, f32, _, _ = quick
        out = pointers(dev, O, bf16, T * Hq * D * 2, lse, f32, (T, Hq), workspace, _ANY_KIND, 0)
    if out is None:
        _, bf16, f32, _ = _fp8_formats()
        out = (_ptr(O, T * Hq * D * 2, "O", dev, bf16), _shaped_ptr(lse, (T, Hq), "lse", dev, f32), _ws(workspace, dev)[0])
    st = lib().svdq_kv8_attention(qp, qst, *p, T, B, max_pages, P, Hq, Hk, D, scale, 1 if causal else 0, window, out[0],
                                  out[1], out[2], 0 if workspace is None else workspace.nbytes, _stream(stream))
    _check("svdq_kv8_attention", st)


def svdq_debug_group_partials(qx, qw, P, M, N, K, group=GROUP, qfmt=QFMT_INT4, stream=None):
    dev = _current_device()
    R = svdq_qrow_bytes(K, qfmt)
    G = K // group if group > 0 else 0
    st = lib().svdq_debug_group_partials(_dev_ptr(qx, 1, M * R, "qx", dev), _dev_ptr(qw, 1, N * R, "qw", dev),
                                         M, N, K, group, qfmt, _dev_ptr(P, 4, G * M * N * 4, "P", dev),
                                         _stream(stream))
    _check("svdq_debug_group_partials", st)


def w8a8_debug_acc(qx, qw, acc, M, N, K, stream=None):
    dev = _current_device()
    st = lib().w8a8_debug_acc(_dev_ptr(qx, 1, M * K, "qx", dev), _dev_ptr(qw, 1, N * K, "qw", dev), M, N, K,
                              _dev_ptr(acc, 4, M * N * 4, "acc", dev), _stream(stream))
    _check("w8a8_debug_acc", st)


def svdq_debug_mfma_ops(kind, blocks, iters) -> int:
    return int(lib().svdq_debug_mfma_ops(kind, blocks, iters))


def svdq_debug_mfma_rate(kind, blocks, iters, out, stream=None):
    """Back-to-back MFMAs of one kind on every SIMD; out: uint64 device tensor
    of 8 * blocks values (per wave: shader-clock span, real-time span)."""
    dev = _current_device()
    st = lib().svdq_debug_mfma_rate(kind, blocks, iters, _dev_ptr(out, 8, 8 * 8 * blocks, "out", dev),
                                    _stream(stream))
    _check("svdq_debug_mfma_rate", st)


# ------------------------------------------------ convenience allocation --

def w8a8_workspace_offset_codes() -> int:
    """Byte offset of the int8 codes of X inside the w8a8 workspace."""
    return 8192


def w8a8_workspace_offset_scale() -> int:
    """Byte offset of the fp32 activation scale inside the w8a8 workspace."""
    return 4096
