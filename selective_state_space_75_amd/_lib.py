"""ctypes binding of libmamba_scan.so (the C ABI of include/mamba_scan.h,
include/mamba_gdr.h, include/mamba_state_cache.h, include/mamba_glr.h and
include/mamba_norm.h).

Argument marshalling only: tensors are checked (device, dtype, shape,
contiguity), outputs and the workspace are allocated with torch, and raw
device pointers plus torch's current HIP stream are handed to the library.
Every step of the computation runs in the library's HIP kernels; there is no
fallback.  If the library is missing, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import itertools
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmamba_scan.so")

MAMBA_F32, MAMBA_BF16 = 0, 1
FLAG_DELTA_B = 0x1
FLAG_ACCURATE_EXPM1 = 0x2
FLAG_QK_NORM = 0x4
FLAG_BLEND = 0x8
FLAG_RMS = 0x10

STATUS = {
    0: "MAMBA_OK", -1: "MAMBA_ERR_NULL", -2: "MAMBA_ERR_SHAPE", -3: "MAMBA_ERR_DTYPE",
    -4: "MAMBA_ERR_ALIGN", -5: "MAMBA_ERR_UNSUPPORTED", -6: "MAMBA_ERR_WORKSPACE", -7: "MAMBA_ERR_HIP",
}

_lock = threading.Lock()
_lib = None


class TestKnobs(ctypes.Structure):
    """mamba_test_knobs_t of include/mamba_scan.h."""
    _fields_ = [("scan_chunks", ctypes.c_int64), ("scan_kernel", ctypes.c_int32),
                ("scan_no_balance", ctypes.c_int32), ("handover_spin", ctypes.c_int64),
                ("ssd_segments", ctypes.c_int64)]


class MambaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (what, STATUS.get(status, status), status_string(status)))


def lib() -> ctypes.CDLL:
    """The loaded library with argument types set.  Raises if it is not built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libmamba_scan.so is not built (%s); run "
                                   "`python -m selective_state_space_75_amd.build`" % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            vp, i64, u32, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint, ctypes.c_int
            L.mamba_scan_workspace_size.argtypes = [i64, i64, i64, i64]
            L.mamba_scan_workspace_size.restype = ctypes.c_size_t
            L.mamba_scan_fwd.argtypes = ([vp] * 10 + [i64] * 4 + [c_int, c_int, c_int, u32, vp,
                                                                 ctypes.c_size_t, vp])
            L.mamba_scan_fwd.restype = c_int
            L.mamba_scan_fwd_noalloc.argtypes = [vp] * 10 + [i64] * 4 + [c_int, c_int, c_int, u32, vp]
            L.mamba_scan_fwd_noalloc.restype = c_int
            L.mamba_state_update.argtypes = [vp] * 10 + [i64] * 3 + [c_int, c_int, u32, vp]
            L.mamba_state_update.restype = c_int
            L.mamba_scan_bwd_workspace_size.argtypes = [i64, i64, i64, i64]
            L.mamba_scan_bwd_workspace_size.restype = ctypes.c_size_t
            L.mamba_scan_bwd.argtypes = [vp] * 17 + [i64] * 4 + [c_int, c_int, u32, vp, ctypes.c_size_t, vp]
            L.mamba_scan_bwd.restype = c_int
            L.mamba_conv1d_fwd.argtypes = [vp] * 5 + [i64] * 4 + [c_int, c_int, c_int, vp]
            L.mamba_conv1d_fwd.restype = c_int
            L.mamba_conv1d_update.argtypes = [vp] * 5 + [i64] * 3 + [c_int, c_int, vp]
            L.mamba_conv1d_update.restype = c_int
            L.mamba_ssd_fwd.argtypes = [vp] * 10 + [i64] * 5 + [c_int, c_int, c_int, u32, vp, ctypes.c_size_t, vp]
            L.mamba_ssd_fwd.restype = c_int
            L.mamba_ssd_workspace_size.argtypes = [i64] * 5
            L.mamba_ssd_workspace_size.restype = ctypes.c_size_t
            f32, sz = ctypes.c_float, ctypes.c_size_t
            L.mamba_gdr_workspace_size.argtypes = [i64] * 6 + [c_int]
            L.mamba_gdr_workspace_size.restype = sz
            L.mamba_gdr_fwd.argtypes = [vp] * 11 + [i64] * 9 + [f32, c_int, c_int, u32, vp, sz, vp]
            L.mamba_gdr_fwd.restype = c_int
            L.mamba_gdr_bwd_workspace_size.argtypes = [i64] * 6 + [c_int, c_int]
            L.mamba_gdr_bwd_workspace_size.restype = sz
            L.mamba_gdr_bwd.argtypes = [vp] * 19 + [i64] * 9 + [f32, c_int, c_int, u32, vp, sz, vp]
            L.mamba_gdr_bwd.restype = c_int
            L.mamba_gdr_update.argtypes = [vp] * 10 + [i64] * 9 + [f32, c_int, c_int, u32, vp]
            L.mamba_gdr_update.restype = c_int
            L.mamba_gdr_set_test_knobs.argtypes = [c_int, i64]
            L.mamba_gdr_set_test_knobs.restype = c_int
            L.mamba_state_cache_write.argtypes = [vp] * 4 + [i64] * 3 + [c_int, vp]
            L.mamba_state_cache_write.restype = c_int
            L.mamba_state_cache_read.argtypes = [vp] * 4 + [i64] * 3 + [c_int, vp]
            L.mamba_state_cache_read.restype = c_int
            L.mamba_glr_workspace_size.argtypes = [i64] * 3
            L.mamba_glr_workspace_size.restype = sz
            L.mamba_glr_fwd.argtypes = [vp] * 11 + [i64] * 7 + [c_int, c_int, u32, vp, sz, vp]
            L.mamba_glr_fwd.restype = c_int
            L.mamba_glr_update.argtypes = [vp] * 10 + [i64] * 7 + [c_int, c_int, u32, vp]
            L.mamba_glr_update.restype = c_int
            L.mamba_glr_bwd_workspace_size.argtypes = [i64] * 3
            L.mamba_glr_bwd_workspace_size.restype = sz
            L.mamba_glr_bwd.argtypes = [vp] * 19 + [i64] * 7 + [c_int, c_int, u32, vp, sz, vp]
            L.mamba_glr_bwd.restype = c_int
            L.mamba_glr_set_test_knobs.argtypes = [c_int, i64]
            L.mamba_glr_set_test_knobs.restype = c_int
            L.mamba_layer_norm_workspace_size.argtypes = [i64] * 4
            L.mamba_layer_norm_workspace_size.restype = sz
            L.mamba_layer_norm_fwd.argtypes = [vp] * 5 + [i64] * 6 + [f32, c_int, c_int, u32, vp, sz, vp]
            L.mamba_layer_norm_fwd.restype = c_int
            L.mamba_layer_norm_bwd_workspace_size.argtypes = [i64] * 4
            L.mamba_layer_norm_bwd_workspace_size.restype = sz
            L.mamba_layer_norm_bwd.argtypes = [vp] * 9 + [i64] * 6 + [f32, c_int, c_int, u32, vp, sz, vp]
            L.mamba_layer_norm_bwd.restype = c_int
            L.mamba_scan_kernel.argtypes = [i64, i64, i64, i64]
            L.mamba_scan_kernel.restype = c_int
            L.mamba_set_test_knobs.argtypes = [ctypes.POINTER(TestKnobs)]
            L.mamba_set_test_knobs.restype = c_int
            L.mamba_status_string.argtypes = [c_int]
            L.mamba_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().mamba_status_string(int(status)).decode()
    except Exception:
        return "?"


SCAN_KERNELS = {"planner": 0, "general": 1, "wave_tile": 2, "row": 3, "row_lean": 4}


def set_test_knobs(scan_chunks: int = 0, scan_kernel: str = "planner", scan_no_balance: bool = False,
                   handover_spin: int = -1, ssd_segments: int = 0) -> None:
    """Process-wide test knobs of the library (mamba_set_test_knobs); no
    arguments restores the defaults.  scan_kernel: planner, general,
    wave_tile, row or row_lean."""
    k = TestKnobs(scan_chunks, SCAN_KERNELS[scan_kernel], int(scan_no_balance), handover_spin, ssd_segments)
    st = lib().mamba_set_test_knobs(ctypes.byref(k))
    if st != 0:
        raise MambaError(st, "mamba_set_test_knobs")


class test_knobs:  # noqa: N801 (used as a context manager)
    """``with test_knobs(scan_chunks=5): ...`` sets the knobs for the block and
    restores the defaults after it."""
    __test__ = False   # not a pytest test class

    def __init__(self, **kw):
        self.kw = kw

    def __enter__(self):
        set_test_knobs(**self.kw)
        return self

    def __exit__(self, *exc):
        set_test_knobs()
        return False


def scan_kernel(B: int, D: int, N: int, L: int) -> str:
    """Name of the kernel mamba_scan_fwd runs for this shape (mamba_scan_kernel)."""
    k = lib().mamba_scan_kernel(B, D, N, L)
    if k < 0:
        raise MambaError(k, "mamba_scan_kernel")
    return {1: "general", 2: "wave_tile", 3: "row", 4: "row_lean"}[k]


def workspace_size(B: int, D: int, N: int, L: int) -> int:
    n = lib().mamba_scan_workspace_size(B, D, N, L)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_scan_workspace_size")
    return n


# ----------------------------------------------------------------------------- torch marshalling
def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return MAMBA_BF16
    if t.dtype == torch.float32:
        return MAMBA_F32
    raise TypeError("unsupported dtype %s (bfloat16 or float32)" % t.dtype)


def _check(t, name, shape, dtype, device):
    if t is None:
        return None
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def scan_fwd(u, delta, z, Bt, Ct, A, Dskip=None, delta_bias=None, *, return_final_state=False,
             out_dtype=None, delta_b=False, accurate_expm1=False, y=None, final_state=None,
             workspace=None, stream=None):
    """Selective scan forward.  u, delta, z: (B, D, L); Bt, Ct: (B, N, L); A: (D, N) fp32.

    Returns y (B, D, L), or (y, final_state (B, D, N) fp32) when return_final_state.
    Outputs and workspace may be passed in to avoid allocation.
    """
    torch = _torch()
    if u.dim() != 3 or Bt.dim() != 3:
        raise ValueError("u must be (B, D, L) and Bt (B, N, L)")
    B, D, L = u.shape
    N = Bt.shape[1]
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    in_dt = u.dtype
    _dtype_code(u)
    _check(u, "u", (B, D, L), in_dt, dev)
    _check(delta, "delta", (B, D, L), in_dt, dev)
    _check(z, "z", (B, D, L), in_dt, dev)
    _check(Bt, "Bt", (B, N, L), in_dt, dev)
    _check(Ct, "Ct", (B, N, L), in_dt, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(Dskip, "Dskip", (D,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (D,), torch.float32, dev)
    out_dt = in_dt if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty((B, D, L), dtype=out_dt, device=dev)
    _check(y, "y", (B, D, L), out_dt, dev)
    if return_final_state:
        if final_state is None:
            final_state = torch.empty((B, D, N), dtype=torch.float32, device=dev)
        _check(final_state, "final_state", (B, D, N), torch.float32, dev)
    ws_bytes = workspace_size(B, D, N, L)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    flags = (FLAG_DELTA_B if delta_b else 0) | (FLAG_ACCURATE_EXPM1 if accurate_expm1 else 0)
    st = lib().mamba_scan_fwd(
        _ptr(u), _ptr(delta), _ptr(z), _ptr(Bt), _ptr(Ct), _ptr(A), _ptr(Dskip), _ptr(delta_bias),
        _ptr(y), _ptr(final_state if return_final_state else None), B, D, N, L,
        _dtype_code(u), _dtype_code(y), 1 if return_final_state else 0, flags,
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_scan_fwd")
    return (y, final_state) if return_final_state else y


def scan_fwd_noalloc(u, delta, z, Bt, Ct, A, Dskip=None, delta_bias=None, *, y, final_state=None,
                     out_dtype=None, delta_b=False, accurate_expm1=False, stream=None):
    """scan_fwd through mamba_scan_fwd_noalloc: the library's own per-GPU
    scratch instead of a workspace, and caller-provided outputs (y, and
    final_state when given), so nothing is allocated."""
    B, D, L = u.shape
    N = Bt.shape[1]
    dev = u.device
    in_dt = u.dtype
    _dtype_code(u)
    for t, name, shape, dt in ((u, "u", (B, D, L), in_dt), (delta, "delta", (B, D, L), in_dt),
                               (z, "z", (B, D, L), in_dt), (Bt, "Bt", (B, N, L), in_dt),
                               (Ct, "Ct", (B, N, L), in_dt), (A, "A", (D, N), _torch().float32),
                               (Dskip, "Dskip", (D,), _torch().float32),
                               (delta_bias, "delta_bias", (D,), _torch().float32)):
        _check(t, name, shape, dt, dev)
    _check(y, "y", (B, D, L), y.dtype if out_dtype is None else out_dtype, dev)
    _check(final_state, "final_state", (B, D, N), _torch().float32, dev)
    flags = (FLAG_DELTA_B if delta_b else 0) | (FLAG_ACCURATE_EXPM1 if accurate_expm1 else 0)
    st = lib().mamba_scan_fwd_noalloc(
        _ptr(u), _ptr(delta), _ptr(z), _ptr(Bt), _ptr(Ct), _ptr(A), _ptr(Dskip), _ptr(delta_bias),
        _ptr(y), _ptr(final_state), B, D, N, L, _dtype_code(u), _dtype_code(y),
        1 if final_state is not None else 0, flags, _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_scan_fwd_noalloc")
    return (y, final_state) if final_state is not None else y


def ssd_workspace_size(B: int, H: int, P: int, N: int, L: int) -> int:
    n = lib().mamba_ssd_workspace_size(B, H, P, N, L)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-5, "mamba_ssd_workspace_size")
    return n


def ssd_fwd(x, delta, z, Bt, Ct, A, Dskip=None, delta_bias=None, *, P=64, return_final_state=False,
            out_dtype=None, delta_b=False, y=None, final_state=None, workspace=None, stream=None):
    """Mamba-2 (SSD) layer forward.  x, z: (B, H*P, L) bf16; delta: (B, H, L) bf16;
    Bt, Ct: (B, N, L) bf16; A, delta_bias: (H) fp32; Dskip: (H*P) fp32.

    Returns y (B, H*P, L), or (y, final_state (B, H*P, N) fp32) when return_final_state.
    """
    torch = _torch()
    if x.dim() != 3 or Bt.dim() != 3 or delta.dim() != 3:
        raise ValueError("x must be (B, H*P, L), delta (B, H, L) and Bt (B, N, L)")
    B, D, L = x.shape
    H = delta.shape[1]
    N = Bt.shape[1]
    if H * P != D:
        raise ValueError("x has %d channels, delta %d heads of P = %d" % (D, H, P))
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    in_dt = x.dtype
    _dtype_code(x)
    _check(x, "x", (B, D, L), in_dt, dev)
    _check(delta, "delta", (B, H, L), in_dt, dev)
    _check(z, "z", (B, D, L), in_dt, dev)
    _check(Bt, "Bt", (B, N, L), in_dt, dev)
    _check(Ct, "Ct", (B, N, L), in_dt, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(Dskip, "Dskip", (D,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (H,), torch.float32, dev)
    out_dt = in_dt if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty((B, D, L), dtype=out_dt, device=dev)
    _check(y, "y", (B, D, L), out_dt, dev)
    if return_final_state:
        if final_state is None:
            final_state = torch.empty((B, D, N), dtype=torch.float32, device=dev)
        _check(final_state, "final_state", (B, D, N), torch.float32, dev)
    ws_bytes = ssd_workspace_size(B, H, P, N, L) if (N in (64, 128) and P % 64 == 0) else 0
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = lib().mamba_ssd_fwd(
        _ptr(x), _ptr(delta), _ptr(z), _ptr(Bt), _ptr(Ct), _ptr(A), _ptr(Dskip), _ptr(delta_bias),
        _ptr(y), _ptr(final_state if return_final_state else None), B, H, P, N, L,
        _dtype_code(x), _dtype_code(y), 1 if return_final_state else 0, FLAG_DELTA_B if delta_b else 0,
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_ssd_fwd")
    return (y, final_state) if return_final_state else y


def state_update(state, u, delta, z, Bt, Ct, A, Dskip=None, delta_bias=None, *, out_dtype=None,
                 delta_b=False, accurate_expm1=False, y=None, stream=None):
    """One decoding step; `state` (B, D, N) fp32 is updated in place.  Returns y (B, D)."""
    torch = _torch()
    if state.dim() != 3:
        raise ValueError("state must be (B, D, N)")
    B, D, N = state.shape
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    in_dt = u.dtype
    _dtype_code(u)
    _check(state, "state", (B, D, N), torch.float32, dev)
    _check(u, "u", (B, D), in_dt, dev)
    _check(delta, "delta", (B, D), in_dt, dev)
    _check(z, "z", (B, D), in_dt, dev)
    _check(Bt, "Bt", (B, N), in_dt, dev)
    _check(Ct, "Ct", (B, N), in_dt, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(Dskip, "Dskip", (D,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (D,), torch.float32, dev)
    out_dt = in_dt if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty((B, D), dtype=out_dt, device=dev)
    _check(y, "y", (B, D), out_dt, dev)
    st = lib().mamba_state_update(
        _ptr(state), _ptr(u), _ptr(delta), _ptr(z), _ptr(Bt), _ptr(Ct), _ptr(A), _ptr(Dskip),
        _ptr(delta_bias), _ptr(y), B, D, N, _dtype_code(u), _dtype_code(y),
        (FLAG_DELTA_B if delta_b else 0) | (FLAG_ACCURATE_EXPM1 if accurate_expm1 else 0),
        _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_state_update")
    return y


def conv1d_fwd(x, weight, bias=None, *, return_final_state=False, out_dtype=None, y=None, final_state=None,
               stream=None):
    """Causal depthwise conv1d + SiLU.  x: (B, D, L); weight: (D, K) fp32 with
    weight[d, i] multiplying x[..., t - i]; bias: (D) fp32 or None.

    Returns y (B, D, L), or (y, final_state (B, D, K) fp32) when return_final_state.
    """
    torch = _torch()
    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be (B, D, L) and weight (D, K)")
    B, D, L = x.shape
    K = weight.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    _dtype_code(x)
    _check(x, "x", (B, D, L), x.dtype, dev)
    _check(weight, "weight", (D, K), torch.float32, dev)
    _check(bias, "bias", (D,), torch.float32, dev)
    out_dt = x.dtype if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty((B, D, L), dtype=out_dt, device=dev)
    _check(y, "y", (B, D, L), out_dt, dev)
    if return_final_state:
        if final_state is None:
            final_state = torch.empty((B, D, K), dtype=torch.float32, device=dev)
        _check(final_state, "final_state", (B, D, K), torch.float32, dev)
    st = lib().mamba_conv1d_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(y),
                                _ptr(final_state if return_final_state else None), B, D, L, K,
                                _dtype_code(x), _dtype_code(y), 1 if return_final_state else 0,
                                _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_conv1d_fwd")
    return (y, final_state) if return_final_state else y


def conv1d_update(state, x, weight, bias=None, *, out_dtype=None, y=None, stream=None):
    """One decoding step of the convolution; `state` (B, D, K) fp32 (the K most
    recent inputs, oldest first) is updated in place.  x: (B, D).  Returns y (B, D)."""
    torch = _torch()
    if state.dim() != 3:
        raise ValueError("state must be (B, D, K)")
    B, D, K = state.shape
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    _dtype_code(x)
    _check(state, "state", (B, D, K), torch.float32, dev)
    _check(x, "x", (B, D), x.dtype, dev)
    _check(weight, "weight", (D, K), torch.float32, dev)
    _check(bias, "bias", (D,), torch.float32, dev)
    out_dt = x.dtype if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty((B, D), dtype=out_dt, device=dev)
    _check(y, "y", (B, D), out_dt, dev)
    st = lib().mamba_conv1d_update(_ptr(state), _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), B, D, K,
                                   _dtype_code(x), _dtype_code(y), _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_conv1d_update")
    return y


def scan_bwd_workspace_size(B: int, D: int, N: int, L: int) -> int:
    n = lib().mamba_scan_bwd_workspace_size(B, D, N, L)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_scan_bwd_workspace_size")
    return n


def scan_bwd(u, delta, z, Bt, Ct, A, Dskip, delta_bias, dy, *, grad_dtype=None, delta_b=False,
             accurate_expm1=False, workspace=None, stream=None):
    """Gradients of scan_fwd (zero initial state) for output gradient dy (B, D, L).

    Returns a dict: du, ddelta, dz (B, D, L) in grad_dtype (dz None when z is
    None); dBt, dCt (B, N, L), dA (D, N), dDskip (D), ddelta_bias (D) fp32.
    """
    torch = _torch()
    if u.dim() != 3 or Bt.dim() != 3:
        raise ValueError("u must be (B, D, L) and Bt (B, N, L)")
    B, D, L = u.shape
    N = Bt.shape[1]
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    in_dt = u.dtype
    _dtype_code(u)
    for t, n, shp in ((u, "u", (B, D, L)), (delta, "delta", (B, D, L)), (z, "z", (B, D, L)),
                      (Bt, "Bt", (B, N, L)), (Ct, "Ct", (B, N, L))):
        _check(t, n, shp, in_dt, dev)
    _check(A, "A", (D, N), torch.float32, dev)
    _check(Dskip, "Dskip", (D,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (D,), torch.float32, dev)
    gdt = dy.dtype if grad_dtype is None else grad_dtype
    _check(dy, "dy", (B, D, L), gdt, dev)
    out = {"du": torch.empty((B, D, L), dtype=gdt, device=dev), "ddelta": torch.empty((B, D, L), dtype=gdt, device=dev),
           "dz": torch.empty((B, D, L), dtype=gdt, device=dev) if z is not None else None,
           "dBt": torch.empty((B, N, L), dtype=torch.float32, device=dev),
           "dCt": torch.empty((B, N, L), dtype=torch.float32, device=dev),
           "dA": torch.empty((D, N), dtype=torch.float32, device=dev),
           "dDskip": torch.empty((D,), dtype=torch.float32, device=dev),
           "ddelta_bias": torch.empty((D,), dtype=torch.float32, device=dev)}
    wsb = scan_bwd_workspace_size(B, D, N, L)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    st = lib().mamba_scan_bwd(
        _ptr(u), _ptr(delta), _ptr(z), _ptr(Bt), _ptr(Ct), _ptr(A), _ptr(Dskip), _ptr(delta_bias), _ptr(dy),
        _ptr(out["du"]), _ptr(out["ddelta"]), _ptr(out["dz"]), _ptr(out["dBt"]), _ptr(out["dCt"]), _ptr(out["dA"]),
        _ptr(out["dDskip"]), _ptr(out["ddelta_bias"]), B, D, N, L, _dtype_code(u), _dtype_code(dy),
        (FLAG_DELTA_B if delta_b else 0) | (FLAG_ACCURATE_EXPM1 if accurate_expm1 else 0),
        _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_scan_bwd")
    return out


# ----------------------------------------------------------------------------- gated delta rule
def _check_rows(t, name, shape, dtype, device):
    """Like _check for (B, C, ...) tensors whose batch rows are each dense: a
    channel range of a wider tensor is taken as it is.  Returns the row stride."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    row = 1
    for n in shape[1:]:
        row *= n
    if not t[:1].is_contiguous() or (shape[0] > 1 and t.stride(0) < row):
        raise ValueError("%s must be dense within each batch row" % name)
    return t.stride(0) if shape[0] > 1 else row


def _gdr_sizes(q, v, delta, groups, dims):
    """(B, H, G, P, N) from the arguments' shapes."""
    if q.dim() != dims or v.dim() != dims or delta.dim() != dims:
        raise ValueError("q, v and delta must have %d dimensions" % dims)
    B, H = delta.shape[:2]
    G = H if groups is None else int(groups)
    if G < 1 or H % G or q.shape[1] % G or v.shape[1] % H or not q.shape[1] or not v.shape[1]:
        raise ValueError("q has %d channels, v %d and delta %d heads, which do not divide into %d key heads"
                         % (q.shape[1], v.shape[1], H, G))
    if q.device.type != "cuda":
        raise ValueError("inputs must be on a GPU device")
    _dtype_code(q)
    return B, H, G, v.shape[1] // H, q.shape[1] // G


GDR_KERNELS = {"planner": 0, "token": 1, "chunk": 2}


class gdr_test_knobs:  # noqa: N801 (used as a context manager)
    """``with gdr_test_knobs(kernel="chunk", segments=3): ...`` sets the gated delta
    rule's test knobs (mamba_gdr_set_test_knobs) for the block and restores the
    planner's choices after it."""
    __test__ = False   # not a pytest test class

    def __init__(self, kernel: str = "planner", segments: int = 0):
        self.args = (GDR_KERNELS[kernel], segments)

    def __enter__(self):
        st = lib().mamba_gdr_set_test_knobs(*self.args)
        if st != 0:
            raise MambaError(st, "mamba_gdr_set_test_knobs")
        return self

    def __exit__(self, *exc):
        lib().mamba_gdr_set_test_knobs(0, 0)
        return False


def _gdr_scale(scale, N):
    return float(N) ** -0.5 if scale is None else float(scale)


def gdr_workspace_size(B: int, H: int, G: int, P: int, N: int, L: int, dtype=None) -> int:
    """Bytes gdr_fwd needs for these sizes and this input dtype (bfloat16 by default)."""
    code = MAMBA_F32 if dtype is not None and dtype == _torch().float32 else MAMBA_BF16
    n = lib().mamba_gdr_workspace_size(B, H, G, P, N, L, code)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_gdr_workspace_size")
    return n


def _on(dev, stream):
    """The device of a call, and the stream whose pool its own tensors come from: memory of
    another stream's pool could be handed out again while the call's kernels still use it."""
    torch = _torch()
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError("stream is on %s, expected %s" % (stream.device, dev))
    return torch.cuda.stream(stream)


def _workspace(workspace, need, dev):
    torch = _torch()
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    if workspace.device != dev:
        raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def gdr_fwd(q, k, v, delta, beta, A, delta_bias=None, *, groups=None, initial_state=None, lengths=None,
            qk_norm=False, scale=None, return_final_state=False, out_dtype=None, y=None, final_state=None,
            workspace=None, stream=None):
    """Gated delta rule over whole sequences (include/mamba_gdr.h).

    q, k: (B, G*N, L); v: (B, H*P, L); delta, beta: (B, H, L), raw; A, delta_bias: (H)
    fp32.  groups = G (default H) key heads serve the H heads of delta.  q, k and v may be
    channel ranges of a wider tensor.  initial_state: (B, H*P, N) fp32; lengths: (B)
    int32, tokens per row; scale: default N**-0.5.  The number of rows B takes part in the
    choice of the kernel: a row alone and in a batch agrees to fp32 rounding.

    Returns y (B, H*P, L), or (y, final_state (B, H*P, N) fp32) when return_final_state.
    """
    torch = _torch()
    B, H, G, P, N = _gdr_sizes(q, v, delta, groups, 3)
    L, dev, in_dt = q.shape[2], q.device, q.dtype
    qs = _check_rows(q, "q", (B, G * N, L), in_dt, dev)
    ks = _check_rows(k, "k", (B, G * N, L), in_dt, dev)
    vs = _check_rows(v, "v", (B, H * P, L), in_dt, dev)
    _check(delta, "delta", (B, H, L), in_dt, dev)
    _check(beta, "beta", (B, H, L), in_dt, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (H,), torch.float32, dev)
    _check(initial_state, "initial_state", (B, H * P, N), torch.float32, dev)
    _check(lengths, "lengths", (B,), torch.int32, dev)
    out_dt = in_dt if out_dtype is None else out_dtype
    with _on(dev, stream):
        if y is None:
            y = torch.empty((B, H * P, L), dtype=out_dt, device=dev)
        _check(y, "y", (B, H * P, L), out_dt, dev)
        if return_final_state:
            if final_state is None:
                final_state = torch.empty((B, H * P, N), dtype=torch.float32, device=dev)
            _check(final_state, "final_state", (B, H * P, N), torch.float32, dev)
        workspace = _workspace(workspace, gdr_workspace_size(B, H, G, P, N, L, in_dt), dev)
        st = lib().mamba_gdr_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(delta), _ptr(beta), _ptr(A), _ptr(delta_bias), _ptr(initial_state),
            _ptr(lengths), _ptr(y), _ptr(final_state if return_final_state else None), B, H, G, P, N, L, qs, ks, vs,
            _gdr_scale(scale, N), _dtype_code(q), _dtype_code(y), FLAG_QK_NORM if qk_norm else 0,
            _ptr(workspace), _nbytes(workspace), _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_gdr_fwd")
    return (y, final_state) if return_final_state else y


def gdr_bwd_workspace_size(B: int, H: int, G: int, P: int, N: int, L: int, dtype=None, grad_dtype=None) -> int:
    """Bytes gdr_bwd needs for these sizes and dtypes (bfloat16 by default; gradients like the inputs)."""
    f32 = _torch().float32
    code = MAMBA_F32 if dtype == f32 else MAMBA_BF16
    gcode = code if grad_dtype is None else MAMBA_F32 if grad_dtype == f32 else MAMBA_BF16
    n = lib().mamba_gdr_bwd_workspace_size(B, H, G, P, N, L, code, gcode)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_gdr_bwd_workspace_size")
    return n


def gdr_bwd(q, k, v, delta, beta, A, delta_bias, dy, *, groups=None, initial_state=None, dfinal_state=None,
            lengths=None, qk_norm=False, scale=None, workspace=None, stream=None):
    """Gradients of gdr_fwd for the output gradient dy (B, H*P, L) and, optionally, the
    final state's dfinal_state (B, H*P, N) fp32; the other arguments as for gdr_fwd.

    Returns a dict: dq, dk (B, G*N, L), dv (B, H*P, L), ddelta, dbeta (B, H, L) in dy's
    dtype; dA, ddelta_bias (H) fp32; dinitial_state (B, H*P, N) fp32 (None without
    initial_state).
    """
    torch = _torch()
    B, H, G, P, N = _gdr_sizes(q, v, delta, groups, 3)
    L, dev, in_dt = q.shape[2], q.device, q.dtype
    qs = _check_rows(q, "q", (B, G * N, L), in_dt, dev)
    ks = _check_rows(k, "k", (B, G * N, L), in_dt, dev)
    vs = _check_rows(v, "v", (B, H * P, L), in_dt, dev)
    _check(delta, "delta", (B, H, L), in_dt, dev)
    _check(beta, "beta", (B, H, L), in_dt, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (H,), torch.float32, dev)
    _check(initial_state, "initial_state", (B, H * P, N), torch.float32, dev)
    _check(dfinal_state, "dfinal_state", (B, H * P, N), torch.float32, dev)
    _check(lengths, "lengths", (B,), torch.int32, dev)
    _dtype_code(dy)
    _check(dy, "dy", (B, H * P, L), None, dev)
    gdt = dy.dtype
    with _on(dev, stream):
        def new(*shape, dtype=gdt):
            return torch.empty(shape, dtype=dtype, device=dev)

        out = {"dq": new(B, G * N, L), "dk": new(B, G * N, L), "dv": new(B, H * P, L), "ddelta": new(B, H, L),
               "dbeta": new(B, H, L), "dA": new(H, dtype=torch.float32), "ddelta_bias": new(H, dtype=torch.float32),
               "dinitial_state": None if initial_state is None else new(B, H * P, N, dtype=torch.float32)}
        workspace = _workspace(workspace, gdr_bwd_workspace_size(B, H, G, P, N, L, in_dt, gdt), dev)
        st = lib().mamba_gdr_bwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(delta), _ptr(beta), _ptr(A), _ptr(delta_bias), _ptr(initial_state),
            _ptr(lengths), _ptr(dy), _ptr(dfinal_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
            _ptr(out["ddelta"]), _ptr(out["dbeta"]), _ptr(out["dA"]), _ptr(out["ddelta_bias"]),
            _ptr(out["dinitial_state"]), B, H, G, P, N, L, qs, ks, vs, _gdr_scale(scale, N), _dtype_code(q),
            _dtype_code(dy), FLAG_QK_NORM if qk_norm else 0, _ptr(workspace), _nbytes(workspace), _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_gdr_bwd")
    return out


def gdr_update(state, q, k, v, delta, beta, A, delta_bias=None, *, groups=None, slots=None, qk_norm=False,
               scale=None, out_dtype=None, y=None, stream=None):
    """One token of the gated delta rule for every row; `state` (S, H*P, N) fp32 is
    updated in place at the rows' slots (int32 (B); None: row b has state b; negative:
    an empty row, y = 0).  q, k: (B, G*N); v: (B, H*P); delta, beta: (B, H).  Returns y
    (B, H*P)."""
    torch = _torch()
    B, H, G, P, N = _gdr_sizes(q, v, delta, groups, 2)
    dev, in_dt = q.device, q.dtype
    if state.dim() != 3:
        raise ValueError("state must be (S, H*P, N)")
    S = state.shape[0]
    qs = _check_rows(q, "q", (B, G * N), in_dt, dev)
    ks = _check_rows(k, "k", (B, G * N), in_dt, dev)
    vs = _check_rows(v, "v", (B, H * P), in_dt, dev)
    _check(delta, "delta", (B, H), in_dt, dev)
    _check(beta, "beta", (B, H), in_dt, dev)
    _check(A, "A", (H,), torch.float32, dev)
    _check(delta_bias, "delta_bias", (H,), torch.float32, dev)
    _check(state, "state", (S, H * P, N), torch.float32, dev)
    _check(slots, "slots", (B,), torch.int32, dev)
    out_dt = in_dt if out_dtype is None else out_dtype
    with _on(dev, stream):
        if y is None:
            y = torch.empty((B, H * P), dtype=out_dt, device=dev)
        _check(y, "y", (B, H * P), out_dt, dev)
        st = lib().mamba_gdr_update(
            _ptr(state), _ptr(slots), _ptr(q), _ptr(k), _ptr(v), _ptr(delta), _ptr(beta), _ptr(A), _ptr(delta_bias),
            _ptr(y), B, H, G, P, N, S, qs, ks, vs, _gdr_scale(scale, N), _dtype_code(q), _dtype_code(y),
            FLAG_QK_NORM if qk_norm else 0, _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_gdr_update")
    return y


# ----------------------------------------------------------------------------- 8-bit state cache
CACHE_GROUP = 32


def state_cache(n_slots: int, n: int, device):
    """An empty cache of n_slots rows of n numbers: (codes int8 (n_slots, n), exps uint8
    (n_slots, ceil(n / 32))).  Every row reads as zeros until it is written."""
    torch = _torch()
    return (torch.zeros((n_slots, n), dtype=torch.int8, device=device),
            torch.zeros((n_slots, (n + CACHE_GROUP - 1) // CACHE_GROUP), dtype=torch.uint8, device=device))


def _check_codes(codes):
    if not isinstance(codes, _torch().Tensor):
        raise TypeError("codes must be a torch.Tensor")
    if codes.dim() != 2:
        raise ValueError("codes must be (n_slots, n)")


def _cache_args(codes, exps, slots, state, what):
    torch = _torch()
    _check_codes(codes)
    S, n = codes.shape
    dev = codes.device
    if dev.type != "cuda":
        raise ValueError("%s must be on a GPU device" % what)
    _check(codes, "codes", (S, n), torch.int8, dev)
    _check(exps, "exps", (S, (n + CACHE_GROUP - 1) // CACHE_GROUP), torch.uint8, dev)
    if state.dim() < 1 or not state.shape[0] or state.numel() != state.shape[0] * n:
        raise ValueError("%s has shape %s, expected (rows, ...) with %d numbers a row" % (what, tuple(state.shape), n))
    _dtype_code(state)
    _check(state, what, tuple(state.shape), None, dev)
    _check(slots, "slots", (state.shape[0],), torch.int32, dev)
    return state.shape[0], n, S, dev


def state_cache_write(state, codes, exps, *, slots=None, stream=None):
    """Keep the rows of `state` (rows, ...) fp32 or bf16 in 8 bits (include/
    mamba_state_cache.h): row r in slot slots[r] (int32 (rows); None: slot r;
    negative: not kept) of codes (n_slots, n) int8 and exps (n_slots, ceil(n / 32)) uint8."""
    rows, n, S, dev = _cache_args(codes, exps, slots, state, "state")
    with _on(dev, stream):
        st = lib().mamba_state_cache_write(_ptr(state), _ptr(slots), _ptr(codes), _ptr(exps), rows, n, S,
                                           _dtype_code(state), _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_state_cache_write")


def state_cache_read(codes, exps, *, slots=None, out=None, dtype=None, stream=None):
    """Rows of an 8-bit state cache: out[r] = the row kept in slot slots[r] (int32
    (rows); None: every slot in order; negative: zeros).  `out` (rows, ...) fp32 or bf16
    is written when given, else a (rows, n) tensor of `dtype` (fp32) is made."""
    torch = _torch()
    _check_codes(codes)
    if out is None:
        if slots is not None and (not isinstance(slots, torch.Tensor) or slots.dim() != 1):
            raise ValueError("slots must be an int32 tensor of one dimension")
        rows = codes.shape[0] if slots is None else slots.shape[0]
        with _on(codes.device, stream) if codes.is_cuda else contextlib.nullcontext():
            out = torch.empty((rows, codes.shape[1]), dtype=dtype or torch.float32, device=codes.device)
    rows, n, S, dev = _cache_args(codes, exps, slots, out, "out")
    with _on(dev, stream):
        st = lib().mamba_state_cache_read(_ptr(codes), _ptr(exps), _ptr(slots), _ptr(out), rows, n, S,
                                          _dtype_code(out), _stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_state_cache_read")
    return out


# ----------------------------------------------------------------------------- gated linear recurrence
class glr_test_knobs:  # noqa: N801 (used as a context manager)
    """``with glr_test_knobs(waves=2, segments=3): ...`` sets the gated linear recurrence's
    test knobs (mamba_glr_set_test_knobs) for the block and restores the planner's choices
    after it."""
    __test__ = False   # not a pytest test class

    def __init__(self, waves: int = 0, segments: int = 0):
        self.args = (waves, segments)

    def __enter__(self):
        st = lib().mamba_glr_set_test_knobs(*self.args)
        if st != 0:
            raise MambaError(st, "mamba_glr_set_test_knobs")
        return self

    def __exit__(self, *exc):
        lib().mamba_glr_set_test_knobs(0, 0)
        return False


def _row_stride(t, name, shape, dtype, device, row):
    """_check_rows without the view it makes: for a call of one token the checks are most of the
    call.  (B, D, L) or (B, D) of `row` numbers a batch row; an absent tensor has stride 0.  What is not
    plainly right is left to _check_rows, which names it."""
    if t is None:
        return 0
    if isinstance(t, _torch().Tensor) and t.dtype == dtype and t.shape == shape and t.device == device:
        if t.is_contiguous():
            return row
        s = t.stride()
        if shape[0] > 1 and s[0] >= row and s[-1] == 1 and (len(s) == 2 or s[1] == shape[2]):
            return s[0]
    return _check_rows(t, name, shape, dtype, device)


def _plain(t, name, shape, dtype, device):
    """_check for a tensor or None, the address in its place."""
    if t is None:
        return None
    if not (isinstance(t, _torch().Tensor) and t.dtype == dtype and t.shape == shape and t.is_contiguous()
            and t.device == device):
        _check(t, name, shape, dtype, device)
    return t.data_ptr()


def _addr(t):
    return None if t is None else t.data_ptr()


def _like(x, dtype):
    """A dense tensor of x's shape (empty_like is the shorter call)."""
    torch = _torch()
    if x.dtype == dtype and x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, dtype=dtype, device=x.device)


def _apart(out, name, ins, strides, dense):
    """The caller's output, which must not lie over an input (batch rows `strides` apart), nor over the `dense`
    parameters, states and outputs of the call: workgroups read and write in no order."""
    lo = out.data_ptr()
    hi = lo + out.numel() * out.element_size()
    for t, s in itertools.chain(zip(ins, strides), zip(dense, itertools.repeat(None))):
        if t is not None and t.numel():
            at, B = t.data_ptr(), t.shape[0]
            n = t.numel() if s is None else (B - 1) * s + t.numel() // B
            if at < hi and lo < at + n * t.element_size():
                raise ValueError("%s must not overlap the inputs or another output" % name)


_HERE = contextlib.nullcontext()


def _there(dev, stream):
    """_on, which is entered only where the call's device is not the current one or a stream is given."""
    if stream is None and _torch().cuda.current_device() == dev.index:
        return _HERE
    return _on(dev, stream)


def _raw_stream(dev, stream):
    return _torch()._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _first(x, dims, what):
    """Checks the input that the others are held to, and returns its device, dtype and dtype code."""
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() not in dims:
        raise ValueError("x must be %s" % what)
    if not x.is_cuda:
        raise ValueError("inputs must be on a GPU device")
    return x.device, x.dtype, _dtype_code(x)


def _glr_inputs(x, r, i, z, A, r_bias, i_bias, blend):
    """Checks of the inputs that every call of the recurrence has; returns the addresses of x, r, i, z, A
    and the biases, and the batch strides."""
    shape, dev, dt = x.shape, x.device, x.dtype
    if r is None:
        raise TypeError("r must be a torch.Tensor")
    row = shape[1] * shape[2] if len(shape) == 3 else shape[1]
    strides = (_row_stride(x, "x", shape, dt, dev, row), _row_stride(r, "r", shape, dt, dev, row),
               _row_stride(i, "i", shape, dt, dev, row), _row_stride(z, "z", shape, dt, dev, row))
    if blend:
        if A is not None:
            raise ValueError("A is not used with blend=True and must be None")
    elif A is None:
        raise ValueError("A is needed unless blend=True")
    if i is None and i_bias is not None:
        raise ValueError("i_bias without i")
    per, f32 = (shape[1],), _torch().float32
    return (x.data_ptr(), r.data_ptr(), _addr(i), _addr(z), _plain(A, "A", per, f32, dev),
            _plain(r_bias, "r_bias", per, f32, dev), _plain(i_bias, "i_bias", per, f32, dev)), strides


def glr_workspace_size(B: int, D: int, L: int) -> int:
    """Bytes glr_fwd needs for these sizes."""
    n = lib().mamba_glr_workspace_size(B, D, L)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_glr_workspace_size")
    return n


def glr_fwd(x, r, i=None, A=None, r_bias=None, i_bias=None, z=None, *, blend=False, initial_state=None, lengths=None,
            return_final_state=False, out_dtype=None, y=None, final_state=None, workspace=None, stream=None):
    """Gated linear recurrence over whole sequences (include/mamba_glr.h), per channel

        h_t = a_t h_(t-1) + n_t sigmoid(i_t + i_bias) x_t,   y_t = h_t silu(z_t)

    with s = sigmoid(r + r_bias), a = exp(A s) and n = sqrt(1 - a^2), or a = 1 - s and n = s with
    blend=True (then A is None).  x, r, i, z: (B, D, L), i and z optional; they may be channel ranges
    of a wider tensor.  A (below zero), r_bias, i_bias: (D) fp32.  initial_state: (B, D) fp32;
    lengths: (B) int32, tokens per row.

    Returns y (B, D, L), or (y, final_state (B, D) fp32) when return_final_state.  A y or final_state
    passed in must lie apart from the inputs, initial_state among them (ValueError).
    """
    torch = _torch()
    dev, in_dt, code = _first(x, (3,), "(B, D, L)")
    B, D, L = shape = x.shape
    ins, strides = _glr_inputs(x, r, i, z, A, r_bias, i_bias, blend)
    init = _plain(initial_state, "initial_state", (B, D), torch.float32, dev)
    ends = _plain(lengths, "lengths", (B,), torch.int32, dev)
    out_dt = in_dt if out_dtype is None else out_dtype
    with _there(dev, stream):
        if y is None:
            y = _like(x, out_dt)
            yp = y.data_ptr()
        else:
            yp = _plain(y, "y", shape, out_dt, dev)
            _apart(y, "y", (x, r, i, z), strides, (A, r_bias, i_bias, initial_state, lengths))
        last = None
        if return_final_state:
            if final_state is None:
                final_state = torch.empty((B, D), dtype=torch.float32, device=dev)
                last = final_state.data_ptr()
            else:
                last = _plain(final_state, "final_state", (B, D), torch.float32, dev)
                _apart(final_state, "final_state", (x, r, i, z), strides, (A, r_bias, i_bias, initial_state, lengths, y))
        workspace = _workspace(workspace, glr_workspace_size(B, D, L), dev)
        st = lib().mamba_glr_fwd(*ins, init, ends, yp, last, B, D, L, *strides, code, _dtype_code(y),
                                 FLAG_BLEND if blend else 0, _addr(workspace), _nbytes(workspace),
                                 _raw_stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_glr_fwd")
    return (y, final_state) if return_final_state else y


def glr_bwd_workspace_size(B: int, D: int, L: int) -> int:
    """Bytes glr_bwd needs for these sizes."""
    n = lib().mamba_glr_bwd_workspace_size(B, D, L)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_glr_bwd_workspace_size")
    return n


def glr_bwd(x, r, i, A, r_bias, i_bias, z, dy, *, blend=False, initial_state=None, dfinal_state=None, lengths=None,
            workspace=None, stream=None):
    """Gradients of glr_fwd for the output gradient dy (B, D, L) and, optionally, the final
    state's dfinal_state (B, D) fp32; the other arguments as for glr_fwd.

    Returns a dict: dx, dr, di, dz (B, D, L) in dy's dtype (di and dz None without i and z); dA
    (None with blend), dr_bias, di_bias (None without i) (D) fp32; dinitial_state (B, D) fp32
    (None without initial_state).
    """
    torch = _torch()
    dev, _, code = _first(x, (3,), "(B, D, L)")
    B, D, L = shape = x.shape
    ins, strides = _glr_inputs(x, r, i, z, A, r_bias, i_bias, blend)
    init = _plain(initial_state, "initial_state", (B, D), torch.float32, dev)
    dfinal = _plain(dfinal_state, "dfinal_state", (B, D), torch.float32, dev)
    ends = _plain(lengths, "lengths", (B,), torch.int32, dev)
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch.Tensor")
    gdt, gcode = dy.dtype, _dtype_code(dy)
    dyp = _plain(dy, "dy", shape, gdt, dev)
    with _there(dev, stream):
        sums = torch.empty((3, D), dtype=torch.float32, device=dev).unbind()
        out = {"dx": torch.empty_like(dy), "dr": torch.empty_like(dy), "di": None if i is None else torch.empty_like(dy),
               "dz": None if z is None else torch.empty_like(dy), "dA": None if blend else sums[0], "dr_bias": sums[1],
               "di_bias": None if i is None else sums[2],
               "dinitial_state": None if init is None else torch.empty_like(initial_state)}
        workspace = _workspace(workspace, glr_bwd_workspace_size(B, D, L), dev)
        st = lib().mamba_glr_bwd(*ins, init, ends, dyp, dfinal, *[_addr(t) for t in out.values()], B, D, L, *strides,
                                 code, gcode, FLAG_BLEND if blend else 0, _addr(workspace), _nbytes(workspace),
                                 _raw_stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_glr_bwd")
    return out


def glr_update(state, x, r, i=None, A=None, r_bias=None, i_bias=None, z=None, *, blend=False, slots=None,
               out_dtype=None, y=None, stream=None):
    """One token of the gated linear recurrence for every row; `state` (S, D) fp32 is updated in
    place at the rows' slots (int32 (B); None: row b has state b; negative: an empty row, y = 0).
    x, r, i, z: (B, D).  Returns y (B, D).  A y passed in must lie apart from state and the inputs, and
    those apart from state (ValueError)."""
    torch = _torch()
    dev, in_dt, code = _first(x, (2,), "(B, D)")
    B, D = shape = x.shape
    if not isinstance(state, torch.Tensor) or state.dim() != 2:
        raise ValueError("state must be (S, D)")
    ins, strides = _glr_inputs(x, r, i, z, A, r_bias, i_bias, blend)
    S = state.shape[0]
    pool = _plain(state, "state", (S, D), torch.float32, dev)
    if code == MAMBA_F32:                      # as _apart, by the addresses at hand; inputs of another type are no states
        hi = pool + 4 * S * D
        for at, s in zip(ins, strides):
            if at is not None and at < hi and pool < at + 4 * ((B - 1) * s + D):
                raise ValueError("state must not overlap the inputs")
    rows = _plain(slots, "slots", (B,), torch.int32, dev)
    out_dt = in_dt if out_dtype is None else out_dtype
    with _there(dev, stream):
        if y is None:
            y = _like(x, out_dt)
            yp = y.data_ptr()
        else:
            yp = _plain(y, "y", shape, out_dt, dev)
            _apart(y, "y", (x, r, i, z), strides, (state, A, r_bias, i_bias, slots))
        st = lib().mamba_glr_update(pool, rows, *ins, yp, B, D, S, *strides, code,
                                    _dtype_code(y), FLAG_BLEND if blend else 0, _raw_stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_glr_update")
    return y


# ----------------------------------------------------------------------------- layer norm over channels
def _norm_inputs(x, weight, bias, z, groups):
    """Checks of the norm's inputs; returns the device, x's dtype code, the addresses of x, z, weight and
    bias, and (B, D, L, groups, batch strides of x and z)."""
    f32 = _torch().float32
    dev, dt, code = _first(x, (2, 3), "(B, D, L) or (rows, D)")
    shape, groups = x.shape, int(groups)
    D = shape[1]
    if groups < 1 or D % groups:
        raise ValueError("%d channels do not divide into %d groups" % (D, groups))
    L = shape[2] if len(shape) == 3 else 1
    strides = _row_stride(x, "x", shape, dt, dev, D * L), _row_stride(z, "z", shape, dt, dev, D * L)
    ins = (x.data_ptr(), _addr(z), _plain(weight, "weight", (D,), f32, dev), _plain(bias, "bias", (D,), f32, dev))
    return dev, code, ins, (shape[0], D, L, groups) + strides


def layer_norm_workspace_size(B: int, D: int, L: int, groups: int = 1) -> int:
    """Bytes layer_norm_fwd needs for these sizes (L = 1 for token-major rows)."""
    n = lib().mamba_layer_norm_workspace_size(B, D, L, groups)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_layer_norm_workspace_size")
    return n


def layer_norm_fwd(x, weight=None, bias=None, z=None, *, groups=1, eps=1e-5, rms=False, out_dtype=None, y=None,
                   workspace=None, stream=None):
    """Layer norm of every token over its channels, or over each of `groups` equal ranges of them,
    with the output gate (include/mamba_norm.h): (xh weight + bias) silu(z), xh = (x - mean) /
    sqrt(var + eps), or x / sqrt(mean x^2 + eps) with rms=True.  x, z: (B, D, L), or (rows, D) for
    token-major rows; both may be channel ranges of a wider tensor.  weight, bias: (D) fp32 or None.
    Returns y like x, in out_dtype.  A y passed in must lie apart from the inputs (ValueError)."""
    torch = _torch()
    dev, code, ins, sizes = _norm_inputs(x, weight, bias, z, groups)
    out_dt = x.dtype if out_dtype is None else out_dtype
    with _there(dev, stream):
        if y is None:
            y = _like(x, out_dt)
            yp = y.data_ptr()
        else:
            yp = _plain(y, "y", x.shape, out_dt, dev)
            _apart(y, "y", (x, z), sizes[4:], (weight, bias))
        workspace = _workspace(workspace, layer_norm_workspace_size(*sizes[:4]), dev)
        st = lib().mamba_layer_norm_fwd(*ins, yp, *sizes, eps, code, _dtype_code(y),
                                        FLAG_RMS if rms else 0, _addr(workspace), _nbytes(workspace),
                                        _raw_stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_layer_norm_fwd")
    return y


def layer_norm_bwd_workspace_size(B: int, D: int, L: int, groups: int = 1) -> int:
    """Bytes layer_norm_bwd needs for these sizes (L = 1 for token-major rows)."""
    n = lib().mamba_layer_norm_bwd_workspace_size(B, D, L, groups)
    if n == ctypes.c_size_t(-1).value:
        raise MambaError(-2, "mamba_layer_norm_bwd_workspace_size")
    return n


def layer_norm_bwd(x, weight, bias, z, dy, *, groups=1, eps=1e-5, rms=False, workspace=None, stream=None):
    """Gradients of layer_norm_fwd for the output gradient dy (like x).  Returns a dict: dx, dz like x
    in dy's dtype (dz None without z); dweight, dbias (D) fp32, also where weight or bias is None."""
    torch = _torch()
    dev, code, ins, sizes = _norm_inputs(x, weight, bias, z, groups)
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch.Tensor")
    shape, gdt, gcode = x.shape, dy.dtype, _dtype_code(dy)
    dyp = _plain(dy, "dy", shape, gdt, dev)
    with _there(dev, stream):
        sums = torch.empty((2, shape[1]), dtype=torch.float32, device=dev).unbind()
        out = {"dx": torch.empty_like(dy), "dz": None if z is None else torch.empty_like(dy),
               "dweight": sums[0], "dbias": sums[1]}
        workspace = _workspace(workspace, layer_norm_bwd_workspace_size(*sizes[:4]), dev)
        st = lib().mamba_layer_norm_bwd(*ins, dyp, *[_addr(t) for t in out.values()], *sizes, eps, code, gcode,
                                        FLAG_RMS if rms else 0, _addr(workspace), _nbytes(workspace),
                                        _raw_stream(dev, stream))
    if st != 0:
        raise MambaError(st, "mamba_layer_norm_bwd")
    return out
