"""ctypes binding of libssmscan.so: argument marshalling only.

Every step of the scan runs in the library's CUDA kernels; this module only
checks tensor metadata, allocates outputs/workspace with torch when the
caller does not pass them, and forwards raw device pointers and the current
CUDA stream. There is no CPU fallback: without the built library (or without
a GPU) calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import build as _build

SSM_DTYPE_F32, SSM_DTYPE_BF16 = 0, 1
_STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported size or dtype",
           -3: "workspace missing or too small", -4: "CUDA error",
           -5: "a kernel wait timed out"}


class SsmError(RuntimeError):
    def __init__(self, code: int, where: str, with_detail: bool = False):
        self.code = code
        detail = ""
        if (with_detail or code in (-4, -5)) and _lib is not None:
            detail = _lib.ssm_last_error_detail().decode(errors="replace")
        msg = f"{where}: {_STATUS.get(code, 'unknown status')} ({code})"
        super().__init__(msg + (f": {detail}" if detail else ""))


class ScanPlan(ctypes.Structure):
    _fields_ = [("segments", ctypes.c_int32), ("segment_steps", ctypes.c_int32),
                ("channel_tiles", ctypes.c_int32), ("channels_per_cta", ctypes.c_int32),
                ("ctas_carry", ctypes.c_int32), ("ctas_main", ctypes.c_int32),
                ("kernels", ctypes.c_int32), ("workspace_bytes", ctypes.c_int64)]


_lib = None
_VP = ctypes.c_void_p
_I64 = ctypes.c_int64


def lib() -> ctypes.CDLL:
    """Load libssmscan.so from the package directory, or the build named by
    $SSM_SCAN_LIBRARY (raises if absent)."""
    global _lib
    if _lib is None:
        # SSM_SCAN_LIBRARY may point at another build of the same library
        path = os.environ.get("SSM_SCAN_LIBRARY") or _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m selective_state_space_39_b200.build`"
                " (the CUDA library is required; there is no CPU fallback)")
        L = ctypes.CDLL(path)
        L.ssm_scan_version.restype = ctypes.c_int
        L.ssm_status_string.restype = ctypes.c_char_p
        L.ssm_status_string.argtypes = [ctypes.c_int]
        L.ssm_last_error_detail.restype = ctypes.c_char_p
        L.ssm_last_error_detail.argtypes = []
        L.ssm_scan_workspace_bytes.restype = ctypes.c_size_t
        L.ssm_scan_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int]
        L.ssm_scan_plan.restype = ctypes.c_int
        L.ssm_scan_plan.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(ScanPlan)]
        L.ssm_scan_fwd.restype = ctypes.c_int
        L.ssm_scan_fwd.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _VP, _VP, _VP, _VP, _VP,
                                   _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP,
                                   ctypes.c_size_t, _VP]
        L.ssm_scan_fwd_zoh.restype = ctypes.c_int
        L.ssm_scan_fwd_zoh.argtypes = L.ssm_scan_fwd.argtypes
        L.ssm_scan_fwd_noalloc.restype = ctypes.c_int
        L.ssm_scan_fwd_noalloc.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _VP, _VP, _VP,
                                           _VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP,
                                           _VP]
        L.ssm_scan_status.restype = ctypes.c_int
        L.ssm_scan_status.argtypes = [_VP, ctypes.c_size_t, _I64, _I64, _I64, _I64, ctypes.c_int,
                                      _VP]
        L.ssm_scan_status_noalloc.restype = ctypes.c_int
        L.ssm_scan_status_noalloc.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _VP]
        L.ssm_scan_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ssm_scan_bwd_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int]
        L.ssm_scan_bwd.restype = ctypes.c_int
        L.ssm_scan_bwd.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int] + [_VP] * 8 + \
            [ctypes.c_int] + [_VP] * 13 + [ctypes.c_size_t, _VP]
        L.ssm_conv1d_silu_fwd.restype = ctypes.c_int
        L.ssm_conv1d_silu_fwd.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _VP, _VP, _VP,
                                          ctypes.c_int, _VP, _VP]
        L.ssm_conv1d_silu_update.restype = ctypes.c_int
        L.ssm_conv1d_silu_update.argtypes = [_I64, _I64, _I64, ctypes.c_int, _VP, _VP, _VP, _VP,
                                             ctypes.c_int, _VP, _VP]
        L.ssm_conv1d_silu_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ssm_conv1d_silu_bwd_workspace_bytes.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int]
        L.ssm_conv1d_silu_bwd.restype = ctypes.c_int
        L.ssm_conv1d_silu_bwd.argtypes = [_I64, _I64, _I64, _I64, ctypes.c_int, _VP, _VP, _VP,
                                          ctypes.c_int, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t,
                                          _VP]
        L.ssm_state_update.restype = ctypes.c_int
        L.ssm_state_update.argtypes = [_I64, _I64, _I64, ctypes.c_int, _VP, _VP, _VP, _VP, _VP,
                                       _VP, _VP, _VP, _VP, ctypes.c_int, _VP, _VP]
        L.ssm_delta_sum.restype = ctypes.c_int
        L.ssm_delta_sum.argtypes = [_I64, _I64, _I64, ctypes.c_int, _VP, _VP, ctypes.c_int, _VP,
                                    _VP]
        L.ssm_compose_carries.restype = ctypes.c_int
        L.ssm_compose_carries.argtypes = [_I64, _I64, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP]
        L.ssm_state_update_zoh.restype = ctypes.c_int
        L.ssm_state_update_zoh.argtypes = L.ssm_state_update.argtypes
        L.ssm_ssd_state_update.restype = ctypes.c_int
        L.ssm_ssd_state_update.argtypes = [_I64] * 4 + [ctypes.c_int] + [_VP] * 8 + \
            [ctypes.c_int, _VP, _VP]
        L.ssm_ssd_scan_status.restype = ctypes.c_int
        L.ssm_ssd_scan_status.argtypes = [_VP]
        L.ssm_ssd_scan_fwd.restype = ctypes.c_int
        L.ssm_ssd_scan_fwd.argtypes = [_I64] * 5 + [ctypes.c_int] + [_VP] * 7 + \
            [ctypes.c_int, _VP, _VP, _VP, _VP]
        L.ssm_gated_delta_workspace_bytes.restype = ctypes.c_size_t
        L.ssm_gated_delta_workspace_bytes.argtypes = [_I64] * 6 + [ctypes.c_int]
        L.ssm_gated_delta_fwd.restype = ctypes.c_int
        L.ssm_gated_delta_fwd.argtypes = [_I64] * 6 + [ctypes.c_int] + [_VP] * 7 + \
            [ctypes.c_int] * 3 + [ctypes.c_float] + [_VP] * 4 + [ctypes.c_size_t, _VP]
        L.ssm_gated_delta_update.restype = ctypes.c_int
        L.ssm_gated_delta_update.argtypes = [_I64] * 5 + [ctypes.c_int] + [_VP] * 8 + \
            [ctypes.c_int] * 3 + [ctypes.c_float, _VP, _VP]
        L.ssm_gated_delta_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ssm_gated_delta_bwd_workspace_bytes.argtypes = [_I64] * 6 + [ctypes.c_int]
        L.ssm_gated_delta_bwd.restype = ctypes.c_int
        L.ssm_gated_delta_bwd.argtypes = [_I64] * 6 + [ctypes.c_int] + [_VP] * 7 + \
            [ctypes.c_int] * 3 + [ctypes.c_float] + [_VP] * 12 + [ctypes.c_size_t, _VP]
        L.ssm_gated_delta_status.restype = ctypes.c_int
        L.ssm_gated_delta_status.argtypes = [_VP]
        L.ssm_gated_norm_fwd.restype = ctypes.c_int
        L.ssm_gated_norm_fwd.argtypes = [_I64] * 3 + [ctypes.c_int] * 2 + \
            [_VP, _VP, ctypes.c_float, _VP, ctypes.c_int, _VP, ctypes.c_float, _VP, _VP, _VP]
        L.ssm_gated_norm_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.ssm_gated_norm_bwd_workspace_bytes.argtypes = [_I64] * 3 + [ctypes.c_int]
        L.ssm_gated_norm_bwd.restype = ctypes.c_int
        L.ssm_gated_norm_bwd.argtypes = [_I64] * 3 + [ctypes.c_int] * 2 + \
            [_VP, ctypes.c_float, _VP, ctypes.c_int, _VP, ctypes.c_float] + [_VP] * 7 + \
            [ctypes.c_size_t, _VP]
        _lib = L
    return _lib


def _io_code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return SSM_DTYPE_F32
    if dtype == torch.bfloat16:
        return SSM_DTYPE_BF16
    raise TypeError(f"io tensors must be float32 or bfloat16, got {dtype}")


def _ptr(t, name, dtype=None, shape=None, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _stream_ptr(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def scan_plan(batch, seqlen, dim, dstate, dtype=torch.bfloat16) -> ScanPlan:
    out = ScanPlan()
    rc = lib().ssm_scan_plan(batch, seqlen, dim, dstate, _io_code(dtype), ctypes.byref(out))
    if rc != 0:
        raise SsmError(rc, "ssm_scan_plan")
    return out


def scan_workspace_bytes(batch, seqlen, dim, dstate, dtype=torch.bfloat16) -> int:
    return int(lib().ssm_scan_workspace_bytes(batch, seqlen, dim, dstate, _io_code(dtype)))


def ssm_scan_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True, h0=None,
                 y=None, h_last=None, workspace=None, return_last_state=True, stream=None,
                 zoh=False, return_y=True):
    """Selective scan through ssm_scan_fwd of libssmscan.so (ssm_scan_fwd_zoh
    with ``zoh=True``: the exact zero-order-hold input term).

    x, delta, z: (batch, L, dim); B, C: (batch, L, N) -- all float32 or all
    bfloat16. A: (dim, N), D and delta_bias: (dim,), h0: (batch, dim, N),
    float32. Returns (y, h_last); h_last is None when not requested, y is None
    with ``return_y=False`` (the final state only: no y is written)."""
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    batch, L, dim = x.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be (dim, dstate)")
    N = A.shape[1]
    dev = x.device
    io = _io_code(x.dtype)
    bld, bln = (batch, L, dim), (batch, L, N)
    args_io = [_ptr(x, "x", x.dtype, bld), _ptr(delta, "delta", x.dtype, bld, dev)]
    pA = _ptr(A, "A", torch.float32, (dim, N), dev)
    pB = _ptr(B, "B", x.dtype, bln, dev)
    pC = _ptr(C, "C", x.dtype, bln, dev)
    pD = _ptr(D, "D", torch.float32, (dim,), dev)
    pz = _ptr(z, "z", x.dtype, bld, dev)
    pbias = _ptr(delta_bias, "delta_bias", torch.float32, (dim,), dev)
    ph0 = _ptr(h0, "h0", torch.float32, (batch, dim, N), dev)
    if y is None and return_y:
        y = torch.empty(bld, dtype=x.dtype, device=dev)
    py = _ptr(y, "y", x.dtype, bld, dev)
    if h_last is None and (return_last_state or not return_y):
        h_last = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    ph = _ptr(h_last, "h_last", torch.float32, (batch, dim, N), dev)
    with torch.cuda.device(dev):
        need = scan_workspace_bytes(batch, L, dim, N, x.dtype)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        pws = _ptr(workspace, "workspace", None, None, dev)
        fn = lib().ssm_scan_fwd_zoh if zoh else lib().ssm_scan_fwd
        rc = fn(batch, L, dim, N, io, args_io[0], args_io[1], pA, pB, pC, pD, pz,
                pbias, 1 if softplus else 0, ph0, py, ph, pws,
                workspace.numel() * workspace.element_size(), _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_scan_fwd_zoh" if zoh else "ssm_scan_fwd")
    return y, h_last


def scan_bwd_workspace_bytes(batch, seqlen, dim, dstate, dtype=torch.bfloat16) -> int:
    return int(lib().ssm_scan_bwd_workspace_bytes(batch, seqlen, dim, dstate, _io_code(dtype)))


def ssm_scan_bwd(x, delta, A, B, C, dy, D=None, z=None, delta_bias=None, softplus=True, h0=None,
                 dh_last=None, workspace=None, want_dD=True, want_ddelta_bias=True, want_dh0=True,
                 stream=None):
    """Gradients of the selective scan through ssm_scan_bwd of libssmscan.so,
    for the loss sum(dy * y) + sum(dh_last * h_last) (dh_last may be None).

    Inputs as for ssm_scan_fwd, plus dy (batch, L, dim) in the io dtype and
    dh_last (batch, dim, N) float32. Returns a dict: dx, ddelta, dz (io
    dtype; dz None without z), dA (dim, N), dB, dC (batch, L, N), dD,
    ddelta_bias (dim,), dh0 (batch, dim, N), all float32 except the first
    three (a gradient not asked for is None)."""
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    batch, L, dim = x.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be (dim, dstate)")
    N = A.shape[1]
    dev = x.device
    io = _io_code(x.dtype)
    bld, bln, bdn = (batch, L, dim), (batch, L, N), (batch, dim, N)
    f32 = torch.float32
    ins = [_ptr(x, "x", x.dtype, bld), _ptr(delta, "delta", x.dtype, bld, dev),
           _ptr(A, "A", f32, (dim, N), dev), _ptr(B, "B", x.dtype, bln, dev),
           _ptr(C, "C", x.dtype, bln, dev), _ptr(D, "D", f32, (dim,), dev),
           _ptr(z, "z", x.dtype, bld, dev), _ptr(delta_bias, "delta_bias", f32, (dim,), dev)]
    ph0 = _ptr(h0, "h0", f32, bdn, dev)
    pdy = _ptr(dy, "dy", x.dtype, bld, dev)
    pdh = _ptr(dh_last, "dh_last", f32, bdn, dev)
    g = {"dx": torch.empty(bld, dtype=x.dtype, device=dev),
         "ddelta": torch.empty(bld, dtype=x.dtype, device=dev),
         "dz": torch.empty(bld, dtype=x.dtype, device=dev) if z is not None else None,
         "dA": torch.empty((dim, N), dtype=f32, device=dev),
         "dB": torch.empty(bln, dtype=f32, device=dev),
         "dC": torch.empty(bln, dtype=f32, device=dev),
         "dD": torch.empty((dim,), dtype=f32, device=dev) if want_dD else None,
         "ddelta_bias": torch.empty((dim,), dtype=f32, device=dev) if want_ddelta_bias else None,
         "dh0": torch.empty(bdn, dtype=f32, device=dev) if want_dh0 else None}
    P = {k: (v.data_ptr() if v is not None else None) for k, v in g.items()}
    with torch.cuda.device(dev):
        need = scan_bwd_workspace_bytes(batch, L, dim, N, x.dtype)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        pws = _ptr(workspace, "workspace", None, None, dev)
        rc = lib().ssm_scan_bwd(batch, L, dim, N, io, *ins, 1 if softplus else 0, ph0, pdy, pdh,
                                P["dx"], P["ddelta"], P["dA"], P["dB"], P["dC"], P["dD"],
                                P["dz"], P["ddelta_bias"], P["dh0"], pws,
                                workspace.numel() * workspace.element_size(),
                                _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_scan_bwd", with_detail=True)
    return g


def ssm_conv1d_silu_fwd(x, w, bias=None, silu=True, out=None, stream=None):
    """The Mamba block's causal depthwise conv1d (+ SiLU) through
    ssm_conv1d_silu_fwd of libssmscan.so. x: (batch, L, dim) float32 or
    bfloat16; w: (dim, width) float32; bias: (dim,) float32. Returns out
    (batch, L, dim) in x's dtype."""
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be (batch, seqlen, dim) and w (dim, width)")
    batch, L, dim = x.shape
    width = w.shape[1]
    dev = x.device
    px = _ptr(x, "x", x.dtype, (batch, L, dim))
    pw = _ptr(w, "w", torch.float32, (dim, width), dev)
    pb = _ptr(bias, "bias", torch.float32, (dim,), dev)
    if out is None:
        out = torch.empty((batch, L, dim), dtype=x.dtype, device=dev)
    po = _ptr(out, "out", x.dtype, (batch, L, dim), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_conv1d_silu_fwd(batch, L, dim, width, _io_code(x.dtype), px, pw, pb,
                                       1 if silu else 0, po, _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_conv1d_silu_fwd", with_detail=True)
    return out


def ssm_conv1d_silu_update(conv_state, x, w, bias=None, silu=True, out=None, stream=None):
    """One decode step of the causal conv through ssm_conv1d_silu_update of
    libssmscan.so: conv_state (batch, dim, width-1) in x's dtype (the last
    inputs, oldest first) is updated in place; returns out (batch, dim)."""
    if x.dim() != 2 or conv_state.dim() != 3:
        raise ValueError("x must be (batch, dim) and conv_state (batch, dim, width-1)")
    batch, dim = x.shape
    width = conv_state.shape[2] + 1
    dev = x.device
    ps = _ptr(conv_state, "conv_state", x.dtype, (batch, dim, width - 1), dev)
    px = _ptr(x, "x", x.dtype, (batch, dim))
    pw = _ptr(w, "w", torch.float32, (dim, width), dev)
    pb = _ptr(bias, "bias", torch.float32, (dim,), dev)
    if out is None:
        out = torch.empty((batch, dim), dtype=x.dtype, device=dev)
    po = _ptr(out, "out", x.dtype, (batch, dim), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_conv1d_silu_update(batch, dim, width, _io_code(x.dtype), ps, px, pw, pb,
                                          1 if silu else 0, po, _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_conv1d_silu_update", with_detail=True)
    return out


def conv1d_silu_bwd_workspace_bytes(batch, seqlen, dim, width, dtype=torch.bfloat16) -> int:
    return int(lib().ssm_conv1d_silu_bwd_workspace_bytes(batch, seqlen, dim, width,
                                                         _io_code(dtype)))


def ssm_conv1d_silu_bwd(x, w, dout, bias=None, silu=True, workspace=None, stream=None):
    """Gradients of sum(dout * out) for ssm_conv1d_silu_fwd: returns a dict
    dx (batch, L, dim) in x's dtype, dw (dim, width) and dbias (dim,) float32."""
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be (batch, seqlen, dim) and w (dim, width)")
    batch, L, dim = x.shape
    width = w.shape[1]
    dev = x.device
    px = _ptr(x, "x", x.dtype, (batch, L, dim))
    pw = _ptr(w, "w", torch.float32, (dim, width), dev)
    pb = _ptr(bias, "bias", torch.float32, (dim,), dev)
    pg = _ptr(dout, "dout", x.dtype, (batch, L, dim), dev)
    g = {"dx": torch.empty((batch, L, dim), dtype=x.dtype, device=dev),
         "dw": torch.empty((dim, width), dtype=torch.float32, device=dev),
         "dbias": torch.empty((dim,), dtype=torch.float32, device=dev)}
    with torch.cuda.device(dev):
        need = conv1d_silu_bwd_workspace_bytes(batch, L, dim, width, x.dtype)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        pws = _ptr(workspace, "workspace", None, None, dev)
        rc = lib().ssm_conv1d_silu_bwd(batch, L, dim, width, _io_code(x.dtype), px, pw, pb,
                                       1 if silu else 0, pg, g["dx"].data_ptr(),
                                       g["dw"].data_ptr(), g["dbias"].data_ptr(), pws,
                                       workspace.numel() * workspace.element_size(),
                                       _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_conv1d_silu_bwd", with_detail=True)
    return g


def ssm_delta_sum(delta, delta_bias=None, softplus=True, out=None, stream=None):
    """dsum (batch, dim) float32 = sum over the sequence of Delta =
    softplus(delta + delta_bias), through ssm_delta_sum of libssmscan.so."""
    if delta.dim() != 3:
        raise ValueError("delta must be (batch, seqlen, dim)")
    batch, L, dim = delta.shape
    dev = delta.device
    pd = _ptr(delta, "delta", delta.dtype, (batch, L, dim))
    pb = _ptr(delta_bias, "delta_bias", torch.float32, (dim,), dev)
    if out is None:
        out = torch.empty((batch, dim), dtype=torch.float32, device=dev)
    po = _ptr(out, "out", torch.float32, (batch, dim), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_delta_sum(batch, L, dim, _io_code(delta.dtype), pd, pb, 1 if softplus else 0,
                                 po, _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_delta_sum")
    return out


def ssm_compose_carries(rank, A, hend_all, dsum_all, h0=None, out=None, stream=None):
    """The state entering chunk `rank` of a sequence cut into chunks: h0 (or
    zero) carried through chunks 0..rank-1, each given by its end state from
    zero (hend_all[r], (batch, dim, N)) and its sum of Delta (dsum_all[r],
    (batch, dim)), through ssm_compose_carries of libssmscan.so."""
    R, batch, dim, N = hend_all.shape
    dev = hend_all.device
    pA = _ptr(A, "A", torch.float32, (dim, N), dev)
    ph = _ptr(hend_all, "hend_all", torch.float32, (R, batch, dim, N), dev)
    pd = _ptr(dsum_all, "dsum_all", torch.float32, (R, batch, dim), dev)
    p0 = _ptr(h0, "h0", torch.float32, (batch, dim, N), dev)
    if not 0 <= rank <= R:
        raise ValueError("rank out of range")
    if out is None:
        out = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    po = _ptr(out, "out", torch.float32, (batch, dim, N), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_compose_carries(rank, batch, dim, N, pA, p0, ph, pd, po,
                                       _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_compose_carries")
    return out


def ssm_scan_fwd_noalloc(x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                         h0=None, y=None, h_last=None, return_last_state=True, stream=None):
    """The selective scan through ssm_scan_fwd_noalloc of libssmscan.so.

    For callers that cannot allocate device memory around the call: the
    library takes its scratch from a 16 MiB array it reserves on each GPU, so
    apart from the outputs (allocated here only when not passed in) nothing
    is allocated. Problems needing more scratch raise SsmError (-3). Calls
    that may overlap on the GPU share that scratch and must be ordered by the
    caller. Same arguments and results as ssm_scan_fwd."""
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    batch, L, dim = x.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError("A must be (dim, dstate)")
    N = A.shape[1]
    dev = x.device
    bld, bln = (batch, L, dim), (batch, L, N)
    px = _ptr(x, "x", x.dtype, bld)
    pdl = _ptr(delta, "delta", x.dtype, bld, dev)
    pA = _ptr(A, "A", torch.float32, (dim, N), dev)
    pB = _ptr(B, "B", x.dtype, bln, dev)
    pC = _ptr(C, "C", x.dtype, bln, dev)
    pD = _ptr(D, "D", torch.float32, (dim,), dev)
    pz = _ptr(z, "z", x.dtype, bld, dev)
    pbias = _ptr(delta_bias, "delta_bias", torch.float32, (dim,), dev)
    ph0 = _ptr(h0, "h0", torch.float32, (batch, dim, N), dev)
    if y is None:
        y = torch.empty(bld, dtype=x.dtype, device=dev)
    py = _ptr(y, "y", x.dtype, bld, dev)
    if h_last is None and return_last_state:
        h_last = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    ph = _ptr(h_last, "h_last", torch.float32, (batch, dim, N), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_scan_fwd_noalloc(batch, L, dim, N, _io_code(x.dtype), px, pdl, pA, pB, pC,
                                        pD, pz, pbias, 1 if softplus else 0, ph0, py, ph,
                                        _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_scan_fwd_noalloc", with_detail=True)
    return y, h_last


def ssm_scan_status(workspace, batch, seqlen, dim, dstate, dtype=torch.bfloat16, stream=None):
    """Synchronise the stream and return the status code of the last scan that
    used `workspace` (0 = every CTA finished; -5 = a bounded wait timed out)."""
    dev = workspace.device
    with torch.cuda.device(dev):
        return int(lib().ssm_scan_status(workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), batch,
                                         seqlen, dim, dstate, _io_code(dtype),
                                         _stream_ptr(stream, dev)))


def ssm_scan_status_noalloc(batch, seqlen, dim, dstate, dtype=torch.bfloat16, device=None,
                            stream=None):
    """Synchronise the stream and return the status code of the last
    ssm_scan_fwd_noalloc call on the device (0 = every CTA finished; -5 = a
    bounded wait timed out), read from the library's reserved scratch."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return int(lib().ssm_scan_status_noalloc(batch, seqlen, dim, dstate, _io_code(dtype),
                                                 _stream_ptr(stream, dev)))


def ssm_ssd_scan_status(device=None, stream=None):
    """Synchronise the stream and return 0, or -5 if a CTA of an SSD scan on
    the device gave up a bounded wait since the last call (the flag is then
    cleared)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return int(lib().ssm_ssd_scan_status(_stream_ptr(stream, dev)))


def ssm_state_update(state, x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                     y=None, stream=None, zoh=False):
    """One decode step through ssm_state_update of libssmscan.so
    (ssm_state_update_zoh with ``zoh=True``); updates the float32 state
    (batch, dim, N) in place and returns y (batch, dim)."""
    if state.dim() != 3:
        raise ValueError("state must be (batch, dim, dstate)")
    batch, dim, N = state.shape
    dev = state.device
    io = _io_code(x.dtype)
    bd, bn = (batch, dim), (batch, N)
    ps = _ptr(state, "state", torch.float32, (batch, dim, N))
    px = _ptr(x, "x", x.dtype, bd, dev)
    pdl = _ptr(delta, "delta", x.dtype, bd, dev)
    pA = _ptr(A, "A", torch.float32, (dim, N), dev)
    pB = _ptr(B, "B", x.dtype, bn, dev)
    pC = _ptr(C, "C", x.dtype, bn, dev)
    pD = _ptr(D, "D", torch.float32, (dim,), dev)
    pz = _ptr(z, "z", x.dtype, bd, dev)
    pbias = _ptr(delta_bias, "delta_bias", torch.float32, (dim,), dev)
    if y is None:
        y = torch.empty(bd, dtype=x.dtype, device=dev)
    py = _ptr(y, "y", x.dtype, bd, dev)
    with torch.cuda.device(dev):
        fn = lib().ssm_state_update_zoh if zoh else lib().ssm_state_update
        rc = fn(batch, dim, N, io, ps, px, pdl, pA, pB, pC, pD, pz, pbias,
                1 if softplus else 0, py, _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_state_update_zoh" if zoh else "ssm_state_update")
    return y


def ssm_ssd_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, softplus=True, h0=None,
                     return_last_state=False, y=None, stream=None, h_last=None):
    """The multi-head SSD scan through ssm_ssd_scan_fwd of libssmscan.so:
    x (batch, L, heads, headdim) bf16, dt (batch, L, heads) bf16, A (heads,)
    fp32, B, C (batch, L, dstate) bf16, D and dt_bias (heads,) fp32 or None,
    h0 (batch, heads, headdim, dstate) fp32 or None. Returns y (and h_last
    with ``return_last_state``; ``h_last`` may be given, and may be h0)."""
    if x.dim() != 4:
        raise ValueError("x must be (batch, seqlen, heads, headdim)")
    batch, L, H, P = x.shape
    N = B.shape[-1]
    dev = x.device
    io = _io_code(x.dtype)
    px = _ptr(x, "x", x.dtype)
    pdt = _ptr(dt, "dt", x.dtype, (batch, L, H), dev)
    pA = _ptr(A, "A", torch.float32, (H,), dev)
    pB = _ptr(B, "B", x.dtype, (batch, L, N), dev)
    pC = _ptr(C, "C", x.dtype, (batch, L, N), dev)
    pD = _ptr(D, "D", torch.float32, (H,), dev)
    pbias = _ptr(dt_bias, "dt_bias", torch.float32, (H,), dev)
    ph0 = _ptr(h0, "h0", torch.float32, (batch, H, P, N), dev)
    if y is None:
        y = torch.empty((batch, L, H, P), dtype=x.dtype, device=dev)
    py = _ptr(y, "y", x.dtype, (batch, L, H, P), dev)
    if h_last is None and return_last_state:
        h_last = torch.empty((batch, H, P, N), dtype=torch.float32, device=dev)
    ph = _ptr(h_last, "h_last", torch.float32, (batch, H, P, N), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_ssd_scan_fwd(batch, L, H, P, N, io, px, pdt, pA, pB, pC, pD, pbias,
                                    1 if softplus else 0, ph0, py, ph, _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_ssd_scan_fwd", with_detail=True)
    return (y, h_last) if return_last_state else y


def ssm_ssd_state_update(state, x, dt, A, B, C, D=None, dt_bias=None, softplus=True, y=None,
                         stream=None):
    """One SSD decode step through ssm_ssd_state_update of libssmscan.so:
    updates the float32 state (batch, heads, headdim, dstate) in place and
    returns y (batch, heads, headdim) in x's dtype."""
    if state.dim() != 4:
        raise ValueError("state must be (batch, heads, headdim, dstate)")
    batch, H, P, N = state.shape
    dev = state.device
    io = _io_code(x.dtype)
    ps = _ptr(state, "state", torch.float32)
    px = _ptr(x, "x", x.dtype, (batch, H, P), dev)
    pdt = _ptr(dt, "dt", x.dtype, (batch, H), dev)
    pA = _ptr(A, "A", torch.float32, (H,), dev)
    pB = _ptr(B, "B", x.dtype, (batch, N), dev)
    pC = _ptr(C, "C", x.dtype, (batch, N), dev)
    pD = _ptr(D, "D", torch.float32, (H,), dev)
    pbias = _ptr(dt_bias, "dt_bias", torch.float32, (H,), dev)
    if y is None:
        y = torch.empty((batch, H, P), dtype=x.dtype, device=dev)
    py = _ptr(y, "y", x.dtype, (batch, H, P), dev)
    with torch.cuda.device(dev):
        rc = lib().ssm_ssd_state_update(batch, H, P, N, io, ps, px, pdt, pA, pB, pC, pD, pbias,
                                        1 if softplus else 0, py, _stream_ptr(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_ssd_state_update", with_detail=True)
    return y



# The calls below are made once per layer and generated token, so their checks
# are kept to one test per tensor; what is wrong with one is found afterwards.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _at(t, name, dtype, shape, dev):
    """The pointer of a tensor that is as it must be, or _ptr's error."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev.index
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, name, dtype, shape, dev)


def _cuda_device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return dev


def _stream_of(stream, dev):
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev.index)
    return _stream_ptr(stream, dev)


def _streamed(fn):
    """Runs a call given a stream with that stream current, so that its results
    and its workspace are allocated there too. The stream is one of the tensors'
    device: any object's pointer (cuda_stream) is taken as that, a torch stream
    of another device is refused."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        dev = next((t.device for t in (*args, *kw.values())
                    if isinstance(t, torch.Tensor) and t.is_cuda), None)
        if dev is None:  # refused by the call itself
            return fn(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream.cuda_stream, device=dev)
        elif stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _on(dev, fn, *args):
    """fn(*args) with dev current."""
    if torch.cuda.current_device() == dev.index:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


@functools.lru_cache(maxsize=256)
def _bytes_of(fn, *sizes):
    """What a C function of sizes alone answers (the call costs as much as a
    third of a launch)."""
    return int(getattr(lib(), fn)(*sizes))


def _scratch(like, need):
    return like.new_empty(need, dtype=torch.uint8)


def _delta_sizes(q, v, tokens):
    """(batch, L, heads, key heads, headdim, dstate) of v (batch[, L], heads,
    headdim) and q (batch[, L], key heads, dstate)."""
    vs, qs = v.shape, q.shape
    if len(qs) != 3 + tokens or len(vs) != 3 + tokens:
        raise ValueError("q and v must be (batch, seqlen, heads, width)" if tokens
                         else "q and v must be (batch, heads, width)")
    return vs[0], vs[1] if tokens else 1, vs[-2], qs[-2], vs[-1], qs[-1]


def _delta_inputs(sizes, dev, q, k, v, dt, A, beta, dt_bias, tokens):
    """Checked pointers of a gated delta rule call's inputs, in the C order."""
    B, L, H, Hk, P, N = sizes
    ty = v.dtype
    f32 = torch.float32
    qk, gate = ((B, L, Hk, N), (B, L, H)) if tokens else ((B, Hk, N), (B, H))
    if dt_bias is not None:
        try:  # one test of everything; what is wrong is found below
            i = dev.index
            if (q.shape == qk and k.shape == qk and dt.shape == gate and beta.shape == gate
                    and A.shape == (H,) and dt_bias.shape == (H,)
                    and q.dtype is ty and k.dtype is ty and dt.dtype is ty and beta.dtype is ty
                    and A.dtype is f32 and dt_bias.dtype is f32
                    and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
                    and dt.is_contiguous() and beta.is_contiguous() and A.is_contiguous()
                    and dt_bias.is_contiguous()
                    and q.get_device() == i and k.get_device() == i and dt.get_device() == i
                    and beta.get_device() == i and A.get_device() == i
                    and dt_bias.get_device() == i):
                return (q.data_ptr(), k.data_ptr(), v.data_ptr(), dt.data_ptr(), A.data_ptr(),
                        beta.data_ptr(), dt_bias.data_ptr())
        except AttributeError:
            pass
    return (_at(q, "q", ty, qk, dev), _at(k, "k", ty, qk, dev), _at(v, "v", ty, v.shape, dev),
            _at(dt, "dt", ty, gate, dev), _at(A, "A", f32, (H,), dev),
            _at(beta, "beta", ty, gate, dev), _at(dt_bias, "dt_bias", f32, (H,), dev))


def gated_delta_workspace_bytes(batch, seqlen, nheads, nkheads, headdim, dstate,
                                dtype=torch.bfloat16) -> int:
    return int(lib().ssm_gated_delta_workspace_bytes(batch, seqlen, nheads, nkheads, headdim,
                                                     dstate, _io_code(dtype)))


def gated_delta_bwd_workspace_bytes(batch, seqlen, nheads, nkheads, headdim, dstate,
                                    dtype=torch.bfloat16) -> int:
    return int(lib().ssm_gated_delta_bwd_workspace_bytes(batch, seqlen, nheads, nkheads, headdim,
                                                         dstate, _io_code(dtype)))


@_streamed
def ssm_gated_delta_fwd(q, k, v, dt, A, beta, dt_bias=None, softplus=True, beta_sigmoid=True,
                        qk_norm=True, scale=None, h0=None, y=None, h_last=None, workspace=None,
                        return_last_state=True, stream=None):
    """The gated delta rule over a sequence through ssm_gated_delta_fwd of
    libssmscan.so: q, k (batch, L, key heads, dstate), v (batch, L, heads,
    headdim), dt, beta (batch, L, heads), all float32 or all bfloat16; A and
    dt_bias (heads,), h0 (batch, heads, headdim, dstate) float32. ``scale``
    defaults to dstate ** -0.5. Returns (y, h_last); h_last is None when not
    requested, and may be given (it may be h0)."""
    dev = _cuda_device(v, "v")
    sizes = _delta_sizes(q, v, True)
    B, L, H, Hk, P, N = sizes
    io, st, f32 = _io_code(v.dtype), (B, H, P, N), torch.float32
    ins = _delta_inputs(sizes, dev, q, k, v, dt, A, beta, dt_bias, True)
    ph0 = _at(h0, "h0", f32, st, dev)
    if y is None:
        y = torch.empty_like(v)
    if h_last is None and return_last_state:
        h_last = torch.empty_like(h0) if h0 is not None else torch.empty(st, dtype=f32, device=dev)
    if workspace is None:
        need = _bytes_of("ssm_gated_delta_workspace_bytes", *sizes, io)
        workspace = _scratch(v, need) if need else None
    rc = _on(dev, lib().ssm_gated_delta_fwd, *sizes, io, *ins, 1 if softplus else 0,
             1 if beta_sigmoid else 0, 1 if qk_norm else 0, N ** -0.5 if scale is None else scale,
             ph0, _at(y, "y", v.dtype, v.shape, dev), _at(h_last, "h_last", f32, st, dev),
             _ptr(workspace, "workspace", None, None, dev),
             workspace.numel() * workspace.element_size() if workspace is not None else 0,
             _stream_of(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_gated_delta_fwd", with_detail=True)
    return y, h_last


@_streamed
def ssm_gated_delta_update(state, q, k, v, dt, A, beta, dt_bias=None, softplus=True,
                           beta_sigmoid=True, qk_norm=True, scale=None, y=None, stream=None):
    """One decode step of the gated delta rule through ssm_gated_delta_update
    of libssmscan.so: updates the float32 state (batch, heads, headdim, dstate)
    in place and returns y (batch, heads, headdim) in v's dtype; q, k (batch,
    key heads, dstate), v (batch, heads, headdim), dt, beta (batch, heads)."""
    dev = _cuda_device(v, "v")
    sizes = _delta_sizes(q, v, False)
    B, _, H, Hk, P, N = sizes
    ins = _delta_inputs(sizes, dev, q, k, v, dt, A, beta, dt_bias, False)
    if y is None:
        y = torch.empty_like(v)
    rc = _on(dev, lib().ssm_gated_delta_update, B, H, Hk, P, N, _io_code(v.dtype),
             _at(state, "state", torch.float32, (B, H, P, N), dev), *ins, 1 if softplus else 0,
             1 if beta_sigmoid else 0, 1 if qk_norm else 0, N ** -0.5 if scale is None else scale,
             _at(y, "y", v.dtype, v.shape, dev), _stream_of(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_gated_delta_update", with_detail=True)
    return y


@_streamed
def ssm_gated_delta_bwd(q, k, v, dt, A, beta, dy, dt_bias=None, softplus=True, beta_sigmoid=True,
                        qk_norm=True, scale=None, h0=None, dh_last=None, workspace=None,
                        want_dA=True, want_ddt_bias=True, want_dh0=True, stream=None):
    """Gradients of sum(dy * y) + sum(dh_last * h_last) through
    ssm_gated_delta_bwd of libssmscan.so (bfloat16; inputs as for
    ssm_gated_delta_fwd, dh_last may be None). Returns a dict: dq, dk, dv, ddt,
    dbeta in bfloat16, dA, ddt_bias (heads,) and dh0 in float32 (None when not
    asked for)."""
    dev = _cuda_device(v, "v")
    sizes = _delta_sizes(q, v, True)
    B, L, H, Hk, P, N = sizes
    io, st, f32 = _io_code(v.dtype), (B, H, P, N), torch.float32
    ins = _delta_inputs(sizes, dev, q, k, v, dt, A, beta, dt_bias, True)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "ddt": torch.empty_like(dt), "dbeta": torch.empty_like(beta),
         "dA": torch.empty_like(A) if want_dA else None,
         "ddt_bias": torch.empty((H,), dtype=f32, device=dev) if want_ddt_bias else None,
         "dh0": torch.empty(st, dtype=f32, device=dev) if want_dh0 else None}
    if workspace is None:
        need = _bytes_of("ssm_gated_delta_bwd_workspace_bytes", *sizes, io)
        workspace = _scratch(v, max(need, 1))
    rc = _on(dev, lib().ssm_gated_delta_bwd, *sizes, io, *ins, 1 if softplus else 0,
             1 if beta_sigmoid else 0, 1 if qk_norm else 0, N ** -0.5 if scale is None else scale,
             _at(h0, "h0", f32, st, dev), _at(dy, "dy", v.dtype, v.shape, dev),
             _at(dh_last, "dh_last", f32, st, dev),
             *[t.data_ptr() if t is not None else None for t in g.values()],
             _ptr(workspace, "workspace", None, None, dev),
             workspace.numel() * workspace.element_size(), _stream_of(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_gated_delta_bwd", with_detail=True)
    return g


def ssm_gated_delta_status(device=None, stream=None):
    """Synchronise the stream and return 0, or -5 if a CTA of a chunked gated
    delta rule call on the device gave up a bounded wait since the last call
    (the flag is then cleared)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        return int(lib().ssm_gated_delta_status(_stream_ptr(stream, dev)))


def gated_norm_bwd_workspace_bytes(rows, dim, groups=1, dtype=torch.bfloat16) -> int:
    return int(lib().ssm_gated_norm_bwd_workspace_bytes(rows, dim, groups, _io_code(dtype)))


@_streamed
def ssm_gated_norm_fwd(x, w, z=None, norm_before_gate=False, residual=None, residual_scale=1.0,
                       groups=1, eps=1e-5, y=None, h=None, stream=None):
    """The norm before and after a block through ssm_gated_norm_fwd of
    libssmscan.so: RMSNorm over groups of the last axis of x (..., dim), fp32
    weights w (dim,), the SiLU gate z (x's shape and type) before the norm or
    after it (``norm_before_gate``), and residual + residual_scale * x in front
    of it (residual of x's shape, x's type or float32). Returns (y, h): h is
    the sum (``h`` may be given, and may be residual), or x without a residual."""
    dev = _cuda_device(x, "x")
    shape, ty = x.shape, x.dtype
    if not shape:
        raise ValueError("x must be (..., dim)")
    dim = shape[-1]
    rt = residual.dtype if residual is not None else ty
    if y is None:
        y = torch.empty_like(x)
    if residual is None:
        if h is not None:
            raise ValueError("h is an output only with a residual")
    elif h is None:
        h = torch.empty_like(residual)
    rc = _on(dev, lib().ssm_gated_norm_fwd, x.numel() // dim if dim else 0, dim, groups,
             _io_code(ty), _io_code(rt), _at(x, "x", ty, shape, dev),
             _at(residual, "residual", rt, shape, dev), residual_scale, _at(z, "z", ty, shape, dev),
             1 if norm_before_gate else 0, _at(w, "w", torch.float32, (dim,), dev), eps,
             _at(y, "y", ty, shape, dev), _at(h, "h", rt, shape, dev), _stream_of(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_gated_norm_fwd", with_detail=True)
    return y, (x if residual is None else h)


@_streamed
def ssm_gated_norm_bwd(h, w, dy, z=None, norm_before_gate=False, dh=None, residual=False,
                       residual_scale=1.0, groups=1, eps=1e-5, workspace=None, want_dw=True,
                       stream=None):
    """Gradients of sum(dy * y) + sum(dh * h) through ssm_gated_norm_bwd of
    libssmscan.so, from the h that ssm_gated_norm_fwd returned (x itself without
    a residual). ``residual``: whether there was one (dresidual is returned,
    and dx is residual_scale times it). Returns a dict: dx, dz (dy's type),
    dresidual (h's type), dw (dim,) float32; what does not apply is None."""
    dev = _cuda_device(h, "h")
    shape, ht, ty = h.shape, h.dtype, dy.dtype
    if not shape:
        raise ValueError("h must be (..., dim)")
    if not residual and (ht != ty or residual_scale != 1.0):
        raise ValueError("without a residual h has dy's type and residual_scale is 1")
    dim = shape[-1]
    rows, io = (h.numel() // dim if dim else 0), _io_code(ty)
    g = {"dx": torch.empty_like(dy), "dz": torch.empty_like(dy) if z is not None else None,
         "dresidual": torch.empty_like(h) if residual else None,
         "dw": torch.empty_like(w) if want_dw else None}
    if workspace is None and want_dw:
        need = _bytes_of("ssm_gated_norm_bwd_workspace_bytes", rows, dim, groups, io)
        workspace = _scratch(dy, max(need, 1))
    P = [t.data_ptr() if t is not None else None for t in g.values()]
    rc = _on(dev, lib().ssm_gated_norm_bwd, rows, dim, groups, io, _io_code(ht),
             _at(h, "h", ht, shape, dev), residual_scale, _at(z, "z", ty, shape, dev),
             1 if norm_before_gate else 0, _at(w, "w", torch.float32, (dim,), dev), eps,
             _at(dy, "dy", ty, shape, dev), _at(dh, "dh", ht, shape, dev), P[0], P[2], P[1], P[3],
             _ptr(workspace, "workspace", None, None, dev),
             workspace.numel() * workspace.element_size() if workspace is not None else 0,
             _stream_of(stream, dev))
    if rc != 0:
        raise SsmError(rc, "ssm_gated_norm_bwd", with_detail=True)
    return g
