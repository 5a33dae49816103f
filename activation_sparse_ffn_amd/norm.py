"""The root-mean-square norm between the halves of a decoder layer, with the residual's
addition in the same pass and its output in the input's type or in 8 bits.

    y, h = add_rms_norm(x, residual, weight)                       # h = x + residual, y its norm
    q, scale, h = add_rms_norm(x, residual, weight, quant="int8")  # value: q scale[:, None]
    grads = add_rms_norm_backward(h, g_y, weight, g_h=g_h)

A thin ctypes binding of include/sparse_ffn_norm.h: the arithmetic runs in the
library's HIP kernels, asynchronously on torch's current stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import SFFN_BF16, SFFN_F32, _need_buffer, _ptr, _run, load_library

__all__ = ["add_rms_norm", "add_rms_norm_backward"]

_DTYPES = {torch.bfloat16: SFFN_BF16, torch.float32: SFFN_F32}
# of the output: the library's kind and torch's type (None: the input's)
NORM_OUTPUTS = {None: (0, None), "int8": (1, torch.int8), "e4m3": (2, torch.float8_e4m3fn)}
_empty_strided = torch.empty_strided


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class _NormConfig(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("dtype", ctypes.c_int), ("out", ctypes.c_int), ("eps", ctypes.c_float)]


EXPORTED_SYMBOLS = ("add_rms_norm", "add_rms_norm_backward", "add_rms_norm_backward_workspace_size")


def declare(lib):
    """The signatures of include/sparse_ffn_norm.h."""
    P, S, I64, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int
    C, R = ctypes.POINTER(_NormConfig), ctypes.POINTER(_Rows)
    lib.add_rms_norm.argtypes = [C, I64, R, R, P, R, P, R, P]
    lib.add_rms_norm.restype = st
    lib.add_rms_norm_backward_workspace_size.argtypes = [C, I64]
    lib.add_rms_norm_backward_workspace_size.restype = S
    lib.add_rms_norm_backward.argtypes = [C, I64, R, R, R, P, R, P, P, S, P]
    lib.add_rms_norm_backward.restype = st


@functools.lru_cache(maxsize=256)
def _config(d, dtype, out, eps):
    """The library's config, a constant of its arguments."""
    return _NormConfig(d, _DTYPES[dtype], out, eps)


@functools.lru_cache(maxsize=1024)
def _backward_workspace(d, dtype, T, device):
    """Its bytes, a constant of its arguments (the device's compute units are)."""
    return load_library().add_rms_norm_backward_workspace_size(_config(d, dtype, 0, 1.0), T)


def _rows(t, name, shape=None, dtype=None, device=None):
    """A [T, d] view on the GPU as the library takes it. Without a shape, the tensor that
    sets it: bfloat16 or float32."""
    if type(t) is not torch.Tensor or (t.shape != shape or t.dtype is not dtype or t.device != device
                                       if shape is not None else t.dim() != 2 or t.dtype not in _DTYPES or not t.is_cuda):
        _check_rows(t, name, shape, dtype, device)
    s, one = t.stride()
    T, d = t.shape if shape is None else shape
    if one != 1 and d > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return _Rows(t.data_ptr(), s if T > 1 else d)       # a dimension of one element may carry any stride


def _check_rows(t, name, shape, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {tuple(shape) if shape else '[T, d]'} (got {tuple(t.shape)})")
    if t.dtype != dtype if dtype is not None else t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be {dtype or 'bfloat16 or float32'} (got {t.dtype})")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on {device or 'the GPU'} (got {t.device})")


def _new(T, d, dtype, device):
    t = _empty_strided((T, d), (d, 1), dtype=dtype, device=device)
    return t, _Rows(t.data_ptr(), d)


def _weight(weight, d, dtype, device):
    if weight is None:
        return None
    if type(weight) is not torch.Tensor or weight.dtype is not dtype or weight.device != device \
            or weight.shape != (d,) or not weight.is_contiguous():
        _need_buffer(weight, "weight", (d,), dtype, device)
    return weight.data_ptr()


def add_rms_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, quant: Optional[str] = None, y_out: Optional[torch.Tensor] = None,
                 h_out: Optional[torch.Tensor] = None):
    """h = x + residual, rounded to their type, and y = h rsqrt(mean(h^2) + eps) weight for
    every row of x, residual [T, d] (views with any row stride; bfloat16 or float32).

    quant None: returns (y, h), y in x's type. "int8" or "e4m3": returns (y, scale, h), y
    torch.int8 or torch.float8_e4m3fn and scale fp32 [T]; y scale[:, None] are the values,
    a row's largest one at 127 or 448. Without a residual h is x itself. weight [d] (None:
    ones). y_out and h_out take the results; h_out, and y_out without quant, may be x or
    residual (without a residual a y_out that is x leaves no h). A row of zeros has scale 0,
    one with a NaN or an infinity in h or in h weight scale NaN."""
    lib = load_library()
    hx = _rows(x, "x")
    T, d = shape = x.shape
    dtype, dev = x.dtype, x.device
    try:
        kind, small = NORM_OUTPUTS[quant]
    except (KeyError, TypeError):
        raise ValueError(f"quant must be one of {tuple(NORM_OUTPUTS)} (got {quant!r})") from None
    cfg = _config(d, dtype, kind, eps)
    w = _weight(weight, d, dtype, dev)
    hr = hh = scale = None
    if y_out is None:
        y_out, hy = _new(T, d, small or dtype, dev)
    else:
        hy = _rows(y_out, "y_out", shape, small or dtype, dev)
    if residual is not None:
        hr = _rows(residual, "residual", shape, dtype, dev)
        if h_out is None:
            h_out, hh = _new(T, d, dtype, dev)
        else:
            hh = _rows(h_out, "h_out", shape, dtype, dev)
    elif h_out is not None:
        raise ValueError("h_out takes the sum with a residual, which is not given")
    else:
        h_out = x
    if small is not None:
        scale = _empty_strided((T,), (1,), dtype=torch.float32, device=dev)
    _run(lib, dev, lib.add_rms_norm, cfg, T, hx, hr, w, hy, _ptr(scale), hh)
    return (y_out, h_out) if small is None else (y_out, scale, h_out)


def add_rms_norm_backward(h: torch.Tensor, g_y: torch.Tensor, weight: Optional[torch.Tensor] = None,
                          g_h: Optional[torch.Tensor] = None, eps: float = 1e-6) -> dict:
    """Gradients of add_rms_norm (quant None) for the gradients g_y of y and g_h of h (None:
    zero); h is the sum that the forward returned. Returns "x", the gradient of x and of the
    residual alike (h's type), and "weight" (fp32; None where no weight was given)."""
    lib = load_library()
    hh = _rows(h, "h")
    T, d = shape = h.shape
    dtype, dev = h.dtype, h.device
    cfg = _config(d, dtype, 0, eps)
    hg = _rows(g_y, "g_y", shape, dtype, dev)
    hgh = None if g_h is None else _rows(g_h, "g_h", shape, dtype, dev)
    w = _weight(weight, d, dtype, dev)
    gx, hgx = _new(T, d, dtype, dev)
    gw = ws = None
    need = 0
    if w is not None:
        gw = _empty_strided((d,), (1,), dtype=torch.float32, device=dev)
        need = _backward_workspace(d, dtype, T, dev)
        ws = _empty_strided((need,), (1,), dtype=torch.uint8, device=dev) if need else None
    _run(lib, dev, lib.add_rms_norm_backward, cfg, T, hh, hg, hgh, w, hgx, _ptr(gw), _ptr(ws), need)
    return {"x": gx, "weight": gw}
