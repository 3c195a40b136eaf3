"""ctypes binding of the layer norm (``include/esa.h``, esa_norm_*).

    h = x + residual,  y = (h - mean) rstd weight + bias   over the last axis

* :func:`esa_norm_fwd` -- forward, with the residual addition before it
* :func:`esa_norm_bwd` -- dx, dweight, dbias

Argument marshalling only, as in ``esa.py``; float32, float16 and bfloat16
rows of up to 16384 elements, weights in the rows' dtype or float32,
statistics float32.
"""
from __future__ import annotations

import torch

from .delta import _check_workspace, _like, _ptr, _scratch, _stream
from .esa import EsaError, _on, load_library

_DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _rows(name, t, like=None):
    """Elements between consecutive rows of a tensor [..., N] whose rows are
    contiguous and evenly spaced."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() < 1:
        raise TypeError(f"{name} must be a CUDA tensor [..., N] (the ESA library has no CPU path)")
    if like is not None and (t.shape != like.shape or t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, dtype {like.dtype}, {like.device}")
    N = int(t.shape[-1])
    if t.is_contiguous() or t.numel() == 0:
        return N
    ld, expect = N, None
    if N > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if expect is None:
            ld = stride
        elif stride != expect:
            raise ValueError(f"{name}'s rows must be evenly spaced")
        expect = stride * size
    if ld < N:
        raise ValueError(f"{name}'s rows must not overlap")
    return ld


def _check_x(x, name="x"):
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() < 1:
        raise TypeError(f"{name} must be a CUDA tensor [..., N] (the ESA library has no CPU path)")
    if x.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {x.dtype} (float32, float16 or bfloat16)")
    N = x.shape[-1]
    if N < 1:
        raise ValueError(f"{name} must have at least one channel")
    return x.numel() // N, N


def _check_param(name, p, x, N):
    if not isinstance(p, torch.Tensor) or p.get_device() != x.get_device() or p.shape != (N,) or not p.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {(N,)} on {x.device}")
    if p.dtype is not torch.float32 and p.dtype is not x.dtype:
        raise TypeError(f"{name} must be {x.dtype} or float32")
    return p.dtype


def _out(name, t, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def esa_norm_fwd(x, weight=None, bias=None, eps=1e-5, residual=None, y=None, h=None, stats=None, want_stats=True,
                 stream=None):
    """Layer norm of ``x`` [..., N], or of ``h = x + residual``.

    Returns ``(y, h, stats)``: ``h`` is ``x`` itself without a residual;
    ``stats`` (float32 [rows, 2]: mean, rstd) is what :func:`esa_norm_bwd`
    reads, None with ``want_stats=False``.  ``x`` and ``residual`` may be
    row-strided.
    """
    rows, N = _check_x(x)
    ld_x = _rows("x", x)
    ld_r = N if residual is None else _rows("residual", residual, x)
    wdt = None if weight is None else _check_param("weight", weight, x, N)
    if bias is not None:
        if _check_param("bias", bias, x, N) is not (wdt or bias.dtype):
            raise TypeError("weight and bias must share one dtype")
        wdt = bias.dtype
    y = _like(x) if y is None else _out("y", y, x.shape, x.dtype, x.device)
    if residual is None:
        if h is not None:
            raise ValueError("h is an output of the residual addition: give residual too")
    else:
        h = _like(y) if h is None else _out("h", h, x.shape, x.dtype, x.device)
    if stats is not None:
        _out("stats", stats, (rows, 2), torch.float32, x.device)
    elif want_stats:
        stats = x.new_empty((rows, 2), dtype=torch.float32)
    with _on(x.device):
        rc = load_library().esa_norm_fwd(_ptr(x), ld_x, _ptr(residual), ld_r, _ptr(weight), _ptr(bias), _ptr(y),
                                         _ptr(h), _ptr(stats), rows, N, float(eps), _DTYPE_CODE[x.dtype],
                                         _DTYPE_CODE[wdt or x.dtype], _stream(x.device, stream))
    if rc != 0:
        raise EsaError("esa_norm_fwd", rc)
    return y, (x if residual is None else h), stats


def esa_norm_bwd(dy, h, weight, stats, dh=None, dx=None, dweight=None, dbias=None, want_dweight=True,
                 want_dbias=True, wdtype=None, workspace=None, stream=None):
    """Backward of :func:`esa_norm_fwd`.  Returns ``(dx, dweight, dbias)``.

    ``h`` and ``stats`` are the forward's; ``dh`` is the gradient that reaches
    ``h`` through the residual stream and is added to ``dx``, which is the
    gradient of ``x`` and of ``residual`` alike.  ``dweight`` and ``dbias``
    have the weight's dtype (``wdtype``, or ``h``'s, without a weight).
    ``stream`` is :func:`~.delta.esa_delta_fwd`'s.
    """
    rows, N = _check_x(h, "h")
    ld_h, ld_dy = _rows("h", h), _rows("dy", dy, h)
    ld_dh = N if dh is None else _rows("dh", dh, h)
    wdt = _check_param("weight", weight, h, N) if weight is not None else (wdtype or h.dtype)
    if wdt is not torch.float32 and wdt is not h.dtype:
        raise TypeError(f"wdtype must be {h.dtype} or float32")
    if not isinstance(stats, torch.Tensor) or stats.shape != (rows, 2) or stats.dtype is not torch.float32 \
            or stats.get_device() != h.get_device() or not stats.is_contiguous():
        raise ValueError(f"stats must be the forward's contiguous float32 tensor of shape {(rows, 2)}")
    dx = _like(h) if dx is None else _out("dx", dx, h.shape, h.dtype, h.device)
    if dweight is not None:
        _out("dweight", dweight, (N,), wdt, h.device)
    elif want_dweight:
        dweight = h.new_empty((N,), dtype=wdt)
    if dbias is not None:
        _out("dbias", dbias, (N,), wdt, h.device)
    elif want_dbias:
        dbias = h.new_empty((N,), dtype=wdt)
    lib = load_library()
    codes = (_DTYPE_CODE[h.dtype], _DTYPE_CODE[wdt])
    if workspace is None and (dweight is not None or dbias is not None):
        workspace = _scratch(h, lib.esa_norm_workspace_size(rows, N, *codes), stream)
    nbytes = 0 if workspace is None else _check_workspace(workspace, h.device)
    with _on(h.device):
        rc = lib.esa_norm_bwd(_ptr(dy), ld_dy, _ptr(h), ld_h, _ptr(weight), _ptr(stats), _ptr(dh), ld_dh, _ptr(dx),
                              _ptr(dweight), _ptr(dbias), rows, N, *codes, _ptr(workspace), nbytes,
                              _stream(h.device, stream))
    if rc != 0:
        raise EsaError("esa_norm_bwd", rc)
    return dx, dweight, dbias
