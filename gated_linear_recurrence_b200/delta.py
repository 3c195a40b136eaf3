"""ctypes binding of the gated delta rule (``include/esa.h``, esa_delta_*).

The recurrence with a matrix state S [D, D] (key channels by value channels)
per head, alpha = sigmoid(a), beta = sigmoid(b):

    u_t = beta_t (v_t - alpha_t S_{t-1}^T k_t)
    S_t = alpha_t S_{t-1} + k_t u_t^T
    y_t = scale S_t^T q_t

* :func:`esa_delta_fwd`  -- whole sequence (prefill, training forward)
* :func:`esa_delta_bwd`  -- its backward
* :func:`esa_delta_step` -- one token, in place on S; :class:`PreparedDeltaStep`
  is the same call on fixed buffers with its arguments resolved once

Argument marshalling only, as in ``esa.py``; float32, float16 and bfloat16
tensors, D of 32, 64 or 128, state tensors float32.
"""
from __future__ import annotations

import torch

from . import esa as _esa
from .esa import EsaError, _on, load_library, row_stride

_DTYPE_CODE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
# The current stream's handle without building a Stream object (2 us of a decode step's call).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    """A contiguous tensor of t's shape and type (empty_like is the cheapest call that makes one)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _stream(device, stream):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None and device.index is not None:
        return _current_raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _scratch(like, nbytes, stream):
    """``nbytes`` on ``like``'s device, from the pool of the stream that uses them: once dropped they go to that stream's
    next allocations alone, which come after the kernels still to run on it."""
    if stream is None:
        return like.new_empty(nbytes, dtype=torch.uint8)
    with torch.cuda.stream(stream):
        return like.new_empty(nbytes, dtype=torch.uint8)


def esa_delta_workspace_size(B: int, T: int, H: int, D: int, dtype, keep: bool = True) -> int:
    code = _esa._DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().esa_delta_workspace_size(B, T, H, D, code, int(bool(keep))))


def _new_workspace(B, T, H, D, q, keep, stream):
    n = load_library().esa_delta_workspace_size(B, T, H, D, _DTYPE_CODE[q.dtype], 1 if keep else 0)
    if n == 0:
        raise ValueError(f"unsupported shape for the delta rule: B={B}, T={T}, H={H}, D={D} (D is 32, 64 or 128)")
    return _scratch(q, n, stream)


def _check_workspace(workspace, device):
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.device != device \
            or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")
    return workspace.numel() * workspace.element_size()


def _gate_stride(t):
    """Elements between the logits of consecutive tokens of a [B, T, H] tensor, None for any other layout."""
    B, T, H = (int(x) for x in t.shape)
    st = t.stride()
    if H > 1 and st[2] != 1:
        return None
    if T > 1:
        if B > 1 and st[0] != T * st[1]:
            return None
        ld = st[1]
    else:
        ld = st[0] if B > 1 else H
    return ld if ld >= H else None


def _inputs(q, k, v, a, b):
    """Checked (B, T, H, D, ld_qk, ld_v, ld_g)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor (the ESA library has no CPU path)")
    if q.dim() != 4:
        raise ValueError("sequence tensors must be [B, T, H, D]")
    if q.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {q.dtype} (float32, float16 or bfloat16)")
    shape, dtype, where = q.shape, q.dtype, q.get_device()
    gates, dense = shape[:3], q.is_contiguous()
    for name, t, want in (("k", k, shape), ("v", v, shape), ("a", a, gates), ("b", b, gates)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor (the ESA library has no CPU path)")
        if t.shape != want or t.dtype is not dtype or t.get_device() != where:
            raise ValueError(f"{name} must have shape {tuple(want)}, dtype {dtype}, {q.device}")
        dense = dense and t.is_contiguous()
    B, T, H, D = shape
    if dense or B == 0 or T == 0:
        return B, T, H, D, H * D, H * D, H
    ld_q, ld_k, ld_v, ld_a, ld_b = row_stride(q), row_stride(k), row_stride(v), _gate_stride(a), _gate_stride(b)
    for name, ld in (("q", ld_q), ("k", ld_k), ("v", ld_v)):
        if ld is None:
            raise ValueError(f"{name} must be [B, T, H, D] with each token's H*D channels contiguous")
    if ld_q != ld_k:
        raise ValueError(f"q and k must share one row stride (got {ld_q} and {ld_k})")
    if ld_a is None or ld_a != ld_b:
        raise ValueError("a and b must be [B, T, H] with each token's H logits contiguous and share one row stride")
    return B, T, H, D, ld_q, ld_v, ld_a


def _check_state(name, t, B, H, D, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.device != device:
        raise TypeError(f"{name} must be a CUDA tensor on {device}")
    if tuple(t.shape) != (B, H, D, D) or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(B, H, D, D)}")


def _out(name, t, shape, dtype, device):
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _scale(scale, D):
    return D ** -0.5 if scale is None else float(scale)


def esa_delta_fwd(q, k, v, a, b, scale=None, S_init=None, y=None, S_final=None, workspace=None, keep=True,
                  stream=None, want_S_final=True):
    """Forward over a whole sequence.  Returns ``(y, S_final, workspace)``.

    ``q, k, v`` [B, T, H, D] and the logits ``a, b`` [B, T, H] may be
    row-strided views (column blocks of one projection output; q and k share
    a row stride, a and b another).  ``scale`` defaults to D ** -0.5.
    ``keep`` leaves in the workspace what :func:`esa_delta_bwd` reads (9 times
    ``q``'s bytes with bfloat16 tensors, 11 with float16); an inference call
    passes False (3.4 times at D = 128, 4.7 at D = 64).  ``stream`` runs the call on that stream
    instead of the current one; outputs are allocated on the current one, so
    hold them until that stream is done with them.
    """
    B, T, H, D, ld_qk, ld_v, ld_g = _inputs(q, k, v, a, b)
    y = _like(q) if y is None else _out("y", y, q.shape, q.dtype, q.device)
    if S_final is not None:
        _check_state("S_final", S_final, B, H, D, q.device)
    elif want_S_final:
        S_final = q.new_empty((B, H, D, D), dtype=torch.float32)
    _check_state("S_init", S_init, B, H, D, q.device)
    if workspace is None:
        workspace = _new_workspace(B, T, H, D, q, keep, stream)
    nbytes = _check_workspace(workspace, q.device)
    with _on(q.device):
        rc = load_library().esa_delta_fwd(
            _ptr(q), _ptr(k), ld_qk, _ptr(v), ld_v, _ptr(a), _ptr(b), ld_g, _ptr(y), _ptr(S_final), B, T, H, D,
            _scale(scale, D), _ptr(S_init), _DTYPE_CODE[q.dtype], int(bool(keep)), _ptr(workspace), nbytes,
            _stream(q.device, stream))
    if rc != 0:
        raise EsaError("esa_delta_fwd", rc)
    return y, S_final, workspace


def esa_delta_bwd(q, k, v, a, b, dy, workspace, scale=None, S_init=None, dS_final=None, dq=None, dk=None, dv=None,
                  da=None, db=None, dS_init=None, stream=None, want_dS_init=True):
    """Backward.  ``workspace`` must be the one the matching forward wrote
    (``keep=True``), its inputs unchanged.  Returns
    ``(dq, dk, dv, da, db, dS_init)``."""
    B, T, H, D, ld_qk, ld_v, ld_g = _inputs(q, k, v, a, b)
    if not isinstance(dy, torch.Tensor) or not dy.is_cuda:
        raise TypeError("dy must be a CUDA tensor (the ESA library has no CPU path)")
    dy = _out("dy", dy, q.shape, q.dtype, q.device)
    dq, dk, dv, da, db = (_like(like) if t is None else _out(name, t, like.shape, q.dtype, q.device)
                          for name, t, like in (("dq", dq, q), ("dk", dk, q), ("dv", dv, q), ("da", da, a), ("db", db, a)))
    if dS_init is not None:
        _check_state("dS_init", dS_init, B, H, D, q.device)
    elif want_dS_init:
        dS_init = q.new_empty((B, H, D, D), dtype=torch.float32)
    _check_state("dS_final", dS_final, B, H, D, q.device)
    _check_state("S_init", S_init, B, H, D, q.device)
    if workspace is None:
        raise ValueError("esa_delta_bwd needs the CUDA workspace written by the matching esa_delta_fwd")
    nbytes = _check_workspace(workspace, q.device)
    with _on(q.device):
        rc = load_library().esa_delta_bwd(
            _ptr(q), _ptr(k), ld_qk, _ptr(v), ld_v, _ptr(a), _ptr(b), ld_g, _ptr(dy), _ptr(dS_final), _ptr(dq),
            _ptr(dk), _ptr(dv), _ptr(da), _ptr(db), _ptr(dS_init), B, T, H, D, _scale(scale, D), _ptr(S_init),
            _DTYPE_CODE[q.dtype], _ptr(workspace), nbytes, _stream(q.device, stream))
    if rc != 0:
        raise EsaError("esa_delta_bwd", rc)
    return dq, dk, dv, da, db, dS_init


def _token_stride(name, t, H, width):
    """Elements between consecutive batch entries of [B, H, width] or [B, H]."""
    if t.is_contiguous():
        return H * width
    st = t.stride()
    if (width > 1 and st[-1] != 1) or (H > 1 and st[1] != width) or (t.shape[0] > 1 and st[0] < H * width):
        raise ValueError(f"{name} must have each token's elements contiguous and tokens that do not overlap")
    return st[0] if t.shape[0] > 1 else H * width


def _step_args(q_t, k_t, v_t, a_t, b_t, S, y_t, scale):
    if not isinstance(q_t, torch.Tensor) or not q_t.is_cuda or q_t.dim() != 3:
        raise TypeError("q_t must be a CUDA tensor [B, H, D] (the ESA library has no CPU path)")
    shape, dtype, where = q_t.shape, q_t.dtype, q_t.get_device()
    if dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {dtype} (float32, float16 or bfloat16)")
    B, H, D = shape
    gates, dense = shape[:2], q_t.is_contiguous()
    for name, t, want in (("k_t", k_t, shape), ("v_t", v_t, shape), ("a_t", a_t, gates), ("b_t", b_t, gates)):
        if not isinstance(t, torch.Tensor) or t.get_device() != where:
            raise TypeError(f"{name} must be a CUDA tensor on {q_t.device}")
        if t.shape != want or t.dtype is not dtype:
            raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(want)}")
        dense = dense and t.is_contiguous()
    ld_qk = ld_v = H * D
    ld_g = H
    if not dense:
        ld_qk, ld_v, ld_g = (_token_stride(n, t, H, w) for n, t, w in (("q_t", q_t, D), ("v_t", v_t, D), ("a_t", a_t, 1)))
        if _token_stride("k_t", k_t, H, D) != ld_qk or _token_stride("b_t", b_t, H, 1) != ld_g:
            raise ValueError("q_t and k_t must share one row stride, a_t and b_t another")
    if S is None:
        raise ValueError("S (the recurrent state) is required")
    if not isinstance(S, torch.Tensor) or S.get_device() != where:
        raise TypeError(f"S must be a CUDA tensor on {q_t.device}")
    if S.shape != (B, H, D, D) or S.dtype is not torch.float32 or not S.is_contiguous():
        raise ValueError(f"S must be a contiguous float32 tensor of shape {(B, H, D, D)}")
    y_t = _like(q_t) if y_t is None else _out("y_t", y_t, shape, dtype, q_t.device)
    return y_t, (q_t.data_ptr(), k_t.data_ptr(), ld_qk, v_t.data_ptr(), ld_v, a_t.data_ptr(), b_t.data_ptr(), ld_g,
                 S.data_ptr(), y_t.data_ptr(), B, H, D, D ** -0.5 if scale is None else float(scale),
                 _DTYPE_CODE[dtype])


def esa_delta_step(q_t, k_t, v_t, a_t, b_t, S, y_t=None, scale=None, stream=None):
    """One token: ``S`` (float32 [B, H, D, D]) is updated in place.  Returns
    ``y_t`` [B, H, D].  ``q_t, k_t, v_t`` [B, H, D] and ``a_t, b_t`` [B, H] may
    be row-strided views, as in :func:`esa_delta_fwd`."""
    y_t, args = _step_args(q_t, k_t, v_t, a_t, b_t, S, y_t, scale)
    with _on(q_t.device):
        rc = load_library().esa_delta_step(*args, _stream(q_t.device, stream))
    if rc != 0:
        raise EsaError("esa_delta_step", rc)
    return y_t


class PreparedDeltaStep:
    """:func:`esa_delta_step` on fixed buffers, with the argument checks, the
    device pointers and the stream resolved once, at construction (see
    :class:`~.esa.PreparedStep`).  Calling it returns ``y_t``."""

    def __init__(self, q_t, k_t, v_t, a_t, b_t, S, y_t=None, scale=None, stream=None):
        self.y_t, args = _step_args(q_t, k_t, v_t, a_t, b_t, S, y_t, scale)
        self.device = q_t.device
        if self.device.index is not None and self.device.index != torch.cuda.current_device():
            raise ValueError("make the tensors' device current before preparing and calling the step")
        self._keep = (q_t, k_t, v_t, a_t, b_t, S, self.y_t)   # the buffers stay alive as long as this object
        self._fn = load_library().esa_delta_step
        self._args = (*args, _stream(self.device, stream))

    def __call__(self):
        rc = self._fn(*self._args)
        if rc != 0:
            raise EsaError("esa_delta_step", rc)
        return self.y_t
