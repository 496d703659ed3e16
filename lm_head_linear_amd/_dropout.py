"""Dropout from a counter-based generator, alone, with the residual's addition, and with
the addition and the norm (see include/flce.h for the mask's definition). The mask is a
function of (p, seed, offset, step) and is formed again in the backward, never stored.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._ops import _bytes, _flat_rows, _on_gpu, _rows, _run, _stream, _workspace
from ._ops import flce_rms_norm_backward_workspace_size
from ._util import _check_tensor, _dtype_code, _ptr


class DropoutMask(NamedTuple):
    """Which values drop out: each with probability ``p`` (in steps of 2^-16), by the
    generator's ``seed`` and ``offset`` (64 bits each; another offset is another mask)
    and, where a captured graph shall draw another mask on every replay, ``step``: an
    int64 tensor on the device that is added to the offset. The backward reads it again,
    so it changes between steps, not within one."""
    p: float
    seed: int
    offset: int = 0
    step: Optional[torch.Tensor] = None


_U64 = (1 << 64) - 1


def _mask_args(where, dev, p, seed, offset, step):
    if not 0.0 <= p < 1.0:
        raise ValueError(f"{where}: p must be in [0, 1), got {p}")
    if not (0 <= seed <= _U64 and 0 <= offset <= _U64):
        raise ValueError(f"{where}: seed and offset must be in [0, 2^64), got {seed}, {offset}")
    if step is None:
        return p, seed, offset, None
    if step.dtype != torch.int64 or step.numel() != 1 or step.device != dev:
        raise ValueError(f"{where}: step must be one int64 on {dev}")
    return p, seed, offset, step.data_ptr()


def _mat(name, t, N, H, dt, dev):
    """t (or a new matrix) and its row stride."""
    if t is None:
        return torch.empty(N, H, dtype=dt, device=dev), H
    return t, _rows(name, t, N, H, dt, dev)


def flce_dropout_check_args(x, residual=None, *, N, H, p=0.1, seed=0, offset=0, step=None,
                            ld_x=None, ld_res=None, out=None, ld_out=None,
                            dtype=torch.bfloat16) -> int:
    """Dropout's synchronous checks (no GPU work); a status code."""
    ld = lambda v: H if v is None else int(v)  # noqa: E731
    return int(_lib.load().flce_dropout_check_args(
        _ptr(x), ld(ld_x), _ptr(residual), ld(ld_res), N, H, float(p), seed, offset, _ptr(step),
        _ptr(out), ld(ld_out), None, _dtype_code(dtype)))


def flce_dropout(x: torch.Tensor, residual: Optional[torch.Tensor] = None, *, p: float, seed: int,
                 offset: int = 0, step: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + keep * x / (1 - p) for x [N, H], rounded once.

    ``out`` may be x or the residual (in place).
    """
    if x.dim() != 2:
        raise ValueError("x must be [N, H]")
    N, H = x.shape
    dev, dt = x.device, x.dtype
    _on_gpu("flce_dropout", dev)
    code = _dtype_code(dt)
    mask = _mask_args("flce_dropout", dev, p, seed, offset, step)
    ld_x = _rows("x", x, N, H, dt, dev)
    ld_r = H if residual is None else _rows("residual", residual, N, H, dt, dev)
    if out is None:
        out, ld_o = torch.empty(N, H, dtype=dt, device=dev), H
    else:
        ld_o = _rows("out", out, N, H, dt, dev)
    _run("flce_dropout", dev, _lib.load().flce_dropout, x.data_ptr(), ld_x, _ptr(residual), ld_r,
         N, H, *mask, out.data_ptr(), ld_o, _stream(dev), code)
    return out


def flce_dropout_backward(dout: torch.Tensor, *, p: float, seed: int, offset: int = 0,
                          step: Optional[torch.Tensor] = None,
                          dx: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of x: keep * dout / (1 - p). The residual's is dout itself."""
    return flce_dropout(dout, p=p, seed=seed, offset=offset, step=step, out=dx)


def flce_dropout_norm_check_args(x, weight, residual=None, *, N, H, p=0.1, seed=0, offset=0,
                                 step=None, ld_x=None, ld_res=None, eps=1e-6, weight_offset=0.0,
                                 y=None, ld_y=None, s=None, ld_s=None, rstd=None,
                                 dtype=torch.bfloat16, weight_dtype=None) -> int:
    """The synchronous checks of dropout and norm (no GPU work); a status code."""
    ld = lambda v: H if v is None else int(v)  # noqa: E731
    return int(_lib.load().flce_dropout_norm_check_args(
        _ptr(x), ld(ld_x), _ptr(residual), ld(ld_res), _ptr(weight), N, H, float(eps),
        float(weight_offset), float(p), seed, offset, _ptr(step), _ptr(y), ld(ld_y), _ptr(s),
        ld(ld_s), _ptr(rstd), None, _dtype_code(dtype), _dtype_code(weight_dtype or dtype)))


def flce_dropout_norm(x: torch.Tensor, weight: torch.Tensor,
                      residual: Optional[torch.Tensor] = None, *, p: float, seed: int,
                      offset: int = 0, step: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      weight_offset: float = 0.0, y: Optional[torch.Tensor] = None,
                      s: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None):
    """:func:`flce_rms_norm` of s = residual + keep * x / (1 - p), in one pass: (y, s, rstd)."""
    if x.dim() != 2:
        raise ValueError("x must be [N, H]")
    N, H = x.shape
    dev, dt = x.device, x.dtype
    _on_gpu("flce_dropout_norm", dev)
    code, wcode = _dtype_code(dt), _dtype_code(weight.dtype)
    mask = _mask_args("flce_dropout_norm", dev, p, seed, offset, step)
    _check_tensor("weight", weight, (H,), weight.dtype, dev)
    ld_x = _rows("x", x, N, H, dt, dev)
    ld_r = H if residual is None else _rows("residual", residual, N, H, dt, dev)
    y, ld_y = _mat("y", y, N, H, dt, dev)
    s, ld_s = _mat("s", s, N, H, dt, dev)
    if rstd is None:
        rstd = torch.empty(N, dtype=torch.float32, device=dev)
    else:
        _check_tensor("rstd", rstd, (N,), torch.float32, dev)
    _run("flce_dropout_norm", dev, _lib.load().flce_dropout_norm, x.data_ptr(), ld_x,
         _ptr(residual), ld_r, weight.data_ptr(), N, H, float(eps), float(weight_offset), *mask,
         y.data_ptr(), ld_y, s.data_ptr(), ld_s, rstd.data_ptr(), _stream(dev), code, wcode)
    return y, s, rstd


def flce_dropout_norm_backward_check_args(dy, s, weight, rstd, ds=None, *, N, H, p=0.1, seed=0,
                                          offset=0, step=None, ld_dy=None, ld_ds=None, ld_s=None,
                                          weight_offset=0.0, dx=None, ld_dx=None, dresidual=None,
                                          ld_dres=None, dweight=None, accumulate_dweight=False,
                                          dtype=torch.bfloat16, weight_dtype=None,
                                          workspace=None) -> int:
    """The synchronous checks of its backward (no GPU work); a status code."""
    ld = lambda v: H if v is None else int(v)  # noqa: E731
    return int(_lib.load().flce_dropout_norm_backward_check_args(
        _ptr(dy), ld(ld_dy), _ptr(ds), ld(ld_ds), _ptr(s), ld(ld_s), _ptr(weight), _ptr(rstd), N,
        H, float(weight_offset), float(p), seed, offset, _ptr(step), _ptr(dx), ld(ld_dx),
        _ptr(dresidual), ld(ld_dres), _ptr(dweight), int(bool(accumulate_dweight)), None,
        _dtype_code(dtype), _dtype_code(weight_dtype or dtype), _ptr(workspace),
        _bytes(workspace)))


def flce_dropout_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor,
                               rstd: torch.Tensor, ds: Optional[torch.Tensor] = None, *,
                               p: float, seed: int, offset: int = 0,
                               step: Optional[torch.Tensor] = None, weight_offset: float = 0.0,
                               dx: Optional[torch.Tensor] = None,
                               dresidual: Optional[torch.Tensor] = None,
                               want_dresidual: bool = True,
                               dweight: Optional[torch.Tensor] = None, want_dweight: bool = True,
                               accumulate_dweight: bool = False,
                               workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`flce_dropout_norm`: (dx, dresidual, dweight), those not wanted
    None; dresidual is the gradient of the sum s, dx the same masked and scaled."""
    if dy.dim() != 2:
        raise ValueError("dy must be [N, H]")
    N, H = dy.shape
    dev, dt = dy.device, dy.dtype
    where = "flce_dropout_norm_backward"
    _on_gpu(where, dev)
    code, wcode = _dtype_code(dt), _dtype_code(weight.dtype)
    mask = _mask_args(where, dev, p, seed, offset, step)
    _check_tensor("weight", weight, (H,), weight.dtype, dev)
    _check_tensor("rstd", rstd, (N,), torch.float32, dev)
    ld_dy, ld_s = _rows("dy", dy, N, H, dt, dev), _rows("s", s, N, H, dt, dev)
    ld_ds = H if ds is None else _rows("ds", ds, N, H, dt, dev)
    dx, ld_dx = _mat("dx", dx, N, H, dt, dev)
    ld_dres = H
    if dresidual is not None or want_dresidual:
        dresidual, ld_dres = _mat("dresidual", dresidual, N, H, dt, dev)
    if accumulate_dweight and dweight is None:
        raise ValueError("accumulate_dweight needs the dweight tensor to add to")
    if dweight is not None:
        _check_tensor("dweight", dweight, (H,), weight.dtype, dev)
    elif want_dweight:
        dweight = torch.empty(H, dtype=weight.dtype, device=dev)
    if dweight is not None:
        workspace = _workspace(where, workspace, flce_rms_norm_backward_workspace_size(N, H), dev)
    _run(where, dev, _lib.load().flce_dropout_norm_backward, dy.data_ptr(), ld_dy, _ptr(ds), ld_ds,
         s.data_ptr(), ld_s, weight.data_ptr(), rstd.data_ptr(), N, H, float(weight_offset), *mask,
         dx.data_ptr(), ld_dx, _ptr(dresidual), ld_dres, _ptr(dweight),
         int(bool(accumulate_dweight)), _stream(dev), code, wcode, _ptr(workspace),
         _bytes(workspace))
    return dx, dresidual, dweight


# The functions return rows, which their wrappers shape: a view made inside a function could
# not be changed in place by its caller. A step tensor is saved as one, so that autograd
# refuses a backward whose mask would be another one than the forward's.


def _saved_mask(ctx, mask, *tensors):
    ctx.mask = dict(p=mask.p, seed=mask.seed, offset=mask.offset)
    ctx.has_step = mask.step is not None
    ctx.save_for_backward(*tensors, *([mask.step] if ctx.has_step else []))


def _load_mask(ctx):
    t = ctx.saved_tensors
    return (t[:-1], dict(ctx.mask, step=t[-1])) if ctx.has_step else (t, ctx.mask)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, mask):
        ctx.shape, ctx.res_shape = x.shape, None if residual is None else residual.shape
        _saved_mask(ctx, mask)
        return flce_dropout(_flat_rows(x), None if residual is None else _flat_rows(residual),
                            **mask._asdict())

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        _, mask = _load_mask(ctx)
        dx = dres = None
        if ctx.needs_input_grad[0]:
            dx = flce_dropout_backward(_flat_rows(dout), **mask).reshape(ctx.shape)
        if ctx.needs_input_grad[1]:
            dres = dout.reshape(ctx.res_shape)
        return dx, dres, None


def _same_shape(x, residual):
    if residual is not None and residual.shape != x.shape:
        raise ValueError(f"residual must have shape {tuple(x.shape)}, got {tuple(residual.shape)}")


def fused_dropout(x: torch.Tensor, mask: DropoutMask,
                  residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dropout of x [..., H], added to the residual, with gradients. Row r of the mask is
    row r of x.reshape(-1, H)."""
    _same_shape(x, residual)
    return _Dropout.apply(x, residual, mask).view(x.shape)


class _DropoutNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, mask, eps, weight_offset):
        ctx.shape = x.shape
        y, s, rstd = flce_dropout_norm(_flat_rows(x), weight,
                                       None if residual is None else _flat_rows(residual),
                                       eps=eps, weight_offset=weight_offset, **mask._asdict())
        _saved_mask(ctx, mask, s, weight, rstd)
        ctx.weight_offset = weight_offset
        ctx.set_materialize_grads(False)
        return y, s

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds):
        (s, weight, rstd), mask = _load_mask(ctx)
        dw = None
        if dy is None:                       # only the sum was used
            if ds is None:
                return (None,) * 6
            dres = ds
            dx = flce_dropout_backward(_flat_rows(ds), **mask)
        else:
            dx, dres, dw = flce_dropout_norm_backward(
                _flat_rows(dy), s, weight, rstd, None if ds is None else _flat_rows(ds),
                weight_offset=ctx.weight_offset, want_dresidual=ctx.needs_input_grad[2],
                want_dweight=ctx.needs_input_grad[1], **mask)
        return (dx.reshape(ctx.shape), dw,
                dres.reshape(ctx.shape) if ctx.needs_input_grad[2] else None, None, None, None)


def fused_dropout_norm(x: torch.Tensor, weight: torch.Tensor, mask: DropoutMask,
                       residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                       weight_offset: float = 0.0):
    """(y, s) with s = residual + dropout(x) for x [..., H] and y its RMS norm, with
    gradients."""
    _same_shape(x, residual)
    y, s = _DropoutNorm.apply(x, weight.contiguous(), residual, mask, float(eps),
                              float(weight_offset))
    return y.view(x.shape), s.view(x.shape)
