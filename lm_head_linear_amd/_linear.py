"""The linear transform in front of the head, y = act(x W^T + b) + r, with gradients (see
include/flce.h for the contract)."""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._ops import _bytes, _flat_rows, _on_gpu, _out, _rows, _run, _stream, _workspace
from ._util import _check_tensor, _dtype_code, _ptr


def _act_code(activation: str) -> int:
    if activation not in _lib.ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_lib.ACTIVATIONS)}, got {activation!r}")
    return _lib.ACTIVATIONS[activation]


def _slope_dtype(dt):
    return torch.float16 if dt == torch.bfloat16 else torch.float32


def flce_linear_check_args(x, weight, bias=None, residual=None, *, N, I, O, activation="none",
                           ld_x=None, ld_res=None, y=None, ld_y=None, slope=None,
                           dtype=torch.bfloat16, y_dtype=None) -> int:
    """The transform's synchronous checks (no GPU work); a status code."""
    ld = lambda v, n: n if v is None else int(v)  # noqa: E731
    return int(_lib.load().flce_linear_check_args(
        _ptr(x), ld(ld_x, I), _ptr(weight), _ptr(bias), _ptr(residual), ld(ld_res, O), N, I, O,
        activation if isinstance(activation, int) else _act_code(activation), _ptr(y),
        ld(ld_y, O), _ptr(slope), None, _dtype_code(dtype), _dtype_code(y_dtype or dtype)))


def flce_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, *, activation: str = "none",
                save_slope: bool = False, y_dtype: Optional[torch.dtype] = None,
                y: Optional[torch.Tensor] = None, slope: Optional[torch.Tensor] = None):
    """act(x weight^T + bias) + residual for x [N, I], weight [O, I]: (y, slope).

    ``slope`` is the activation's derivative (float32, or float16 with bf16 rows), which
    :func:`flce_linear_backward` takes: formed with ``save_slope`` (or where a tensor for it is
    passed in), otherwise None, and None without an activation. y has x's type, or float32 with ``y_dtype``; ``y`` may be
    the residual (in place).
    """
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [N, I] and weight [O, I]")
    (N, I), O = x.shape, weight.shape[0]
    dev, dt = x.device, x.dtype
    _on_gpu("flce_linear", dev)
    code, act = _dtype_code(dt), _act_code(activation)
    ydt = y_dtype or (dt if y is None else y.dtype)
    ycode = _dtype_code(ydt)
    _check_tensor("weight", weight, (O, I), dt, dev)
    if bias is not None:
        _check_tensor("bias", bias, (O,), dt, dev)
    ld_x = _rows("x", x, N, I, dt, dev)
    ld_r = O if residual is None else _rows("residual", residual, N, O, dt, dev)
    if y is None:
        y, ld_y = torch.empty(N, O, dtype=ydt, device=dev), O
    else:
        ld_y = _rows("y", y, N, O, ydt, dev)
    if act == 0:
        if slope is not None:
            raise ValueError("slope is written only with an activation")
    elif slope is not None or save_slope:
        slope = _out("slope", slope, (N, O), _slope_dtype(dt), dev)
    _run("flce_linear", dev, _lib.load().flce_linear, x.data_ptr(), ld_x, weight.data_ptr(),
         _ptr(bias), _ptr(residual), ld_r, N, I, O, act, y.data_ptr(), ld_y, _ptr(slope),
         _stream(dev), code, ycode)
    return y, slope


def flce_linear_backward_workspace_size(N: int, I: int, O: int, dtype: torch.dtype) -> int:
    return int(_lib.load().flce_linear_backward_workspace_size(N, I, O, _dtype_code(dtype)))


def flce_linear_backward_check_args(dy, x, weight, slope=None, *, N, I, O, ld_dy=None, ld_x=None,
                                    dx=None, ld_dx=None, dweight=None, dbias=None,
                                    accumulate=False, dtype=torch.bfloat16,
                                    workspace=None) -> int:
    """The transform's backward's synchronous checks (no GPU work); a status code."""
    ld = lambda v, n: n if v is None else int(v)  # noqa: E731
    return int(_lib.load().flce_linear_backward_check_args(
        _ptr(dy), ld(ld_dy, O), _ptr(x), ld(ld_x, I), _ptr(weight), _ptr(slope), N, I, O, _ptr(dx),
        ld(ld_dx, I), _ptr(dweight), _ptr(dbias), int(bool(accumulate)), None, _dtype_code(dtype),
        _ptr(workspace), _bytes(workspace)))


def flce_linear_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                         slope: Optional[torch.Tensor] = None, *, bias: bool = True,
                         want_dx: bool = True, want_dweight: bool = True,
                         dx: Optional[torch.Tensor] = None,
                         dweight: Optional[torch.Tensor] = None,
                         dbias: Optional[torch.Tensor] = None, accumulate: bool = False,
                         workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`flce_linear`: (dx, dweight, dbias), None where not wanted. The
    residual's gradient is dy. With ``accumulate`` dweight and dbias are added to the tensors
    passed in."""
    if dy.dim() != 2 or x.dim() != 2 or weight.dim() != 2:
        raise ValueError("dy must be [N, O], x [N, I] and weight [O, I]")
    (N, I), O = x.shape, weight.shape[0]
    dev, dt = x.device, x.dtype
    _on_gpu("flce_linear_backward", dev)
    code = _dtype_code(dt)
    _check_tensor("weight", weight, (O, I), dt, dev)
    ld_dy, ld_x = _rows("dy", dy, N, O, dt, dev), _rows("x", x, N, I, dt, dev)
    if slope is not None:
        _check_tensor("slope", slope, (N, O), _slope_dtype(dt), dev)
    if accumulate and ((want_dweight and dweight is None) or (bias and dbias is None)):
        raise ValueError("accumulate needs the dweight and dbias tensors to add to")
    ld_dx = I
    if dx is not None:
        ld_dx = _rows("dx", dx, N, I, dt, dev)
    elif want_dx:
        dx = torch.empty(N, I, dtype=dt, device=dev)
    if dweight is not None or want_dweight:
        dweight = _out("dweight", dweight, (O, I), dt, dev)
    if dbias is not None or bias:
        dbias = _out("dbias", dbias, (O,), dt, dev)
    lib = _lib.load()
    workspace = _workspace("flce_linear_backward", workspace,
                           lib.flce_linear_backward_workspace_size(N, I, O, code), dev)
    _run("flce_linear_backward", dev, lib.flce_linear_backward, dy.data_ptr(), ld_dy, x.data_ptr(),
         ld_x, weight.data_ptr(), _ptr(slope), N, I, O, _ptr(dx), ld_dx, _ptr(dweight),
         _ptr(dbias), int(bool(accumulate)), _stream(dev), code, workspace.data_ptr(),
         _bytes(workspace))
    return dx, dweight, dbias


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation):
        rows = _flat_rows(x)
        need = any(ctx.needs_input_grad[:3])
        y, slope = flce_linear(rows, weight, bias,
                               None if residual is None else _flat_rows(residual),
                               activation=activation, save_slope=need)
        ctx.save_for_backward(rows, weight, slope)
        ctx.shape = x.shape
        ctx.res_shape = None if residual is None else residual.shape
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, slope = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dw = db = None
        if any(need[:3]):
            dx, dw, db = flce_linear_backward(_flat_rows(dy), x, weight, slope, bias=need[2],
                                              want_dx=need[0], want_dweight=need[1])
        return (None if dx is None else dx.reshape(ctx.shape), dw, db,
                dy.reshape(ctx.res_shape) if need[3] else None, None)


def fused_linear(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 residual: Optional[torch.Tensor] = None, *,
                 activation: str = "none") -> torch.Tensor:
    """act(x weight^T + bias) + residual for x [..., I] and weight [O, I], with gradients."""
    if x.shape[-1] != weight.shape[-1]:
        raise ValueError(f"x has rows of {x.shape[-1]}, weight of {weight.shape[-1]}")
    shape = (*x.shape[:-1], weight.shape[0])
    if residual is not None and residual.shape != shape:
        raise ValueError(f"residual must have shape {shape}, got {tuple(residual.shape)}")
    _act_code(activation)
    return _Linear.apply(x, weight.contiguous(), None if bias is None else bias.contiguous(),
                         residual, activation).view(shape)


class HeadTransform(torch.nn.Module):
    """A block in front of a head: x + act(x W^T + b), as extra prediction heads have it, or
    act(x W^T + b) without the residual, as a masked model's head has it."""

    def __init__(self, hidden_size: int, *, activation: str = "silu", residual: bool = True,
                 bias: bool = True, device=None, dtype=None):
        super().__init__()
        _act_code(activation)
        kw = dict(device=device, dtype=dtype)
        self.weight = torch.nn.Parameter(
            torch.randn(hidden_size, hidden_size, **kw) * (0.02 if residual else hidden_size ** -0.5))
        self.bias = torch.nn.Parameter(torch.zeros(hidden_size, **kw)) if bias else None
        self.activation = activation
        self.residual = residual

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return fused_linear(x, self.weight, self.bias, x if self.residual else None,
                            activation=self.activation)
