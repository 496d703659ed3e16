"""The operators around the head: the norm in front of it and the lookup in the
table it shares with the embedding (see include/flce.h for the contracts).

Like the head's own bindings these only marshal arguments. Matrices may be views
with a row stride (unit stride along a row); outputs and workspaces may be passed
in, so that a call allocates nothing.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._util import FlceError, _check_tensor, _dtype_code, _ptr


def _rows(name, t, N, H, dtype, dev):
    """Checks an [N, H] matrix with unit stride along its rows; its row stride."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (N, H):
        raise ValueError(f"{name} must have shape {(N, H)}, got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.is_contiguous():
        return H
    if H > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    if N == 1:
        return H
    if t.stride(0) < H:
        raise ValueError(f"{name} must not have overlapping rows (row stride {t.stride(0)})")
    return t.stride(0)


def _on_gpu(where, dev):
    if dev.type != "cuda":
        raise ValueError(f"{where} runs on a GPU; tensors are on {dev}")


def _run(where, dev, fn, *args):
    """fn(*args) on dev, which a call makes current only where it is not."""
    if dev.index == torch.cuda.current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != _lib.OK:
        raise FlceError(rc, where)


def _stream(dev):
    """dev's current stream as a handle (torch.cuda.current_stream builds an object:
    2 us of a call's 11)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def _workspace(where, ws, need, dev):
    if need == 0:                        # sizes the library does not take
        raise FlceError(_lib.ERR_ARG, where)
    if ws is not None and (ws.device != dev or not ws.is_contiguous()):
        raise ValueError(f"the workspace must be contiguous memory of {dev}, got {ws.device}")
    return torch.empty(need, dtype=torch.uint8, device=dev) if _bytes(ws) < need else ws


# ---- root-mean-square norm -----------------------------------------------------------


def flce_rms_norm_check_args(x, weight, residual=None, *, N, H, ld_x=None, ld_res=None, eps=1e-6,
                             weight_offset=0.0, y=None, ld_y=None, s=None, ld_s=None, rstd=None,
                             dtype=torch.bfloat16, weight_dtype=None) -> int:
    """The norm's synchronous checks (no GPU work); a status code."""
    ld = lambda v: H if v is None else int(v)  # noqa: E731
    return int(_lib.load().flce_rms_norm_check_args(
        _ptr(x), ld(ld_x), _ptr(residual), ld(ld_res), _ptr(weight), N, H, float(eps),
        float(weight_offset), _ptr(y), ld(ld_y), _ptr(s), ld(ld_s), _ptr(rstd), None,
        _dtype_code(dtype), _dtype_code(weight_dtype or dtype)))


def flce_rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                  *, eps: float = 1e-6, weight_offset: float = 0.0,
                  y: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None,
                  rstd: Optional[torch.Tensor] = None):
    """RMS norm of the rows of x [N, H], after adding the residual: (y, s, rstd).

    s = x + residual rounded to the rows' type (x itself without a residual),
    y = s * rstd * (weight + weight_offset). weight [H] has the rows' type, or
    float32 with bf16 rows. ``y`` may be x and ``s`` the residual (in place).
    """
    if x.dim() != 2:
        raise ValueError("x must be [N, H]")
    N, H = x.shape
    dev, dt = x.device, x.dtype
    _on_gpu("flce_rms_norm", dev)
    code, wcode = _dtype_code(dt), _dtype_code(weight.dtype)
    _check_tensor("weight", weight, (H,), weight.dtype, dev)
    ld_x, ld_r, ld_s, ld_y = _rows("x", x, N, H, dt, dev), H, H, H
    if y is None:
        y = torch.empty(N, H, dtype=dt, device=dev)
    else:
        ld_y = _rows("y", y, N, H, dt, dev)
    if rstd is None:
        rstd = torch.empty(N, dtype=torch.float32, device=dev)
    else:
        _check_tensor("rstd", rstd, (N,), torch.float32, dev)
    if residual is not None:
        ld_r = _rows("residual", residual, N, H, dt, dev)
        if s is None:
            s = torch.empty(N, H, dtype=dt, device=dev)
        else:
            ld_s = _rows("s", s, N, H, dt, dev)
    elif s is not None:
        raise ValueError("s is written only with a residual")
    _run("flce_rms_norm", dev, _lib.load().flce_rms_norm, x.data_ptr(), ld_x, _ptr(residual), ld_r,
         weight.data_ptr(), N, H, float(eps), float(weight_offset), y.data_ptr(), ld_y, _ptr(s),
         ld_s, rstd.data_ptr(),
         _stream(dev), code, wcode)
    return y, x if residual is None else s, rstd


def flce_rms_norm_backward_workspace_size(N: int, H: int) -> int:
    return int(_lib.load().flce_rms_norm_backward_workspace_size(N, H))


def flce_rms_norm_backward_check_args(dy, s, weight, rstd, ds=None, *, N, H, ld_dy=None,
                                      ld_ds=None, ld_s=None, weight_offset=0.0, dx=None,
                                      ld_dx=None, dweight=None, accumulate_dweight=False,
                                      dtype=torch.bfloat16, weight_dtype=None,
                                      workspace=None) -> int:
    """The norm's backward's synchronous checks (no GPU work); a status code."""
    ld = lambda v: H if v is None else int(v)  # noqa: E731
    return int(_lib.load().flce_rms_norm_backward_check_args(
        _ptr(dy), ld(ld_dy), _ptr(ds), ld(ld_ds), _ptr(s), ld(ld_s), _ptr(weight), _ptr(rstd), N,
        H, float(weight_offset), _ptr(dx), ld(ld_dx), _ptr(dweight), int(bool(accumulate_dweight)),
        None, _dtype_code(dtype), _dtype_code(weight_dtype or dtype), _ptr(workspace),
        _bytes(workspace)))


def flce_rms_norm_backward(dy: torch.Tensor, s: torch.Tensor, weight: torch.Tensor,
                           rstd: torch.Tensor, ds: Optional[torch.Tensor] = None, *,
                           weight_offset: float = 0.0, dx: Optional[torch.Tensor] = None,
                           dweight: Optional[torch.Tensor] = None, want_dweight: bool = True,
                           accumulate_dweight: bool = False,
                           workspace: Optional[torch.Tensor] = None):
    """Gradients of :func:`flce_rms_norm`: (dx, dweight).

    dx is the gradient of x and of the residual alike; ``ds`` is the gradient
    that reaches s itself. dweight is None unless wanted (``want_dweight``) and
    is added to the tensor passed in with ``accumulate_dweight``.
    """
    if dy.dim() != 2:
        raise ValueError("dy must be [N, H]")
    N, H = dy.shape
    dev, dt = dy.device, dy.dtype
    _on_gpu("flce_rms_norm_backward", dev)
    code, wcode = _dtype_code(dt), _dtype_code(weight.dtype)
    _check_tensor("weight", weight, (H,), weight.dtype, dev)
    _check_tensor("rstd", rstd, (N,), torch.float32, dev)
    ld_dy, ld_s = _rows("dy", dy, N, H, dt, dev), _rows("s", s, N, H, dt, dev)
    ld_ds = H if ds is None else _rows("ds", ds, N, H, dt, dev)
    ld_dx = H
    if dx is None:
        dx = torch.empty(N, H, dtype=dt, device=dev)
    else:
        ld_dx = _rows("dx", dx, N, H, dt, dev)
    if accumulate_dweight and dweight is None:
        raise ValueError("accumulate_dweight needs the dweight tensor to add to")
    if dweight is not None:
        _check_tensor("dweight", dweight, (H,), weight.dtype, dev)
    elif want_dweight:
        dweight = torch.empty(H, dtype=weight.dtype, device=dev)
    if dweight is not None:
        workspace = _workspace("flce_rms_norm_backward", workspace,
                               flce_rms_norm_backward_workspace_size(N, H), dev)
    _run("flce_rms_norm_backward", dev, _lib.load().flce_rms_norm_backward, dy.data_ptr(), ld_dy,
         _ptr(ds), ld_ds, s.data_ptr(), ld_s, weight.data_ptr(), rstd.data_ptr(), N, H,
         float(weight_offset), dx.data_ptr(), ld_dx, _ptr(dweight),
         int(bool(accumulate_dweight)), _stream(dev), code, wcode,
         _ptr(workspace), _bytes(workspace))
    return dx, dweight


def _flat_rows(t):
    """t [..., H] as rows that the norm reads in place, or a copy of them."""
    t = t.reshape(-1, t.shape[-1])
    inplace = t.stride(1) == 1 and (t.stride(0) >= t.shape[1] or t.shape[0] <= 1)
    return t if inplace else t.contiguous()


# The functions return rows, which their wrappers shape: a view made inside a function could
# not be changed in place by its caller.


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, weight_offset):
        ctx.shape = x.shape
        y, s, rstd = flce_rms_norm(_flat_rows(x), weight,
                                   None if residual is None else _flat_rows(residual), eps=eps,
                                   weight_offset=weight_offset)
        ctx.save_for_backward(s, weight, rstd)
        ctx.weight_offset = weight_offset
        ctx.has_residual = residual is not None
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, s)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        s, weight, rstd = ctx.saved_tensors
        if dy is None:                       # only the sum was used
            dx, dw = ds, None
        else:
            dx, dw = flce_rms_norm_backward(
                dy.contiguous(), s, weight, rstd, None if ds is None else ds.contiguous(),
                weight_offset=ctx.weight_offset, want_dweight=ctx.needs_input_grad[1])
        # one tensor for both: autograd then copies it where a leaf would keep it
        dx = dx.reshape(ctx.shape)
        return dx, dw, dx if ctx.has_residual else None, None, None


def fused_rms_norm(x: torch.Tensor, weight: torch.Tensor,
                   residual: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
                   weight_offset: float = 0.0):
    """RMS norm of x [..., H] with gradients; with a residual, (y, x + residual).

    The gradients of x and of the residual are the same tensor of values: both
    inputs enter through their sum.
    """
    out = _RMSNorm.apply(x, weight.contiguous(), residual, float(eps), float(weight_offset))
    if residual is None:
        return out.view(x.shape)
    return out[0].view(x.shape), out[1].view(x.shape)


# ---- embedding -----------------------------------------------------------------------


def flce_embedding_check_args(tokens, W, *, N, H, V, padding_index=-100, scale=1.0, out=None,
                              ld_out=None, dtype=torch.bfloat16, status=None) -> int:
    """The lookup's synchronous checks (no GPU work); a status code."""
    return int(_lib.load().flce_embedding_check_args(
        _ptr(tokens), _ptr(W), N, H, V, int(padding_index), float(scale), _ptr(out),
        H if ld_out is None else int(ld_out), None, _dtype_code(dtype), _ptr(status)))


def flce_embedding(tokens: torch.Tensor, W: torch.Tensor, *, scale: float = 1.0,
                   padding_index: int = -100, out: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[i] = scale * W[tokens[i]] (rounded once) for int64 tokens [N], W [V, H].

    A token equal to ``padding_index`` gives zeros; one outside [0, V) gives NaN
    (and FLCE_ERR_LABEL in ``status``, a device int32).
    """
    if W.dim() != 2 or tokens.dim() != 1:
        raise ValueError("tokens must be [N] and W [V, H]")
    (V, H), N = W.shape, tokens.shape[0]
    dev = W.device
    _on_gpu("flce_embedding", dev)
    code = _dtype_code(W.dtype)
    _check_tensor("tokens", tokens, (N,), torch.int64, dev)
    _check_tensor("W", W, (V, H), W.dtype, dev)
    if status is not None:
        _check_tensor("status", status, (), torch.int32, dev)
    ld = H
    if out is None:
        out = torch.empty(N, H, dtype=W.dtype, device=dev)
    else:
        ld = _rows("out", out, N, H, W.dtype, dev)
    _run("flce_embedding", dev, _lib.load().flce_embedding, tokens.data_ptr(), W.data_ptr(), N, H,
         V, int(padding_index), float(scale), out.data_ptr(), ld,
         _stream(dev), code, _ptr(status))
    return out


def flce_embedding_backward_workspace_size(N: int, H: int, V: int) -> int:
    return int(_lib.load().flce_embedding_backward_workspace_size(N, H, V))


def flce_embedding_backward_check_args(tokens, dout, *, N, H, V, dW, ld_dout=None,
                                       padding_index=-100, scale=1.0, accumulate_dW=False,
                                       dtype=torch.bfloat16, grad_dtype=None, workspace=None,
                                       status=None) -> int:
    """The lookup's gradient's synchronous checks (no GPU work); a status code."""
    return int(_lib.load().flce_embedding_backward_check_args(
        _ptr(tokens), _ptr(dout), H if ld_dout is None else int(ld_dout), N, H, V,
        int(padding_index), float(scale), _ptr(dW), int(bool(accumulate_dW)), None,
        _dtype_code(dtype), _dtype_code(grad_dtype or dtype), _ptr(workspace), _bytes(workspace),
        _ptr(status)))


def flce_embedding_backward(tokens: torch.Tensor, dout: torch.Tensor, V: int, *,
                            scale: float = 1.0, padding_index: int = -100,
                            dW: Optional[torch.Tensor] = None, accumulate_dW: bool = False,
                            grad_dtype: Optional[torch.dtype] = None,
                            workspace: Optional[torch.Tensor] = None,
                            status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The table's gradient of :func:`flce_embedding`: dW [V, H].

    dW[v] = scale * (sum of dout[i] over tokens[i] == v), summed in float32 in the
    tokens' order. With ``accumulate_dW`` it is added to the dW passed in (the
    head's gradient of a tied table): only the rows of the tokens are touched.
    """
    if dout.dim() != 2 or tokens.dim() != 1:
        raise ValueError("tokens must be [N] and dout [N, H]")
    N, H = dout.shape
    dev, dt = dout.device, dout.dtype
    _on_gpu("flce_embedding_backward", dev)
    gdt = grad_dtype if grad_dtype is not None else dt if dW is None else dW.dtype
    code, gcode = _dtype_code(dt), _dtype_code(gdt)
    _check_tensor("tokens", tokens, (N,), torch.int64, dev)
    ld = _rows("dout", dout, N, H, dt, dev)
    if dW is None:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs the dW tensor to add to")
        dW = torch.empty(V, H, dtype=gdt, device=dev)
    else:
        _check_tensor("dW", dW, (V, H), gdt, dev)
    if status is not None:
        _check_tensor("status", status, (), torch.int32, dev)
    workspace = _workspace("flce_embedding_backward", workspace,
                           flce_embedding_backward_workspace_size(N, H, V), dev)
    _run("flce_embedding_backward", dev, _lib.load().flce_embedding_backward, tokens.data_ptr(),
         dout.data_ptr(), ld, N, H, V, int(padding_index), float(scale), dW.data_ptr(),
         int(bool(accumulate_dW)), _stream(dev), code, gcode,
         workspace.data_ptr(), _bytes(workspace), _ptr(status))
    return dW


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, W, scale, padding_index):
        ctx.save_for_backward(tokens)
        ctx.args = (W.shape[0], scale, padding_index)
        return flce_embedding(tokens, W, scale=scale, padding_index=padding_index)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (tokens,) = ctx.saved_tensors
        V, scale, padding_index = ctx.args
        dW = flce_embedding_backward(tokens, dout.contiguous(), V, scale=scale,
                                     padding_index=padding_index)
        return None, dW, None, None


def fused_embedding(tokens: torch.Tensor, W: torch.Tensor, *, scale: float = 1.0,
                    padding_index: int = -100) -> torch.Tensor:
    """scale * W[tokens] for tokens of any shape, with the table's gradient."""
    flat = tokens.reshape(-1).contiguous()
    out = _Embedding.apply(flat, W.contiguous(), float(scale), int(padding_index))
    return out.view(*tokens.shape, W.shape[1])


# ---- token log probabilities ---------------------------------------------------------


class TokenLogprobs(NamedTuple):
    """What :func:`flce_logprobs` returns; logp is None without given tokens, the
    alternatives are [N, 0] with top_k = 0."""
    logp: Optional[torch.Tensor]
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logp: torch.Tensor
    top_ids: torch.Tensor


def flce_logprobs_workspace_size(N: int, H: int, V: int, dtype: torch.dtype,
                                 top_k: int = 0) -> int:
    return int(_lib.load().flce_logprobs_workspace_size(N, H, V, _dtype_code(dtype), int(top_k)))


def flce_logprobs_check_args(h, W, tokens=None, *, N, H, V, ignore_index=-100, softcap=0.0,
                             temperature=1.0, top_k=0, logp=None, entropy=None, lse=None,
                             top_logp=None, top_ids=None, dtype=torch.bfloat16, workspace=None,
                             status=None) -> int:
    """The log probabilities' synchronous checks (no GPU work); a status code."""
    return int(_lib.load().flce_logprobs_check_args(
        _ptr(h), _ptr(W), _ptr(tokens), N, H, V, int(ignore_index), float(softcap),
        float(temperature), int(top_k), _ptr(logp), _ptr(entropy), _ptr(lse), _ptr(top_logp),
        _ptr(top_ids), None, _dtype_code(dtype), _ptr(workspace), _bytes(workspace),
        _ptr(status)))


def _out(name, t, shape, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _check_tensor(name, t, shape, dtype, dev)
    return t


def flce_logprobs(h: torch.Tensor, W: torch.Tensor, tokens: Optional[torch.Tensor] = None, *,
                  ignore_index: int = -100, softcap: float = 0.0, temperature: float = 1.0,
                  top_k: int = 0, logp: Optional[torch.Tensor] = None,
                  entropy: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  top_logp: Optional[torch.Tensor] = None,
                  top_ids: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None) -> TokenLogprobs:
    """Log probabilities of tokens [N] under the head W [V, H] at h [N, H].

    Also each position's entropy (nats), log-sum-exp and ``top_k`` (at most 32)
    best alternatives, by logit and then by lowest id. Rows whose token is
    ``ignore_index`` are left out: 0, and ids -1 with -inf. Without ``tokens``
    every row counts and ``logp`` is None. Nothing is synchronised.
    """
    if h.dim() != 2 or W.dim() != 2:
        raise ValueError("h must be [N, H] and W [V, H]")
    (N, H), V = h.shape, W.shape[0]
    dev = W.device
    _on_gpu("flce_logprobs", dev)
    code, f32 = _dtype_code(W.dtype), torch.float32
    _check_tensor("h", h, (N, H), W.dtype, dev)
    _check_tensor("W", W, (V, H), W.dtype, dev)
    top_k = int(top_k)
    if not 0 <= top_k <= _lib.MAX_TOP:
        raise ValueError(f"top_k must be 0 to {_lib.MAX_TOP}, got {top_k}")
    if tokens is not None:
        _check_tensor("tokens", tokens, (N,), torch.int64, dev)
        logp = _out("logp", logp, (N,), f32, dev)
    elif logp is not None:
        raise ValueError("logp needs tokens")
    entropy = _out("entropy", entropy, (N,), f32, dev)
    lse = _out("lse", lse, (N,), f32, dev)
    top_logp = _out("top_logp", top_logp, (N, top_k), f32, dev)
    top_ids = _out("top_ids", top_ids, (N, top_k), torch.int64, dev)
    if status is not None:
        _check_tensor("status", status, (), torch.int32, dev)
    lib = _lib.load()
    need = lib.flce_logprobs_workspace_size(N, H, V, code, top_k)
    workspace = _workspace("flce_logprobs", workspace, need, dev)
    _run("flce_logprobs", dev, lib.flce_logprobs, h.data_ptr(), W.data_ptr(), _ptr(tokens), N, H,
         V, int(ignore_index), float(softcap), float(temperature), top_k, _ptr(logp),
         entropy.data_ptr(), lse.data_ptr(), top_logp.data_ptr() if top_k else None,
         top_ids.data_ptr() if top_k else None, _stream(dev), code,
         workspace.data_ptr(), _bytes(workspace), _ptr(status))
    return TokenLogprobs(logp, entropy, lse, top_logp, top_ids)


def flce_logprobs_backward_workspace_size(N: int, H: int, V: int, dtype: torch.dtype,
                                          grad_dtype: Optional[torch.dtype] = None) -> int:
    return int(_lib.load().flce_logprobs_backward_workspace_size(
        N, H, V, _dtype_code(dtype), _dtype_code(grad_dtype or dtype)))


def flce_logprobs_backward_check_args(h, W, tokens, lse, entropy=None, grad_logp=None,
                                      grad_entropy=None, *, N, H, V, ignore_index=-100,
                                      softcap=0.0, temperature=1.0, dH=None, dW=None,
                                      accumulate_dW=False, dtype=torch.bfloat16, grad_dtype=None,
                                      workspace=None, status=None) -> int:
    """The log probabilities' backward's synchronous checks; a status code."""
    return int(_lib.load().flce_logprobs_backward_check_args(
        _ptr(h), _ptr(W), _ptr(tokens), _ptr(lse), _ptr(entropy), _ptr(grad_logp),
        _ptr(grad_entropy), N, H, V, int(ignore_index), float(softcap), float(temperature),
        _ptr(dH), _ptr(dW), int(bool(accumulate_dW)), None, _dtype_code(dtype),
        _dtype_code(grad_dtype or dtype), _ptr(workspace), _bytes(workspace), _ptr(status)))


def flce_logprobs_backward(h: torch.Tensor, W: torch.Tensor, tokens: torch.Tensor,
                           lse: torch.Tensor, entropy: Optional[torch.Tensor],
                           grad_logp: Optional[torch.Tensor],
                           grad_entropy: Optional[torch.Tensor] = None, *,
                           ignore_index: int = -100, softcap: float = 0.0,
                           temperature: float = 1.0, dH: Optional[torch.Tensor] = None,
                           dW: Optional[torch.Tensor] = None, accumulate_dW: bool = False,
                           grad_dtype: Optional[torch.dtype] = None,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None):
    """(dH, dW) of :func:`flce_logprobs` for the gradients of logp and entropy.

    ``lse`` and (with ``grad_entropy``) ``entropy`` are what the forward returned
    for the same inputs and options.
    """
    if h.dim() != 2 or W.dim() != 2:
        raise ValueError("h must be [N, H] and W [V, H]")
    (N, H), V = h.shape, W.shape[0]
    dev = W.device
    _on_gpu("flce_logprobs_backward", dev)
    gdt = W.dtype if grad_dtype is None else grad_dtype
    code, gcode = _dtype_code(W.dtype), _dtype_code(gdt)
    _check_tensor("h", h, (N, H), W.dtype, dev)
    _check_tensor("W", W, (V, H), W.dtype, dev)
    _check_tensor("tokens", tokens, (N,), torch.int64, dev)
    for name, t in (("lse", lse), ("entropy", entropy), ("grad_logp", grad_logp),
                    ("grad_entropy", grad_entropy)):
        if t is not None:
            _check_tensor(name, t, (N,), torch.float32, dev)
    dH = _out("dH", dH, (N, H), gdt, dev)
    if dW is None and accumulate_dW:
        raise ValueError("accumulate_dW needs the dW tensor to add to")
    dW = _out("dW", dW, (V, H), gdt, dev)
    if status is not None:
        _check_tensor("status", status, (), torch.int32, dev)
    lib = _lib.load()
    need = lib.flce_logprobs_backward_workspace_size(N, H, V, code, gcode)
    if need == 0 and W.dtype == torch.float32 and gdt == torch.bfloat16:
        raise FlceError(_lib.ERR_UNSUPPORTED, "flce_logprobs_backward_workspace_size")
    workspace = _workspace("flce_logprobs_backward", workspace, need, dev)
    _run("flce_logprobs_backward", dev, lib.flce_logprobs_backward, h.data_ptr(), W.data_ptr(),
         tokens.data_ptr(), lse.data_ptr(), _ptr(entropy), _ptr(grad_logp), _ptr(grad_entropy), N,
         H, V, int(ignore_index), float(softcap), float(temperature), dH.data_ptr(),
         dW.data_ptr(), int(bool(accumulate_dW)), _stream(dev), code,
         gcode, workspace.data_ptr(), _bytes(workspace), _ptr(status))
    return dH, dW


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, tokens, ignore_index, softcap, temperature, top_k):
        out = flce_logprobs(h, W, tokens, ignore_index=ignore_index, softcap=softcap,
                            temperature=temperature, top_k=top_k)
        ctx.save_for_backward(h, W, tokens, out.lse, out.entropy)
        ctx.kw = dict(ignore_index=ignore_index, softcap=softcap, temperature=temperature)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(out.lse, out.top_logp, out.top_ids)
        return tuple(out)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logp, grad_entropy, *_):
        h, W, tokens, lse, entropy = ctx.saved_tensors
        if grad_logp is None and grad_entropy is None:
            return (None,) * 7
        flat = lambda g: None if g is None else g.contiguous()  # noqa: E731
        dH, dW = flce_logprobs_backward(h, W, tokens, lse, entropy, flat(grad_logp),
                                        flat(grad_entropy), **ctx.kw)
        return dH, dW, None, None, None, None, None


def token_logprobs(hidden_states: torch.Tensor, tokens: Optional[torch.Tensor],
                   lm_weight: torch.Tensor, *, ignore_index: int = -100, softcap: float = 0.0,
                   temperature: float = 1.0, top_k: int = 0) -> TokenLogprobs:
    """:func:`flce_logprobs` for hidden_states [..., H] and tokens [...], with the
    gradients of logp and entropy (the other outputs have none). Without tokens
    there are no gradients."""
    lead, H = hidden_states.shape[:-1], hidden_states.shape[-1]
    h, W = hidden_states.reshape(-1, H).contiguous(), lm_weight.contiguous()
    if h.data_ptr() % 16:                # a slice that starts inside odd rows
        h = h.clone()
    y = None if tokens is None else tokens.reshape(-1).contiguous()
    if y is None or not torch.is_grad_enabled() or not (h.requires_grad or W.requires_grad):
        out = flce_logprobs(h.detach(), W.detach(), y, ignore_index=ignore_index, softcap=softcap,
                            temperature=temperature, top_k=top_k)
    else:
        out = _TokenLogprobs.apply(h, W, y, ignore_index, float(softcap), float(temperature),
                                   int(top_k))
    logp, entropy, lse, top_logp, top_ids = out
    return TokenLogprobs(None if logp is None else logp.view(lead), entropy.view(lead),
                         lse.view(lead), top_logp.view(*lead, int(top_k)),
                         top_ids.view(*lead, int(top_k)))
