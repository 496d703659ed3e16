"""Sampling of the next token from logits, or from the head itself, with temperature,
top-k, top-p and min-p, from given uniform numbers (see include/flce.h for the
definition)."""
from __future__ import annotations

from typing import NamedTuple, Optional, Union

import torch

from . import _lib
from ._ops import _bytes, _on_gpu, _out, _rows, _run, _stream, _workspace
from ._util import _check_tensor, _dtype_code, _ptr

_Number = Union[float, int, torch.Tensor]


class Sampled(NamedTuple):
    """The tokens (int64) and the log probability each was drawn with, after the filters."""
    tokens: torch.Tensor
    logp: torch.Tensor


def _check_settings(temperature, top_k, top_p, min_p, softcap):
    """As the C-ABI takes them: value, array."""
    one = lambda v, neutral: (neutral, _ptr(v)) if hasattr(v, "data_ptr") else (v, None)  # noqa: E731
    t, ts = one(temperature, 1.0)
    k, ks = one(top_k, 0)
    p, ps = one(top_p, 1.0)
    m, ms = one(min_p, 0.0)
    return float(t), ts, int(k), ks, float(p), ps, float(m), ms, float(softcap)


def _settings(N, dev, temperature, top_k, top_p, min_p, softcap):
    for name, v, dt in (("temperature", temperature, torch.float32),
                        ("top_k", top_k, torch.int32), ("top_p", top_p, torch.float32),
                        ("min_p", min_p, torch.float32)):
        if isinstance(v, torch.Tensor):
            _check_tensor(name, v, (N,), dt, dev)
    if not isinstance(top_k, torch.Tensor) and not 0 <= int(top_k) < 1 << 31:
        raise ValueError(f"top_k must be in [0, 2^31), got {top_k}")
    return _check_settings(temperature, top_k, top_p, min_p, softcap)


def flce_sample_logits_workspace_size(N: int, V: int, dtype: torch.dtype) -> int:
    return int(_lib.load().flce_sample_logits_workspace_size(N, V, _dtype_code(dtype)))


def flce_sample_logits_check_args(logits, uniforms, *, N, V, ld_logits=None, temperature=1.0,
                                  top_k=0, top_p=1.0, min_p=0.0, softcap=0.0, tokens=None,
                                  logp=None, dtype=torch.float32, workspace=None) -> int:
    """The synchronous checks of sampling from logits (no GPU work); a status code."""
    return int(_lib.load().flce_sample_logits_check_args(
        _ptr(logits), V if ld_logits is None else int(ld_logits), N, V, _ptr(uniforms),
        *_check_settings(temperature, top_k, top_p, min_p, softcap), _ptr(tokens), _ptr(logp),
        None, _dtype_code(dtype), _ptr(workspace), _bytes(workspace)))


def flce_sample_logits(logits: torch.Tensor, uniforms: torch.Tensor, *,
                       temperature: _Number = 1.0, top_k: _Number = 0, top_p: _Number = 1.0,
                       min_p: _Number = 0.0, softcap: float = 0.0,
                       tokens: Optional[torch.Tensor] = None,
                       logp: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> Sampled:
    """A token of each row of logits [N, V] from uniform numbers [N] (float32, in [0, 1)).

    Each setting is a number, or a tensor [N] with each row's own (float32, top_k int32).
    temperature 0 is greedy. Nothing is synchronised.
    """
    if logits.dim() != 2:
        raise ValueError("logits must be [N, V]")
    N, V = logits.shape
    dev = logits.device
    _on_gpu("flce_sample_logits", dev)
    code = _dtype_code(logits.dtype)
    ld = _rows("logits", logits, N, V, logits.dtype, dev)
    _check_tensor("uniforms", uniforms, (N,), torch.float32, dev)
    settings = _settings(N, dev, temperature, top_k, top_p, min_p, softcap)
    tokens = _out("tokens", tokens, (N,), torch.int64, dev)
    logp = _out("logp", logp, (N,), torch.float32, dev)
    lib = _lib.load()
    workspace = _workspace("flce_sample_logits", workspace,
                           lib.flce_sample_logits_workspace_size(N, V, code), dev)
    _run("flce_sample_logits", dev, lib.flce_sample_logits, logits.data_ptr(), ld, N, V,
         uniforms.data_ptr(), *settings, tokens.data_ptr(), logp.data_ptr(), _stream(dev), code,
         workspace.data_ptr(), _bytes(workspace))
    return Sampled(tokens, logp)


def flce_sample_workspace_size(N: int, H: int, V: int, dtype: torch.dtype) -> int:
    return int(_lib.load().flce_sample_workspace_size(N, H, V, _dtype_code(dtype)))


def flce_sample_check_args(h, W, uniforms, *, N, H, V, temperature=1.0, top_k=0, top_p=1.0,
                           min_p=0.0, softcap=0.0, tokens=None, logp=None, dtype=torch.bfloat16,
                           workspace=None) -> int:
    """The synchronous checks of sampling from the head (no GPU work); a status code."""
    return int(_lib.load().flce_sample_check_args(
        _ptr(h), _ptr(W), N, H, V, _ptr(uniforms),
        *_check_settings(temperature, top_k, top_p, min_p, softcap), _ptr(tokens), _ptr(logp),
        None, _dtype_code(dtype), _ptr(workspace), _bytes(workspace)))


def flce_sample(h: torch.Tensor, W: torch.Tensor, uniforms: torch.Tensor, *,
                temperature: _Number = 1.0, top_k: _Number = 0, top_p: _Number = 1.0,
                min_p: _Number = 0.0, softcap: float = 0.0,
                tokens: Optional[torch.Tensor] = None, logp: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> Sampled:
    """:func:`flce_sample_logits` of the head W [V, H] at h [N, H]."""
    if h.dim() != 2 or W.dim() != 2:
        raise ValueError("h must be [N, H] and W [V, H]")
    (N, H), V = h.shape, W.shape[0]
    dev = W.device
    _on_gpu("flce_sample", dev)
    code = _dtype_code(W.dtype)
    _check_tensor("h", h, (N, H), W.dtype, dev)
    _check_tensor("W", W, (V, H), W.dtype, dev)
    _check_tensor("uniforms", uniforms, (N,), torch.float32, dev)
    settings = _settings(N, dev, temperature, top_k, top_p, min_p, softcap)
    tokens = _out("tokens", tokens, (N,), torch.int64, dev)
    logp = _out("logp", logp, (N,), torch.float32, dev)
    lib = _lib.load()
    workspace = _workspace("flce_sample", workspace, lib.flce_sample_workspace_size(N, H, V, code),
                           dev)
    _run("flce_sample", dev, lib.flce_sample, h.data_ptr(), W.data_ptr(), N, H, V,
         uniforms.data_ptr(), *settings, tokens.data_ptr(), logp.data_ptr(), _stream(dev), code,
         workspace.data_ptr(), _bytes(workspace))
    return Sampled(tokens, logp)
