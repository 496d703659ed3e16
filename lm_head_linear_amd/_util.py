"""What the bindings share: status codes as errors, types, pointers, tensor checks."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib


class FlceError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = code
        super().__init__(f"{where}: {flce_status_string(code)}" if where else flce_status_string(code))


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return _lib.BF16
    if dt == torch.float32:
        return _lib.F32
    raise ValueError(f"unsupported dtype {dt}; use torch.bfloat16 or torch.float32")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def flce_status_string(code: int) -> str:
    return _lib.load().flce_status_string(int(code)).decode()


def _check_tensor(name, t, shape, dtype, device):
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
