"""Checks of the tensors that a call takes, with the words for what is wrong."""
from __future__ import annotations

from typing import Optional

import torch


def refuse(t, name: str, dtype, shape, device: Optional[int] = None, layout: str = "") -> None:
    """Raise for what is wrong with t, which is not a `dtype` tensor of
    `shape` on CUDA device `device` with the layout that is described."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: need a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: need {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} is not on a CUDA device")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on device {t.get_device()}, the first tensor on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, need {tuple(shape)}")
    raise ValueError(f"{name}: strides {t.stride()}: {layout or 'must be contiguous'}")


def dense(t: Optional[torch.Tensor], name: str, dtype, *shape,
          device: Optional[int] = None) -> Optional[torch.Tensor]:
    """A contiguous CUDA tensor (or None), on `device` where given."""
    if t is not None and not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype
                              and tuple(t.shape) == shape and t.is_contiguous()
                              and (device is None or t.get_device() == device)):
        refuse(t, name, dtype, shape, device)
    return t


current_device = torch._C._cuda_getDevice


def refuse_device(device: int, current: int) -> None:
    raise ValueError(f"the tensors are on device {device}, the current device is {current}: the "
                     "library launches on the current one (torch.cuda.device changes it)")
