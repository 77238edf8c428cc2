"""Activations kept in 8 bits between a forward and its backward pass (include/act8.h):
argument marshalling only."""
from __future__ import annotations

from typing import NamedTuple

import torch

from ._lib import load
from .api import _IO, _call


class Packed8(NamedTuple):
    """Rows of int8 (`data`, any shape) with one fp32 `scale` for each row of the last dim; they
    stand for data * scale in `dtype`."""
    data: torch.Tensor
    scale: torch.Tensor
    dtype: torch.dtype


def pack8(x) -> Packed8:
    """x (bf16 or fp32, contiguous, last dim a multiple of 8 up to 512) as whole numbers in
    [-127, 127] of its row's largest magnitude / 127. An element is off by at most half of that
    (rows whose largest magnitude is below 2^-119: and by what a subnormal fp32 scale loses);
    a row with a NaN or an infinity comes back as NaN."""
    if x.dtype not in _IO:
        raise TypeError(f"unsupported dtype {x.dtype} (bf16 or fp32)")
    if x.device.type != "cuda":
        raise ValueError("x must be on a HIP device")
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous, with at least one dim")
    D = x.shape[-1]
    if D % 8 or not 8 <= D <= 512:
        raise ValueError(f"the last dim must be a multiple of 8 in [8, 512] (got {D})")
    data = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _call(load().act8_pack, "act8_pack", x.device, None, x.data_ptr(), _IO[x.dtype],
          x.numel() // D, D, data.data_ptr(), scale.data_ptr())
    return Packed8(data, scale, x.dtype)


def _check_packed(p, name, dev):
    if p.dtype not in _IO:
        raise TypeError(f"{name}: unsupported dtype {p.dtype} (bf16 or fp32)")
    if p.data.dtype != torch.int8 or p.scale.dtype != torch.float32:
        raise TypeError(f"{name}: expected int8 data and fp32 scales")
    if p.data.dim() < 1 or p.scale.shape != p.data.shape[:-1]:
        raise ValueError(f"{name}: expected one scale for each row of data")
    if p.data.device != dev or p.scale.device != dev or dev.type != "cuda":
        raise ValueError(f"{name}: data and scale must be on one HIP device")
    if not (p.data.is_contiguous() and p.scale.is_contiguous()):
        raise ValueError(f"{name}: data and scale must be contiguous")


def unpack8(p: Packed8):
    """The values that `p` stands for, in p.dtype."""
    dev = p.data.device
    _check_packed(p, "p", dev)
    D = p.data.shape[-1]
    if D % 8 or not 8 <= D <= 512:
        raise ValueError(f"the last dim must be a multiple of 8 in [8, 512] (got {D})")
    x = torch.empty(p.data.shape, dtype=p.dtype, device=dev)
    _call(load().act8_unpack, "act8_unpack", dev, None, p.data.data_ptr(), p.scale.data_ptr(),
          _IO[p.dtype], p.data.numel() // D, D, x.data_ptr())
    return x
