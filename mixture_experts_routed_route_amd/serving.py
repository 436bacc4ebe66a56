"""PyTorch-facing binding of the serving operators (``include/serving/moe_serving.h``): the norm in
front of the layer and block-scaled E4M3 quantisation.

As in ``ops``: argument checks and marshalling only; every step runs in the HIP library on the
tensors' device and its current stream.
"""
from __future__ import annotations

from typing import Optional

import torch

from ._lib import check, lib
from .ops import Routing, _dev, _need, _numel_at_least

__all__ = ["FP8_BLOCK", "moe_rmsnorm", "moe_quantize_fp8_block"]

FP8_BLOCK = 128   # columns under one scale (weights: 128 x 128 blocks)


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _launch(name: str, device: torch.device, *args) -> None:
    """The call on ``device``'s current stream, with that device current (a launch goes to the
    current device's code object, whatever device its stream belongs to)."""
    f = getattr(lib(), name)
    if device.index is None or device.index == torch.cuda.current_device():
        check(f(*args, torch.cuda.current_stream(device).cuda_stream))
    else:
        with torch.cuda.device(device):
            check(f(*args, torch.cuda.current_stream(device).cuda_stream))


def _ptr(t: Optional[torch.Tensor], dtype: torch.dtype, name: str, like: torch.Tensor) -> Optional[int]:
    """``t``'s address (None stays None), on the same device as ``like``."""
    if t is None:
        return None
    p = _dev(t, dtype, name)
    _need(t.device == like.device, f"{name} is on {t.device}, x on {like.device}")
    return p


def moe_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """h = x + residual (rounded to bf16), then h * weight / sqrt(mean(h^2) + eps) over rows of bf16
    ``x`` [rows, k].

    ``residual`` takes h in place, or ``residual_out`` does when given.  Outputs: bf16 ``y`` (allocated
    and returned when neither ``y`` nor ``q`` is given), and with ``q`` (uint8 [rows, k]) E4M3 codes of
    the unrounded norm, under one fp32 scale per row (``scale`` [rows]) or per 128 columns (``scale``
    [rows, ceil(k/128)]).  Returns ``y`` (None with codes only)."""
    who = "moe_rmsnorm"
    _need(x.dim() == 2, f"{who}: x is {tuple(x.shape)}; needs [rows, k]")
    rows, k = x.shape
    _need(weight.dim() == 1 and weight.shape[0] == k, f"{who}: weight is {tuple(weight.shape)}; needs ({k},)")
    _need(residual is not None or residual_out is None, f"{who}: residual_out without residual")
    if residual is not None and residual_out is None:
        residual_out = residual
    _need((q is None) == (scale is None), f"{who}: q and scale go together")
    if y is None and q is None:
        y = torch.empty_like(x)
    for t, name in ((residual, "residual"), (residual_out, "residual_out"), (y, "y"), (q, "q")):
        _need(t is None or t.shape == x.shape, f"{who}: {name} is {tuple(t.shape) if t is not None else ()}; "
                                               f"needs {(rows, k)}")
    block = 0
    if scale is not None:
        block = FP8_BLOCK if scale.dim() == 2 else 0
        want = (rows, _blocks(k)) if block else (rows,)
        _need(tuple(scale.shape) == want, f"{who}: scale is {tuple(scale.shape)}; needs {(rows,)} or {(rows, _blocks(k))}")
    bf = torch.bfloat16
    _launch(who, x.device, _dev(x, bf, "x"), _ptr(residual, bf, "residual", x), _ptr(weight, bf, "weight", x),
            float(eps), rows, k, _ptr(residual_out, bf, "residual_out", x), _ptr(y, bf, "y", x),
            _ptr(q, torch.uint8, "q", x), _ptr(scale, torch.float32, "scale", x), block)
    return y


def moe_quantize_fp8_block(x: torch.Tensor, q: torch.Tensor, scale: torch.Tensor,
                           routing: Optional[Routing] = None) -> None:
    """E4M3 codes ``q`` of bf16 rows ``x`` [rows, k] with one fp32 scale per 128 columns (``scale``
    [rows, ceil(k/128)]); with ``routing`` only the real sorted rows are written."""
    who = "moe_quantize_fp8_block"
    _need(x.dim() == 2, f"{who}: x is {tuple(x.shape)}; needs [rows, k]")
    rows, k = x.shape
    _need(tuple(q.shape) == (rows, k), f"{who}: q is {tuple(q.shape)}; needs {(rows, k)}")
    _need(tuple(scale.shape) == (rows, _blocks(k)), f"{who}: scale is {tuple(scale.shape)}; needs {(rows, _blocks(k))}")
    if routing is not None:
        _numel_at_least(routing.sorted_ids, rows, f"{who}: routing.sorted_ids")
    _launch(who, x.device, _dev(x, torch.bfloat16, "x"), rows, k,
            _ptr(routing.sorted_ids, torch.int32, "sorted_ids", x) if routing is not None else None,
            routing.num_pairs if routing is not None else 0, _ptr(q, torch.uint8, "q", x),
            _ptr(scale, torch.float32, "scale", x))
