"""Plain CPU restatement of the serving operators around the routed expert path — test
infrastructure only: the residual addition and root-mean-square norm, and E4M3 quantisation with a
scale per block of columns.  Values are fp64, widened exactly from their storage types; where a code
is decided by an fp32 product the product is formed in fp32, so both sides decide it from one value.
The operators' definitions are those of ``include/serving/moe_serving.h``.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import bf16_bits_to_f64, e4m3_round, round_bf16

__all__ = ["rmsnorm", "block_amax", "quantize_blocks_fp8", "spread_blocks", "FP8_BLOCK"]

FP8_BLOCK = 128
_FLOOR = np.float32(2.0 ** -100)


def rmsnorm(x_bits: np.ndarray, weight_bits: np.ndarray, eps: float, residual_bits=None):
    """h = bf16(x + residual) and y = h * w / sqrt(mean(h^2) + eps), both as fp64 values."""
    h = bf16_bits_to_f64(x_bits)
    if residual_bits is not None:
        h = round_bf16(h + bf16_bits_to_f64(residual_bits))
    rms = np.sqrt((h * h).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
    return h, h * bf16_bits_to_f64(weight_bits)[None, :] / rms


def spread_blocks(scale: np.ndarray, width: int) -> np.ndarray:
    """One value per block of 128 columns -> one per column."""
    return np.repeat(scale, FP8_BLOCK, axis=-1)[..., :width]


def block_amax(v: np.ndarray) -> np.ndarray:
    """max |v| of each block of 128 columns (NaN ignored), [rows, ceil(width/128)]."""
    rows, width = v.shape
    nb = -(-width // FP8_BLOCK)
    a = np.zeros((rows, nb * FP8_BLOCK), v.dtype)
    a[:, :width] = np.nan_to_num(np.abs(v), nan=0.0, posinf=np.inf)
    return a.reshape(rows, nb, FP8_BLOCK).max(axis=2)


def quantize_blocks_fp8(x: np.ndarray):
    """Codes and scales of fp32-representable values, decided in fp32: a = max(amax, 2^-100), scale
    a / 448 and factor 448 / a (both 1 for an all-zero block), codes e4m3_round(x * factor)."""
    xf = np.asarray(x, dtype=np.float32)
    amax = block_amax(xf)
    a = np.maximum(amax, _FLOOR)
    one = np.float32(1.0)
    scale = np.where(amax > 0, a / np.float32(448.0), one).astype(np.float32)
    factor = np.where(amax > 0, np.float32(448.0) / a, one).astype(np.float32)
    return e4m3_round((xf * spread_blocks(factor, xf.shape[1])).astype(np.float32)), scale
