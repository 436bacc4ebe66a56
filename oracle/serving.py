"""Plain CPU restatement of the serving operators around the routed expert path — test
infrastructure only: the residual addition and root-mean-square norm, and E4M3 quantisation with a
scale per block of columns.  Values are fp64, widened exactly from their storage types; where a code
is decided by an fp32 product the product is formed in fp32, so both sides decide it from one value.
The operators' definitions are those of ``include/serving/moe_serving.h``.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import bf16_bits_to_f64, e4m3_round, e4m3_to_f64, round_bf16, route, silu

__all__ = ["rmsnorm", "block_amax", "quantize_blocks_fp8", "spread_blocks", "FP8_BLOCK",
           "fp8_block_matrix", "few_tokens"]

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


def fp8_block_matrix(w, e: int) -> np.ndarray:
    """Expert e's [N, K] matrix: value(code) * scale of its 128 x 128 block."""
    v = e4m3_to_f64(w["codes"][e])
    rows = np.repeat(np.asarray(w["scales"][e], np.float64), FP8_BLOCK, axis=0)[: v.shape[0]]
    return v * spread_blocks(rows, v.shape[1])


def few_tokens(logits: np.ndarray, x_bits: np.ndarray, gate, up, down, top_k: int, renormalize: bool = True):
    """The routed layer without rounding in between.  gate, up, down: expert id -> [N, K] fp64 matrix.

    Returns (out, ids, w, spread, noise): ``spread[t, n] = sum_j w_j sum_k |h_k| |Wd[n, k]|``, what a relative
    error of h can move out by at most, and ``noise[t, n]``, what one unit of relative fp32 error in the
    products of the first stage can move it by: h = silu(g) u with |silu'| <= 1.1, so
    |dh| <= 1.1 |u| sum |x||Wg| + |silu(g)| sum |x||Wu|."""
    x = bf16_bits_to_f64(x_bits)
    ids, w = route(logits, top_k, renormalize)
    H = x.shape[1]
    out, spread, noise = (np.zeros((x.shape[0], H)) for _ in range(3))
    mats = {int(e): (gate(int(e)), up(int(e)), down(int(e))) for e in np.unique(ids)}
    for t in range(x.shape[0]):
        for j in range(top_k):
            wg, wu, wd = mats[int(ids[t, j])]
            g, u = wg @ x[t], wu @ x[t]
            h = silu(g) * u
            dh = 1.1 * np.abs(u) * (np.abs(wg) @ np.abs(x[t])) + np.abs(silu(g)) * (np.abs(wu) @ np.abs(x[t]))
            wt = float(w[t, j])
            out[t] += wt * (wd @ h)
            spread[t] += wt * (np.abs(wd) @ np.abs(h))
            noise[t] += wt * (np.abs(wd) @ dh)
    return out, ids, w, spread, noise
