"""PyTorch-facing binding of the training operators (``include/training/moe_training.h``): SiLU * up with
dropout and its backward, the grouped products for the gradients of inputs and weights, and the gradient
of the router's logits.

As in ``ops``: argument checks and marshalling only; every step runs in the HIP library on the
tensors' device and its current stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .ops import Bf16Weight, Routing, _check_routing, _numel_at_least
from .serving import _index, _launch, _ptr

__all__ = ["moe_silu_mul_dropout", "moe_silu_mul_backward", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad",
           "moe_route_backward"]


# Messages are made when a check fails only: made beforehand they took half of a small call's time.
def _shape(t: Optional[torch.Tensor], shape: Tuple[int, ...], who: str, name: str) -> None:
    if t is not None and t.shape != shape:
        raise ValueError(f"{who}: {name} is not of shape {shape} (got {tuple(t.shape)})")


def _check_p(p: float, rng: Optional[torch.Tensor], who: str) -> float:
    p = float(p)
    if not 0.0 <= p < 1.0:
        raise ValueError(f"{who}: p is {p}; needs [0, 1)")
    if rng is None and p != 0.0:
        raise ValueError(f"{who}: dropout needs rng")
    if rng is not None and rng.shape != (2,):
        raise ValueError(f"{who}: rng needs seed and offset, shape (2,)")
    return p


def _rows(t: torch.Tensor, routing: Optional[Routing], who: str, name: str) -> Tuple[int, int]:
    """Rows and columns of a call over sorted rows (all rows without a routing)."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{who}: {name} is {tuple(shape)}; needs [rows, n]")
    if routing is not None and routing.sorted_ids.numel() < shape[0]:
        _numel_at_least(routing.sorted_ids, shape[0], f"{who}: routing.sorted_ids")
    return shape


def moe_silu_mul_dropout(gate: torch.Tensor, up: torch.Tensor, routing: Optional[Routing] = None, p: float = 0.0,
                         rng: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out = SiLU(gate) * up, each value dropped with probability ``p`` and the others multiplied by
    1 / (1 - p), on the real sorted rows (all rows, row r as pair r, without ``routing``); bf16 [rows, n].

    ``rng`` (int64 [2] on the device) holds the seed and offset of the counter-based generator: the mask is
    a function of them, the pair and the column, and is never stored.  ``p`` is taken to a multiple of 2^-16.
    ``out`` may be ``gate`` or ``up``."""
    who = "moe_silu_mul_dropout"
    rows, n = _rows(gate, routing, who, "gate")
    p = _check_p(p, rng, who)
    if out is None:
        out = torch.empty_like(gate)
    _shape(up, (rows, n), who, "up")
    _shape(out, (rows, n), who, "out")
    bf = torch.bfloat16
    i = _index(gate, bf, "gate")
    _launch(who, i, gate.data_ptr(), _ptr(up, bf, "up", i), _ptr(out, bf, "out", i),
            _ptr(routing.sorted_ids, torch.int32, "sorted_ids", i) if routing is not None else None,
            routing.num_pairs if routing is not None else rows, rows, n, p, _ptr(rng, torch.int64, "rng", i))
    return out


def moe_silu_mul_backward(gate: torch.Tensor, up: torch.Tensor, d: torch.Tensor, topk_w: torch.Tensor,
                          routing: Optional[Routing] = None, p: float = 0.0, rng: Optional[torch.Tensor] = None,
                          d_gate: Optional[torch.Tensor] = None, d_up: Optional[torch.Tensor] = None,
                          h_weighted: Optional[torch.Tensor] = None, d_topk_w: Optional[torch.Tensor] = None
                          ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Backward of ``moe_silu_mul_dropout`` (same ``p`` and ``rng`` values) for rows that are multiplied by
    their router weight w after the down projection: ``d`` [rows, n] is the gradient of h for w = 1.

    Returns (d_gate, d_up, w * h, d_topk_w): bf16 [rows, n] and fp32 like ``topk_w`` (one weight per pair).
    Each bf16 output may be one of ``gate``, ``up`` and ``d``.  Rows without a pair, and the d_topk_w of
    pairs without a row, are not written (allocated here, those d_topk_w are zero)."""
    who = "moe_silu_mul_backward"
    rows, n = _rows(gate, routing, who, "gate")
    p = _check_p(p, rng, who)
    pairs = routing.num_pairs if routing is not None else rows
    d_gate = torch.empty_like(gate) if d_gate is None else d_gate
    d_up = torch.empty_like(gate) if d_up is None else d_up
    h_weighted = torch.empty_like(gate) if h_weighted is None else h_weighted
    d_topk_w = torch.zeros_like(topk_w) if d_topk_w is None else d_topk_w
    for t, name in ((up, "up"), (d, "d"), (d_gate, "d_gate"), (d_up, "d_up"), (h_weighted, "h_weighted")):
        _shape(t, (rows, n), who, name)
    if topk_w.numel() < pairs or d_topk_w.numel() < pairs:
        _numel_at_least(topk_w, pairs, f"{who}: topk_w")
        _numel_at_least(d_topk_w, pairs, f"{who}: d_topk_w")
    bf, f32 = torch.bfloat16, torch.float32
    i = _index(gate, bf, "gate")
    _launch(who, i, gate.data_ptr(), _ptr(up, bf, "up", i), _ptr(d, bf, "d", i), _ptr(topk_w, f32, "topk_w", i),
            _ptr(routing.sorted_ids, torch.int32, "sorted_ids", i) if routing is not None else None, pairs, rows, n, p,
            _ptr(rng, torch.int64, "rng", i), _ptr(d_gate, bf, "d_gate", i), _ptr(d_up, bf, "d_up", i),
            _ptr(h_weighted, bf, "h_weighted", i), _ptr(d_topk_w, f32, "d_topk_w", i))
    return d_gate, d_up, h_weighted, d_topk_w


def _operand(t: torch.Tensor, width: int, by_token: bool, routing: Routing, who: str, name: str) -> None:
    shape, rows = t.shape, routing.num_pairs // routing.top_k if by_token else routing.max_pad
    if len(shape) != 2 or shape[1] != width:
        raise ValueError(f"{who}: {name} is {tuple(shape)}; its width must be {width}")
    if shape[0] < rows:
        raise ValueError(f"{who}: {name} has {tuple(shape)}; needs >= {rows} rows")


def moe_grouped_gemm_dgrad(dy: torch.Tensor, w: Bf16Weight, routing: Routing, dy1: Optional[torch.Tensor] = None,
                           w1: Optional[Bf16Weight] = None, by_token: bool = False,
                           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                           ) -> torch.Tensor:
    """Gradient of the input of the experts' products y = x W^T: out[r] = dy[r] W_e (+ dy1[r] W1_e) for the
    real sorted rows r of every expert e, bf16 [max_pad, K].

    ``w``, ``w1``: bf16 [E, N, K].  ``dy``, ``dy1``: bf16 [max_pad, N] by sorted row, or with ``by_token``
    [T, N] by token.  ``workspace`` (from ``gemm_workspace``) lets launches of few tiles divide the sum over
    N; calls that share one must not overlap."""
    who = "moe_grouped_gemm_dgrad"
    if not isinstance(w, Bf16Weight) or not (w1 is None or isinstance(w1, Bf16Weight)):
        raise ValueError(f"{who}: gradients go through bf16 weights only")
    E, N, K = w.shape
    if E != routing.num_experts:
        raise ValueError(f"{who}: the weights hold {E} experts, the routing {routing.num_experts}")
    if (dy1 is None) != (w1 is None):
        raise ValueError(f"{who}: dy1 and w1 go together")
    if w1 is not None and tuple(w1.shape) != (E, N, K):
        raise ValueError(f"{who}: the two weights must have one shape")
    _operand(dy, N, by_token, routing, who, "dy")
    if dy1 is not None:
        _operand(dy1, N, by_token, routing, who, "dy1")
    if out is None:
        out = torch.empty((routing.max_pad, K), dtype=torch.bfloat16, device=dy.device)
    if out.dim() != 2 or out.shape[1] != K or out.shape[0] < routing.max_pad:
        raise ValueError(f"{who}: out is {tuple(out.shape)}; needs [>= {routing.max_pad}, {K}]")
    _check_routing(routing)
    bf = torch.bfloat16
    i = _index(dy, bf, "dy")
    _ptr(w.w, bf, "w", i)
    s0, s1 = w.struct(), None
    if w1 is not None:
        _ptr(w1.w, bf, "w1", i)
        s1 = w1.struct()
    _launch(who, i, dy.data_ptr(), ctypes.byref(s0), _ptr(dy1, bf, "dy1", i), ctypes.byref(s1) if s1 is not None else None,
            _ptr(out, bf, "out", i), _ptr(routing.sorted_ids, torch.int32, "sorted_ids", i),
            _ptr(routing.offsets, torch.int32, "offsets", i), routing.num_pairs, routing.top_k, E, N, K,
            routing.block_size, routing.max_pad, int(bool(by_token)), _ptr(workspace, torch.uint8, "workspace", i),
            workspace.numel() if workspace is not None else 0)
    return out


def moe_grouped_gemm_wgrad(dy: torch.Tensor, x: torch.Tensor, routing: Routing, dy_by_token: bool = False,
                           x_by_token: bool = False, base: Optional[torch.Tensor] = None,
                           out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                           ) -> torch.Tensor:
    """Gradient of the experts' weights of y = x W^T: out[e] = base[e] + dy_e^T x_e over the real sorted rows
    of every expert e, [E, N, K]; experts without rows get base, or zeros.

    ``dy`` [.., N] and ``x`` [.., K]: bf16 by sorted row ([max_pad, ..]) or by token ([T, ..]).  ``out``: bf16
    (rounded once, after ``base`` is added) or fp32; allocated like ``base``, else bf16.  ``base`` may be
    ``out``: gradients summed over batches.  ``workspace``: as for ``moe_grouped_gemm_dgrad``, to divide long
    sums over rows."""
    who = "moe_grouped_gemm_wgrad"
    if dy.dim() != 2 or x.dim() != 2:
        raise ValueError(f"{who}: dy is {tuple(dy.shape)}, x {tuple(x.shape)}; need two dimensions")
    E, N, K = routing.num_experts, dy.shape[1], x.shape[1]
    _operand(dy, N, dy_by_token, routing, who, "dy")
    _operand(x, K, x_by_token, routing, who, "x")
    if out is None:
        out = torch.empty((E, N, K), dtype=torch.bfloat16 if base is None else base.dtype, device=dy.device)
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{who}: out must be bfloat16 or float32 (got {out.dtype})")
    _shape(out, (E, N, K), who, "out")
    _shape(base, (E, N, K), who, "base")
    _check_routing(routing)
    bf = torch.bfloat16
    i = _index(dy, bf, "dy")
    _launch(who, i, dy.data_ptr(), _ptr(x, bf, "x", i), _ptr(out, out.dtype, "out", i), _ptr(base, out.dtype, "base", i),
            int(out.dtype is torch.float32), _ptr(routing.sorted_ids, torch.int32, "sorted_ids", i),
            _ptr(routing.offsets, torch.int32, "offsets", i), routing.num_pairs, routing.top_k, E, N, K,
            routing.block_size, routing.max_pad, int(bool(dy_by_token)), int(bool(x_by_token)),
            _ptr(workspace, torch.uint8, "workspace", i), workspace.numel() if workspace is not None else 0)
    return out


def moe_route_backward(topk_ids: torch.Tensor, topk_w: torch.Tensor, d_topk_w: torch.Tensor, num_experts: int,
                       logits: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the router's logits, fp32 [T, num_experts], from the gradient ``d_topk_w`` of the weights that
    ``moe_route`` returned: renormalised over the chosen, or (with its ``logits``) not."""
    who = "moe_route_backward"
    if topk_ids.dim() != 2:
        raise ValueError(f"{who}: topk_ids is {tuple(topk_ids.shape)}; needs [T, k]")
    T, k = topk_ids.shape
    E = int(num_experts)
    _shape(topk_w, (T, k), who, "topk_w")
    _shape(d_topk_w, (T, k), who, "d_topk_w")
    if out is None:
        out = torch.empty((T, E), dtype=torch.float32, device=topk_ids.device)
    _shape(logits, (T, E), who, "logits")
    _shape(out, (T, E), who, "out")
    f32 = torch.float32
    i = _index(topk_ids, torch.int32, "topk_ids")
    _launch(who, i, topk_ids.data_ptr(), _ptr(topk_w, f32, "topk_w", i), _ptr(d_topk_w, f32, "d_topk_w", i),
            _ptr(logits, f32, "logits", i), T, E, k, _ptr(out, f32, "out", i))
    return out
