"""PyTorch-facing binding of the serving operators (``include/serving/moe_serving.h``): the norm in
front of the layer, block-scaled E4M3 quantisation and grouped products, and the whole layer for a few
tokens.

As in ``ops``: argument checks and marshalling only; every step runs in the HIP library on the
tensors' device and its current stream.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from ._lib import (MOE_OK, MOE_W_BF16, MOE_W_FP8, MOE_W_FP8_BLOCK, MOE_W_INT4_GPTQ, MoeWeight, check, lib)
from .ops import Bf16Weight, Fp8Weight, GptqWeight, Routing, _check_gemm_shapes, _dev, _need, _numel_at_least, _zeroed

__all__ = ["FP8_BLOCK", "FEW_TOKENS", "Fp8BlockWeight", "FewTokensPlan", "moe_rmsnorm", "moe_quantize_fp8_block",
           "moe_grouped_gemm_fp8_block", "few_tokens_supported", "few_tokens_fit", "few_tokens_plan", "moe_few_tokens"]

FP8_BLOCK = 128   # columns under one scale (weights: 128 x 128 blocks)
FEW_TOKENS = 32   # most tokens of moe_few_tokens


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


@dataclass
class Fp8BlockWeight:
    """FP8 E4M3 expert weights with one fp32 scale per 128 x 128 block: codes ``[E, N, K]`` uint8,
    scales ``[E, ceil(N/128), ceil(K/128)]``."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self) -> Tuple[int, int, int]:
        return tuple(self.codes.shape)

    def struct(self) -> MoeWeight:
        E, N, K = self.codes.shape
        _need(tuple(self.scales.shape) == (E, _blocks(N), _blocks(K)),
              f"scales is {tuple(self.scales.shape)}; needs {(E, _blocks(N), _blocks(K))}")
        return MoeWeight(MOE_W_FP8_BLOCK, 0, _dev(self.codes, torch.uint8, "codes"),
                         _dev(self.scales, torch.float32, "scales"), None)


# the current stream's handle by device index: torch.cuda.current_stream builds a Stream object first, which
# takes longer (1.9 us) than the rest of a call's marshalling
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(name: str, index: int, *args) -> None:
    """The call on the current stream of device ``index``, with that device current (a launch goes to
    the current device's code object, whatever device its stream belongs to)."""
    f = getattr(lib(), name)
    if index == torch.cuda.current_device():
        check(f(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(index):
            check(f(*args, _raw_stream(index)))


def _ptr(t: Optional[torch.Tensor], dtype: torch.dtype, name: str, index: int) -> Optional[int]:
    """``t``'s address (None stays None), a contiguous tensor on device ``index``."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _dev(t, dtype, name)
    raise ValueError(f"{name} is on {t.device}, the first argument on device {index}")


def _index(t: torch.Tensor, dtype: torch.dtype, name: str) -> int:
    """The device index of a call's leading tensor, checked."""
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        _dev(t, dtype, name)
    return t.get_device()


def _weight_tensors(w):
    return [t for t in vars(w).values() if isinstance(t, torch.Tensor)]


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
    rows, k = shape = x.shape
    _need(tuple(weight.shape) == (k,), f"{who}: weight is {tuple(weight.shape)}; needs ({k},)")
    if residual is None:
        _need(residual_out is None, f"{who}: residual_out without residual")
    elif residual_out is None:
        residual_out = residual
    _need((q is None) == (scale is None), f"{who}: q and scale go together")
    if y is None and q is None:
        y = torch.empty_like(x)
    for t, name in ((residual, "residual"), (residual_out, "residual_out"), (y, "y"), (q, "q")):
        if t is not None and t.shape != shape:
            raise ValueError(f"{who}: {name} is {tuple(t.shape)}; needs {(rows, k)}")
    block = 0
    if scale is not None:
        block = FP8_BLOCK if scale.dim() == 2 else 0
        want = (rows, _blocks(k)) if block else (rows,)
        _need(tuple(scale.shape) == want, f"{who}: scale is {tuple(scale.shape)}; needs {(rows,)} or {(rows, _blocks(k))}")
    bf = torch.bfloat16
    i = _index(x, bf, "x")
    _launch(who, i, x.data_ptr(), _ptr(residual, bf, "residual", i), _ptr(weight, bf, "weight", i),
            eps, rows, k, _ptr(residual_out, bf, "residual_out", i), _ptr(y, bf, "y", i),
            _ptr(q, torch.uint8, "q", i), _ptr(scale, torch.float32, "scale", i), block)
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
    i = _index(x, torch.bfloat16, "x")
    _launch(who, i, x.data_ptr(), rows, k,
            _ptr(routing.sorted_ids, torch.int32, "sorted_ids", i) if routing is not None else None,
            routing.num_pairs if routing is not None else 0, _ptr(q, torch.uint8, "q", i),
            _ptr(scale, torch.float32, "scale", i))


def moe_grouped_gemm_fp8_block(op: int, a: torch.Tensor, a_scale: torch.Tensor, w0: Fp8BlockWeight,
                               w1: Optional[Fp8BlockWeight], routing: Routing, out: Optional[torch.Tensor] = None,
                               q: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """op = MOE_OP_GATE_UP_SILU (a = x codes [T, K] by token) or MOE_OP_DOWN (a = Hs codes [max_pad, K]),
    a_scale [rows, ceil(K/128)].  Returns ``out`` (bf16 [max_pad, N], allocated without one); with ``q``
    (uint8 [max_pad, N]) and ``scale`` ([max_pad, ceil(N/128)]) the gate/up op writes E4M3 codes for the
    down op instead, and returns None."""
    who = "moe_grouped_gemm_fp8_block"
    E, N, K = w0.shape
    _need((q is None) == (scale is None), f"{who}: q and scale go together")
    _need(q is None or out is None, f"{who}: out and q exclude each other")
    mp = routing.max_pad
    if q is None and out is None:
        out = torch.empty((mp, N), dtype=torch.bfloat16, device=a.device)
    _check_gemm_shapes(op, a, w0, w1, routing, out if q is None else q, who)
    _need(a_scale.dim() == 2 and a_scale.shape[1] == _blocks(K) and a_scale.shape[0] >= a.shape[0],
          f"{who}: a_scale is {tuple(a_scale.shape)}; needs [>= {a.shape[0]}, {_blocks(K)}]")
    if scale is not None:
        _need(scale.dim() == 2 and scale.shape[1] == _blocks(N) and scale.shape[0] >= mp,
              f"{who}: scale is {tuple(scale.shape)}; needs [>= {mp}, {_blocks(N)}]")
    s0 = w0.struct()
    s1 = w1.struct() if w1 is not None else None
    i = _index(a, torch.uint8, "a")
    for w in (w0,) if w1 is None else (w0, w1):
        for t in _weight_tensors(w):
            if t.get_device() != i:
                raise ValueError(f"{who}: a weight is on {t.device}, a on device {i}")
    _launch(who, i, op, a.data_ptr(), _ptr(a_scale, torch.float32, "a_scale", i),
            ctypes.byref(s0), ctypes.byref(s1) if s1 is not None else None, _ptr(out, torch.bfloat16, "out", i),
            _ptr(q, torch.uint8, "q", i), _ptr(scale, torch.float32, "scale", i),
            _ptr(routing.sorted_ids, torch.int32, "sorted_ids", i), _ptr(routing.offsets, torch.int32, "offsets", i),
            routing.num_pairs, routing.top_k, routing.num_experts, N, K, routing.block_size, mp,
            _ptr(workspace, torch.uint8, "workspace", i), workspace.numel() if workspace is not None else 0)
    return out


# ----------------------------------------------------------------------------- the layer for a few tokens
@dataclass
class FewTokensPlan:
    """What ``moe_few_tokens`` keeps between calls: the checked weights and the workspace (calls on one
    plan must not overlap: one plan per stream that runs the layer).

    The weights may be replaced, by ``use`` or by giving a weight object other tensors: a call that finds
    another tensor or address than the checked one checks the weights again."""
    gate: object
    up: object
    down: object
    E: int
    H: int
    I: int
    top_k: int
    max_tokens: int
    renormalize: bool
    workspace: torch.Tensor

    def __post_init__(self):
        self.use(self.gate, self.up, self.down)

    @property
    def device(self) -> torch.device:
        return self.workspace.device

    def use(self, gate, up, down) -> None:
        """Check the weights, of the plan's sizes, and note their addresses; refused ones change nothing."""
        who = "moe_few_tokens"
        ws = (gate, up, down)
        _check_weights(*ws, who)
        _need(tuple(gate.shape) == (self.E, self.I, self.H),
              f"{who}: gate is {tuple(gate.shape)}; the plan was made for {(self.E, self.I, self.H)}")
        why = _unsupported(*ws, self.top_k, self.max_tokens)
        _need(why is None, f"{who}: unsupported: {why}")
        _need(all(t.device == self.device for w in ws for t in _weight_tensors(w)),
              f"{who}: the weights are not on {self.device}")
        structs = tuple(w.struct() for w in ws)
        self.gate, self.up, self.down = ws
        self.tensors = tuple((w, name, t, t.data_ptr()) for w in ws for name, t in vars(w).items()
                             if isinstance(t, torch.Tensor))
        self.structs = structs
        self.refs = tuple(ctypes.byref(w) for w in structs)


def _check_weight(w, who: str) -> None:
    """The scales' shapes (the kernels read them by the matrix sizes)."""
    E, N, K = w.shape
    if isinstance(w, GptqWeight):
        G = int(w.group_size)
        _need(G > 0 and K % G == 0 and N % 8 == 0, f"{who}: K={K} is not a multiple of group_size {G}, or N={N} of 8")
        want = {"scales": (E, K // G, N), "qzeros": (E, K // G, N // 8)}
    elif isinstance(w, Fp8Weight):
        want = {"scales": (E, N)}
    else:
        want = {}
    for name, shape in want.items():
        _need(tuple(getattr(w, name).shape) == shape, f"{who}: {name} is {tuple(getattr(w, name).shape)}; needs {shape}")


def _check_weights(gate, up, down, who: str) -> None:
    E, I, H = gate.shape
    _need(type(gate) is type(up) is type(down), f"{who}: gate, up and down must have one type")
    _need(tuple(up.shape) == (E, I, H) and tuple(down.shape) == (E, H, I),
          f"{who}: gate is {(E, I, H)}, up {tuple(up.shape)}, down {tuple(down.shape)}")
    for w in (gate, up, down):
        _check_weight(w, who)


_KINDS = ((Bf16Weight, MOE_W_BF16), (GptqWeight, MOE_W_INT4_GPTQ), (Fp8Weight, MOE_W_FP8),
          (Fp8BlockWeight, MOE_W_FP8_BLOCK))


def _kind(w) -> int:
    return next((kind for c, kind in _KINDS if isinstance(w, c)), -1)


def _unsupported(gate, up, down, top_k: int, num_tokens: int) -> Optional[str]:
    """Why ``moe_few_tokens`` does not take a layer, from its sizes and types alone (None: it does)."""
    E, I, H = gate.shape
    ws = [MoeWeight(_kind(w), int(getattr(w, "group_size", 0)), None, None, None) for w in (gate, up, down)]
    status = lib().moe_few_tokens_check(*[ctypes.byref(w) for w in ws], num_tokens, E, top_k, H, I)
    return None if status == MOE_OK else lib().moe_last_error().decode()


def few_tokens_supported(gate, up, down, top_k: int, num_tokens: int = FEW_TOKENS) -> bool:
    """Whether ``moe_few_tokens`` takes a layer of these weights' sizes, types and group sizes with up to
    ``num_tokens`` tokens.  The grouped GEMMs take layers that it does not: a down projection of
    another type or group size than gate and up, expert matrices of 2 GiB and more, more than 65536 hidden
    columns or 32 experts per token."""
    return _unsupported(gate, up, down, top_k, num_tokens) is None


def _workspace_bytes(gate, top_k: int, num_tokens: int) -> int:
    E, I, H = gate.shape
    return int(lib().moe_few_tokens_workspace_bytes(num_tokens, E, top_k, H, I, _kind(gate)))


def few_tokens_fit(gate, up, down, top_k: int, num_tokens: int, workspace: torch.Tensor) -> bool:
    """Whether ``moe_few_tokens`` takes a layer of these weights with up to ``num_tokens`` tokens on another
    layer's workspace (the weight types divide it differently)."""
    return (few_tokens_supported(gate, up, down, top_k, num_tokens)
            and _workspace_bytes(gate, top_k, num_tokens) <= workspace.numel())


def few_tokens_plan(gate, up, down, top_k: int, max_tokens: int = FEW_TOKENS,
                    renormalize: bool = True, wait: bool = True) -> FewTokensPlan:
    """Check the expert weights of a layer (gate and up ``[E, I, H]``, down ``[E, H, I]``; all bf16, GPTQ
    int4, fp8 with channel scales or fp8 with block scales) once and make the workspace for calls of up
    to ``max_tokens`` tokens.  The workspace is filled when this returns, so that any stream may make the first
    call; without ``wait``, the current one."""
    who = "few_tokens_plan"
    E, I, H = gate.shape
    _need(0 <= max_tokens <= FEW_TOKENS, f"{who}: max_tokens {max_tokens} not in [0, {FEW_TOKENS}]")
    _check_weights(gate, up, down, who)
    why = _unsupported(gate, up, down, top_k, max_tokens)
    _need(why is None, f"{who}: unsupported: {why}")
    for w in (gate, up, down):
        w.struct()                     # types and devices, before the workspace is made
    device = _weight_tensors(gate)[0].device
    _need(all(t.device == device for w in (gate, up, down) for t in _weight_tensors(w)),
          f"{who}: the weights are on more than one device")
    n = _workspace_bytes(gate, top_k, max_tokens)
    return FewTokensPlan(gate, up, down, E, H, I, top_k, max_tokens, bool(renormalize),
                         _zeroed(n, device, wait))


def moe_few_tokens(plan: FewTokensPlan, logits: torch.Tensor, x: torch.Tensor,
                   topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The whole routed layer for ``x`` [T, H] bf16 and router ``logits`` [T, E] fp32, T <= the plan's
    ``max_tokens``, in two launches.  Returns (out [T, H] bf16, topk_ids [T, k] int32, topk_w [T, k]
    fp32).  Activations stay bf16 whatever the weights' type."""
    who = "moe_few_tokens"
    if x.dim() != 2 or x.shape[1] != plan.H:
        raise ValueError(f"{who}: x is {tuple(x.shape)}; its width must be {plan.H}")
    for w, name, t, address in plan.tensors:
        if getattr(w, name) is not t or t.data_ptr() != address:
            plan.use(plan.gate, plan.up, plan.down)
            break
    T, k = x.shape[0], plan.top_k
    if T > plan.max_tokens:
        raise ValueError(f"{who}: {T} tokens; the plan holds {plan.max_tokens}")
    if tuple(logits.shape) != (T, plan.E):
        raise ValueError(f"{who}: logits is {tuple(logits.shape)}; needs {(T, plan.E)}")
    i = _index(x, torch.bfloat16, "x")
    if i != plan.workspace.get_device():
        raise ValueError(f"{who}: x is on {x.device}, the plan on {plan.device}")
    if out is None:
        out = torch.empty_like(x)
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    if out.shape != x.shape:
        raise ValueError(f"{who}: out is {tuple(out.shape)}; needs {tuple(x.shape)}")
    if topk_ids.numel() < T * k or topk_w.numel() < T * k:
        raise ValueError(f"{who}: topk_ids and topk_w hold {topk_ids.numel()} and {topk_w.numel()}; need {T * k}")
    g, u, d = plan.refs
    _launch(who, i, _ptr(logits, torch.float32, "logits", i), x.data_ptr(), g, u, d, T, plan.E, k, plan.H, plan.I,
            plan.renormalize, _ptr(topk_ids, torch.int32, "topk_ids", i), _ptr(topk_w, torch.float32, "topk_w", i),
            _ptr(out, torch.bfloat16, "out", i), plan.workspace.data_ptr(), plan.workspace.numel())
    return out, topk_ids, topk_w
