"""Results of the training operators over their operands, CPU side: refused by the C ABI where a workgroup could read what
another one has written, before anything is enqueued.  The addresses are made up: no call gets past its checks."""
import ctypes
import os
import re

import pytest

from mixture_experts_routed_route_amd._lib import MoeWeight


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routed_route_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_routed_route_amd.build import build
        build()
    return _lib.lib()


def weight(at):
    return ctypes.byref(MoeWeight(0, 0, at, None, None))


def refused(L, call, what):
    rc = getattr(L, call[0])(*call[1])
    assert rc == -1 and re.search(what, L.moe_last_error().decode()), L.moe_last_error()


MB = 1 << 20
P, TOP, E, N, K, BS = 16, 2, 4, 64, 128, 16   # 8 tokens
MP = 2 * 8 + 4 * 16                            # padded rows


def dgrad(dx, dy0=MB, w0=2 * MB, dy1=None, w1=None, by_token=0):
    return "moe_grouped_gemm_dgrad", (dy0, weight(w0), dy1, weight(w1) if w1 else None, dx, 8 * MB, 9 * MB, P, TOP, E, N, K, BS,
                                      MP, by_token, None, 0, None)


def wgrad(dw, dy=MB, x=2 * MB, base=None, f32=0, dy_tok=0, x_tok=0):
    return "moe_grouped_gemm_wgrad", (dy, x, dw, base, f32, 8 * MB, 9 * MB, P, TOP, E, N, K, BS, MP, dy_tok, x_tok, None, 0, None)


DX, DY, W = MP * K * 2, MP * N * 2, E * N * K * 2


@pytest.mark.parametrize("call", [
    dgrad(2 * MB), dgrad(5 * MB, dy1=4 * MB, w1=5 * MB),                               # the weights themselves
    dgrad(2 * MB + W - 16), dgrad(2 * MB - DX + 16), dgrad(5 * MB + 4096, dy1=4 * MB, w1=5 * MB),   # a part of them
    dgrad(MB + DY - 16), dgrad(MB - DX + 16), dgrad(4 * MB + 16, dy1=4 * MB, w1=5 * MB),            # a part of dy
    dgrad(MB + P // TOP * N * 2 - 16, by_token=1)])
def test_dgrad(L, call):
    refused(L, call, "dx is one buffer with an operand")


@pytest.mark.parametrize("call", [
    wgrad(MB + DY - 16), wgrad(MB - W + 16), wgrad(MB - 2 * W + 16, f32=1), wgrad(2 * MB + DX - 16), wgrad(2 * MB - W + 16),
    wgrad(MB + P // TOP * N * 2 - 16, dy_tok=1), wgrad(2 * MB + P // TOP * K * 2 - 16, x_tok=1)])
def test_wgrad(L, call):
    refused(L, call, "dw is one buffer with an operand")


@pytest.mark.parametrize("call", [wgrad(4 * MB, base=4 * MB + W - 16), wgrad(4 * MB, base=4 * MB - 16),
                                  wgrad(4 * MB, base=4 * MB + 2 * W - 16, f32=1)])
def test_base(L, call):
    """base may be dw: each value is read by the thread that writes it.  Shifted, another tile writes it first."""
    refused(L, call, "base lies over a part of dw")


# ------------------------------------------------------------------ row kernels
ROWS, COLS = 40, 64
SIZE, PAIRS = ROWS * COLS * 2, ROWS * 4


def drop(out, gate=MB, up=2 * MB):
    return "moe_silu_mul_dropout", (gate, up, out, None, ROWS, ROWS, COLS, 0.0, None, None)


def back(dg=11 * MB, du=12 * MB, hw=13 * MB, dw=14 * MB, gate=MB, up=2 * MB, d=3 * MB, w=4 * MB):
    return "moe_silu_mul_backward", (gate, up, d, w, None, ROWS, ROWS, COLS, 0.0, None, dg, du, hw, dw, None)


@pytest.mark.parametrize("call", [drop(MB + 16), drop(MB - 16), drop(2 * MB + SIZE - 16), drop(2 * MB, gate=2 * MB + 128)])
def test_shifted_result(L, call):
    """out may be gate or up: a thread loads what it replaces.  Shifted by a row or a chunk, another thread replaces it."""
    refused(L, call, "out lies over a part of an input")


@pytest.mark.parametrize("call", [back(dg=MB + 16), back(du=2 * MB - 128), back(hw=3 * MB + SIZE - 16), back(dg=3 * MB - SIZE + 16)])
def test_shifted_gradients(L, call):
    refused(L, call, "an output lies over a part of an input")


@pytest.mark.parametrize("call", [back(dg=12 * MB + 16), back(du=13 * MB - 16), back(hw=11 * MB + SIZE - 16)])
def test_gradients_over_each_other(L, call):
    refused(L, call, "two outputs are one buffer")


@pytest.mark.parametrize("call", [back(dg=4 * MB), back(hw=4 * MB + PAIRS - 16), back(du=14 * MB - SIZE + 16), back(dw=MB),
                                  back(dw=3 * MB + SIZE - 16)])
def test_gradients_over_weights_of_rows(L, call):
    refused(L, call, "topk_w")


def rback(out, ids=MB, w=2 * MB, dw=3 * MB, logits=None, T=40, experts=8, k=2):
    return "moe_route_backward", (ids, w, dw, logits, T, experts, k, out, None)


@pytest.mark.parametrize("call,what", [
    (rback(MB), "topk_ids"), (rback(2 * MB), "topk_w"), (rback(3 * MB), "d_topk_w"), (rback(3 * MB - 40 * 8 * 4 + 16), "d_topk_w"),
    (rback(2 * MB + 40 * 2 * 4 - 16), "topk_w"), (rback(3 * MB + 16, k=8), "d_topk_w"),
    (rback(4 * MB + 32, logits=4 * MB), "a part of logits"), (rback(4 * MB - 16, logits=4 * MB), "a part of logits")])
def test_route_backward(L, call, what):
    """A token's row of d_logits over other tokens' operands, which their waves may not have read."""
    refused(L, call, what)
