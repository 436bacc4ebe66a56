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
