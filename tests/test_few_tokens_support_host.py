"""Which layers the two-launch form takes, CPU side: one test behind the call, the query, the plan and the
layer, which runs its stages where the form does not take it."""
import ctypes

import pytest
import torch

import mixture_experts_routed_route_amd as m
from mixture_experts_routed_route_amd._lib import MoeWeight, lib

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below is refused or has no tokens
TYPES = {"bf16": 0, "int4": 1, "fp8": 2, "fp8_block": 3}


def check(kind, H, I, E=8, k=2, T=8, groups=(128, 128, 128)):
    ws = [MoeWeight(TYPES[kind], g if kind == "int4" else 0, None, None, None) for g in groups]
    rc = lib().moe_few_tokens_check(*[ctypes.byref(w) for w in ws], T, E, k, H, I)
    return rc, lib().moe_last_error().decode()


def call(kind, H, I, E=8, k=2, T=8, groups=(128, 128, 128)):
    ws = [MoeWeight(TYPES[kind], g if kind == "int4" else 0, FAKE, FAKE, FAKE) for g in groups]
    rc = lib().moe_few_tokens(FAKE, FAKE, *[ctypes.byref(w) for w in ws], T, E, k, H, I, 1, FAKE, FAKE, FAKE, FAKE, 0, None)
    return rc, lib().moe_last_error().decode()


# arguments, status, word of the message.  The grouped GEMMs take all but the first three (of which they
# refuse the widths, or the group size of gate and up)
NOT_TAKEN = [
    (dict(kind="int4", H=2080, I=96, groups=(32,) * 3), -1, "hidden 2080"),
    (dict(kind="int4", H=2048, I=96, groups=(32,) * 3), -1, "inter 96"),
    (dict(kind="int4", H=256, I=128, groups=(64, 128, 64)), -1, "group sizes"),
    (dict(kind="int4", H=256, I=128, groups=(64, 64, 128)), -1, "group sizes"),
    (dict(kind="bf16", H=32768, I=32768), -2, "2 GiB"),
    (dict(kind="bf16", H=65544, I=64), -2, "65536"),
    (dict(kind="bf16", H=256, I=128, E=64, k=33), -2, "top_k=33"),
]


@pytest.mark.parametrize("kw,code,word", NOT_TAKEN)
def test_check_and_call_refuse_alike(kw, code, word):
    for f in (check, call):
        rc, msg = f(**kw)
        assert rc == code and word in msg, (f.__name__, rc, msg)


def test_check_takes_what_the_call_takes():
    """The call gets as far as its workspace (of no bytes) exactly where the query says MOE_OK."""
    widths = (8, 12, 16, 24, 32, 64, 96, 128, 192, 256, 65536, 65544)
    for kind in TYPES:
        for group in ((32, 48, 64, 128, 256) if kind == "int4" else (0,)):
            for H in widths:
                for I in widths:
                    a = dict(kind=kind, H=H, I=I, groups=(group,) * 3)
                    rc, msg = check(**a)
                    got, text = call(**a)
                    assert (rc == 0) == ("workspace_bytes" in text) and (rc == 0 or (got, text) == (rc, msg)), (a, msg, text)


@pytest.mark.parametrize("T,E,k,H,I,t", [(1, 8, 2, 12, 64, 0), (1, 8, 2, 65536, 65536, 0), (1, 8, 2, 2080, 96, 1),
                                        (1, 8, 2, 264, 64, 2), (1, 8, 2, 64, 24, 3), (32, 64, 32, 64, 1 << 20, 3)])
def test_workspace_size_of_unsupported_layers(T, E, k, H, I, t):
    assert lib().moe_few_tokens_workspace_bytes(T, E, k, H, I, t) == -1


def weights(kind, H, I, E=8, groups=(128, 128, 128)):
    def one(n, k, g):
        meta = dict(device="meta")
        if kind == "bf16":
            return m.Bf16Weight(torch.empty((E, n, k), dtype=torch.bfloat16, **meta))
        return m.GptqWeight(torch.empty((E, k // 8, n), dtype=torch.int32, **meta),
                            torch.empty((E, k // g, n), dtype=torch.float16, **meta),
                            torch.empty((E, k // g, n // 8), dtype=torch.int32, **meta), g)
    return one(I, H, groups[0]), one(I, H, groups[1]), one(H, I, groups[2])


@pytest.mark.parametrize("kw", [kw for kw, _, _ in NOT_TAKEN], ids=lambda kw: "-".join(f"{v}" for v in kw.values()))
def test_layer_runs_its_stages_where_the_form_does_not_take_it(kw):
    kw = dict(kw)
    k = kw.pop("k", 2)
    w = weights(**kw)
    assert not m.few_tokens_supported(*w, k)
    layer = m.MoeLayer(kw.get("E", 8), kw["H"], kw["I"], k, 16, *w, few_tokens=True)
    for T in (1, 32):
        assert layer.plan(T, "meta").few is None
    with pytest.raises(ValueError, match="unsupported"):
        m.few_tokens_plan(*w, k)


def test_layer_of_two_weight_types_runs_its_stages():
    gate, up, _ = weights("bf16", 256, 128)
    down = weights("int4", 256, 128)[2]
    assert not m.few_tokens_supported(gate, up, down, 2)
    assert m.MoeLayer(8, 256, 128, 2, 16, gate, up, down, few_tokens=True).plan(4, "meta").few is None


def test_layer_takes_the_form_where_it_is_supported():
    w = weights("bf16", 256, 128)
    assert m.few_tokens_supported(*w, 2) and m.few_tokens_supported(*w, 2, 1)
    layer = m.MoeLayer(8, 256, 128, 2, 16, *w, few_tokens=True)
    assert layer.plan(33, "meta").few is None
    with pytest.raises(ValueError, match="HIP device"):     # it goes on to the plan, whose weights are not on a GPU
        layer.plan(32, "meta")
