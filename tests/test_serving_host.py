"""Serving operators, CPU side: the library exports what serving/moe_serving.h declares, the C ABI and
the binding refuse invalid calls before anything is enqueued, and the oracle's functions are pinned
to closed forms and to torch."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mixture_experts_routed_route_amd as m
import oracle
from _util import ROOT
from moe_synth import f32_to_bf16_bits

HEADER = os.path.join(ROOT, "include", "serving", "moe_serving.h")


@pytest.fixture(scope="module")
def L():
    from mixture_experts_routed_route_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from mixture_experts_routed_route_amd.build import build
        build()
    return _lib.lib()


def test_exports_every_declared_symbol(L):
    from mixture_experts_routed_route_amd import _lib
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^(?:moe_status|int64_t|int32_t)\s+(moe_\w+)\s*\(", src, flags=re.M))
    assert names == set(_lib.SERVING_SIGNATURES)
    for n in names:
        assert hasattr(L, n), f"{n} not exported"


def _rc(L, name, *args):
    rc = getattr(L, name)(*args)
    return rc, L.moe_last_error().decode()


FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation or has no rows
OFF = ctypes.c_void_p((1 << 20) + 8)


# moe_rmsnorm(x, residual, weight, eps, rows, k, residual_out, y, q, scale, scale_block, stream)
RMSNORM_BAD = [
    ((FAKE, None, FAKE, 1e-6, 4, 20, None, FAKE, None, None, 0, None), "k 20"),
    ((FAKE, None, FAKE, 1e-6, 4, 0, None, FAKE, None, None, 0, None), "k 0"),
    ((FAKE, None, FAKE, 1e-6, 4, (1 << 20) + 8, None, FAKE, None, None, 0, None), "2^20"),
    ((FAKE, None, FAKE, 1e-6, 4, 24, None, None, FAKE, FAKE, 0, None), "multiple of 16"),
    ((FAKE, None, FAKE, 1e-6, -1, 64, None, FAKE, None, None, 0, None), "negative"),
    ((FAKE, None, FAKE, -1.0, 4, 64, None, FAKE, None, None, 0, None), "eps"),
    ((FAKE, None, FAKE, float("nan"), 4, 64, None, FAKE, None, None, 0, None), "eps"),
    ((FAKE, None, FAKE, 1e-6, 4, 64, None, None, None, None, 0, None), "one of y_out and q"),
    ((FAKE, FAKE, FAKE, 1e-6, 4, 64, None, FAKE, None, None, 0, None), "go together"),
    ((FAKE, None, FAKE, 1e-6, 4, 64, FAKE, FAKE, None, None, 0, None), "go together"),
    ((FAKE, FAKE, FAKE, 1e-6, 4, 64, FAKE, FAKE, None, None, 0, None), "one buffer"),
    ((FAKE, None, FAKE, 1e-6, 4, 64, None, None, FAKE, None, 0, None), "go together"),
    ((FAKE, None, FAKE, 1e-6, 4, 64, None, None, FAKE, FAKE, 64, None), "scale_block"),
    ((None, None, FAKE, 1e-6, 4, 64, None, FAKE, None, None, 0, None), "x is NULL"),
    ((OFF, None, FAKE, 1e-6, 4, 64, None, FAKE, None, None, 0, None), "aligned"),
    ((FAKE, None, None, 1e-6, 4, 64, None, FAKE, None, None, 0, None), "weight is NULL"),
]


@pytest.mark.parametrize("args,word", RMSNORM_BAD, ids=[str(i) for i in range(len(RMSNORM_BAD))])
def test_rmsnorm_refusals(L, args, word):
    rc, msg = _rc(L, "moe_rmsnorm", *args)
    assert rc == -1 and word in msg, msg


def test_rmsnorm_and_quantize_without_rows_enqueue_nothing(L):
    assert L.moe_rmsnorm(None, None, None, 1e-6, 0, 64, None, FAKE, None, None, 0, None) == 0
    assert L.moe_quantize_fp8_block(None, 0, 64, None, 0, None, None, None) == 0


def test_quantize_block_refusals(L):
    for args, word in [((FAKE, 4, 24, None, 0, FAKE, FAKE, None), "multiple of 16"),
                       ((FAKE, -1, 32, None, 0, FAKE, FAKE, None), "negative"),
                       ((FAKE, 4, 32, None, -1, FAKE, FAKE, None), "num_pairs"),
                       ((None, 4, 32, None, 0, FAKE, FAKE, None), "x is NULL"),
                       ((FAKE, 4, 32, OFF, 8, FAKE, FAKE, None), "aligned"),
                       ((FAKE, 4, 32, None, 0, FAKE, None, None), "scale is NULL")]:
        rc, msg = _rc(L, "moe_quantize_fp8_block", *args)
        assert rc == -1 and word in msg, msg


# ------------------------------------------------------------------------------------- the binding
def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_rmsnorm_binding_refuses_mismatched_buffers():
    x, w = bf(4, 256), bf(256)
    for kw, word in [(dict(weight=bf(128)), "weight"), (dict(residual=bf(4, 128)), "residual is"),
                     (dict(residual_out=bf(4, 256)), "without residual"), (dict(y=bf(3, 256)), "y is"),
                     (dict(q=u8(4, 256)), "go together"), (dict(q=u8(4, 255), scale=torch.zeros(4)), "q is"),
                     (dict(q=u8(4, 256), scale=torch.zeros(3)), "scale is"),
                     (dict(q=u8(4, 256), scale=torch.zeros(4, 3)), "scale is"),
                     (dict(q=u8(4, 256), scale=torch.zeros(4, 1)), "scale is")]:
        args = {"weight": w, **kw}
        with pytest.raises(ValueError, match=word):
            m.moe_rmsnorm(x, args.pop("weight"), 1e-6, **args)
    with pytest.raises(ValueError, match="rows, k"):
        m.moe_rmsnorm(bf(256), w)
    with pytest.raises(ValueError, match="HIP device"):
        m.moe_rmsnorm(x, w)


def test_quantize_block_binding_refuses_mismatched_buffers():
    for q, s, word in [(u8(4, 128), torch.zeros(4, 2), "q is"), (u8(4, 256), torch.zeros(4), "scale is"),
                       (u8(4, 256), torch.zeros(4, 3), "scale is")]:
        with pytest.raises(ValueError, match=word):
            m.moe_quantize_fp8_block(bf(4, 256), q, s)
    r = m.Routing.allocate(4, 2, 2, 16, "cpu")
    rows = r.max_pad + 16
    with pytest.raises(ValueError, match="sorted_ids"):
        m.moe_quantize_fp8_block(bf(rows, 128), u8(rows, 128), torch.zeros(rows, 1), r)


# -------------------------------------------------------------------------------------- the oracle
def test_oracle_rmsnorm_closed_form():
    """A row of one value v has mean square v^2: y = w * sign(v) without eps; x + residual rounds to
    bf16 before the norm (256 + 1 is halfway between bf16 values 256 and 258: ties to even, 256)."""
    x = f32_to_bf16_bits(np.array([[2.0] * 8, [-3.0] * 8, [256.0] * 8], np.float32))
    r = f32_to_bf16_bits(np.array([[0.0] * 8, [0.0] * 8, [1.0] * 8], np.float32))
    w = f32_to_bf16_bits(np.arange(1, 9, dtype=np.float32))
    h, y = oracle.rmsnorm(x, w, 0.0, r)
    assert (h[2] == 256.0).all()
    np.testing.assert_allclose(y, np.array([1.0, -1.0, 1.0])[:, None] * np.arange(1, 9), rtol=1e-15)
    _, y = oracle.rmsnorm(np.zeros((1, 8), np.uint16), w, 1e-6)
    assert (y == 0).all()


def test_oracle_block_quantisation_matches_torch():
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((7, 272)).astype(np.float32)).bfloat16().float()
    x[3, 128:256] = 0
    q, s = oracle.quantize_blocks_fp8(x.numpy())
    assert s.shape == (7, 3) and (s[3, 1] == 1) and (q[3, 128:256] == 0).all()
    for r in range(7):
        for b in range(3):
            part = x[r, 128 * b: 128 * b + 128]
            amax = part.abs().max()
            f = torch.tensor(448.0) / amax if amax > 0 else torch.tensor(1.0)
            want = (part * f).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            assert np.array_equal(want, q[r, 128 * b: 128 * b + 128])
            if amax > 0:
                assert s[r, b] == (amax / 448.0).item()


def test_oracle_block_quantisation_floor():
    x = np.zeros((1, 128), np.float32)
    x[0, 0] = 2.0 ** -120
    q, s = oracle.quantize_blocks_fp8(x)
    assert s[0, 0] == np.float32(2.0 ** -100) / np.float32(448) and not (q & 0x7F).any()


# ------------------------------------------------------------------------ the layer for a few tokens
def mw(type_=0, group=0, data=FAKE, scales=FAKE, qzeros=FAKE):
    from mixture_experts_routed_route_amd._lib import MoeWeight
    return MoeWeight(type_, group, data, scales, qzeros)


def few(L, g=None, u=None, d=None, T=4, E=8, k=2, H=256, I=128, logits=FAKE, x=FAKE, ids=FAKE, w=FAKE, out=FAKE,
        ws=FAKE, nbytes=1 << 40):
    g, u, d = g or mw(), u or mw(), d or mw()
    return _rc(L, "moe_few_tokens", logits, x, ctypes.byref(g), ctypes.byref(u), ctypes.byref(d), T, E, k, H, I, 1,
               ids, w, out, ws, nbytes, None)


def test_few_tokens_refusals(L):
    assert few(L, T=0)[0] == 0      # nothing to do, nothing enqueued
    for kw, code, word in [
            (dict(T=-1), -1, "num_tokens"), (dict(T=33), -2, "33"), (dict(E=0), -1, "num_experts"),
            (dict(E=257, k=2), -2, "256"), (dict(k=0), -1, "top_k"), (dict(k=9), -1, "top_k"), (dict(E=64, k=33), -2, "32"),
            (dict(H=252), -1, "hidden"), (dict(I=4), -1, "inter"), (dict(H=65544), -2, "65536"),
            (dict(H=32768, I=32768), -2, "2 GiB"), (dict(g=mw(1, 128)), -1, "different types"),
            (dict(g=mw(9), u=mw(9), d=mw(9)), -1, "type 9"),
            (dict(g=mw(1, 48), u=mw(1, 48), d=mw(1, 48)), -1, "group_size 48"),
            (dict(g=mw(1, 64), u=mw(1, 128), d=mw(1, 64)), -1, "group sizes"),
            (dict(g=mw(1, 256), u=mw(1, 256), d=mw(1, 256), I=128), -1, "inter"),
            (dict(g=mw(2), u=mw(2), d=mw(2), H=264), -1, "hidden"),
            (dict(nbytes=100), -1, "workspace_bytes"), (dict(ws=None), -1, "workspace is NULL"), (dict(ws=OFF), -1, "aligned"),
            (dict(x=None), -1, "x is NULL"), (dict(logits=OFF), -1, "aligned"), (dict(out=None), -1, "out is NULL"),
            (dict(ids=None), -1, "topk_ids"), (dict(w=OFF), -1, "topk_w"), (dict(d=mw(data=None)), -1, "data is NULL"),
            (dict(g=mw(3, scales=None), u=mw(3), d=mw(3)), -1, "scales is NULL"),
            (dict(g=mw(1, 64, qzeros=None), u=mw(1, 64), d=mw(1, 64)), -1, "qzeros is NULL")]:
        rc, msg = few(L, **kw)
        assert rc == code and word in msg, (kw, rc, msg)


def test_few_tokens_workspace_size_covers_fewer_tokens(L):
    f = L.moe_few_tokens_workspace_bytes
    for E, k, H, I, t in [(64, 6, 2048, 1408, 1), (8, 2, 4096, 14336, 0), (256, 8, 8, 8, 0), (4, 4, 65536, 64, 3)]:
        sizes = [f(T, E, k, H, I, t) for T in range(33)]
        assert sizes[0] > 0 and all(a <= b for a, b in zip(sizes, sizes[1:]))
        assert sizes[32] >= 32 * k * I * 2
    for bad in [(33, 8, 2, 64, 64, 0), (1, 257, 2, 64, 64, 0), (1, 8, 9, 64, 64, 0), (1, 8, 2, 65544, 64, 0),
                (1, 8, 2, 64, 64, 4), (-1, 8, 2, 64, 64, 0)]:
        assert f(*bad) == -1


def test_few_tokens_plan_refuses_mismatched_weights(L):
    def w(*s):
        return m.Bf16Weight(bf(*s))

    def f8(n, k, scales):
        return m.Fp8BlockWeight(u8(4, n, k), torch.zeros(scales))
    for args, word in [((w(4, 32, 64), w(4, 32, 64), w(4, 64, 40)), "down"),
                       ((w(4, 32, 64), w(4, 40, 64), w(4, 64, 32)), "up"),
                       ((w(4, 32, 64), f8(32, 64, (4, 1, 1)), w(4, 64, 32)), "one type"),
                       ((f8(32, 64, (4, 1, 2)),) * 2 + (f8(64, 32, (4, 1, 1)),), "scales"),
                       ((m.Fp8Weight(u8(4, 32, 64), torch.zeros(4, 31)),) * 2 + (m.Fp8Weight(u8(4, 64, 32), torch.zeros(4, 64)),), "scales")]:
        with pytest.raises(ValueError, match=word):
            m.few_tokens_plan(*args, 2)
    q = m.GptqWeight(torch.zeros(4, 16, 64, dtype=torch.int32), torch.zeros(4, 2, 64, dtype=torch.float16),
                     torch.zeros(4, 2, 7, dtype=torch.int32), 64)
    with pytest.raises(ValueError, match="qzeros"):
        m.few_tokens_plan(q, q, m.GptqWeight(torch.zeros(4, 8, 128, dtype=torch.int32), torch.zeros(4, 1, 128, dtype=torch.float16),
                                             torch.zeros(4, 1, 16, dtype=torch.int32), 64), 2)
    with pytest.raises(ValueError, match="max_tokens"):
        m.few_tokens_plan(w(4, 32, 64), w(4, 32, 64), w(4, 64, 32), 2, 33)


def test_oracle_few_tokens_matches_dense_layer():
    """Against oracle.moe_layer (which sorts and combines) on the same inputs, and block scales of one
    against unscaled codes."""
    from moe_synth import MoeConfig, make_inputs
    cfg = MoeConfig("t", T=6, H=64, I=40, E=5, top_k=2, block_size=16, seed=4)
    d = make_inputs(cfg)
    out, ids, w, spread, _ = oracle.few_tokens(d["logits"], d["x"], *[lambda e, k=k: oracle.expert_matrix(d[k], e) for k in ("wg", "wu", "wd")], 2)
    ref = oracle.moe_layer(d)
    assert np.array_equal(ids, ref["ids"]) and np.array_equal(w, ref["w"])
    np.testing.assert_allclose(out, ref["out"], rtol=1e-11, atol=1e-13)
    assert (spread >= np.abs(out) * (1 - 1e-12)).all()
    codes = np.arange(256, dtype=np.uint8).reshape(1, 1, 256) & 0x77
    one = {"codes": codes, "scales": np.array([[[1.0, 2.0]]], np.float32)}
    v = oracle.e4m3_to_f64(codes[0])
    assert np.array_equal(oracle.fp8_block_matrix(one, 0), np.concatenate([v[:, :128], 2 * v[:, 128:]], axis=1))


# ----------------------------------------------------------------- grouped products with block scales
def gemm(L, op=0, a=FAKE, sa=FAKE, w0=None, w1="same", c=FAKE, q=None, qs=None, ids=FAKE, off=FAKE, P=16, k_=2, E=4, n=128,
         k=256, bs=16, mp=None, ws=None, wsb=0):
    w0 = mw(3) if w0 is None else w0
    w1 = w0 if w1 == "same" else w1
    mp = -(-(P + E * (bs - 1)) // bs) * bs if mp is None else mp
    return _rc(L, "moe_grouped_gemm_fp8_block", op, a, sa, ctypes.byref(w0), ctypes.byref(w1) if w1 is not None else None,
               c, q, qs, ids, off, P, k_, E, n, k, bs, mp, ws, wsb, None)


def test_gemm_fp8_block_refusals(L):
    assert gemm(L, P=0, c=FAKE)[0] == 0   # no pairs: nothing enqueued
    for kw, code, word in [
            (dict(op=2), -1, "op 2"), (dict(c=None), -1, "exactly one"), (dict(q=FAKE, qs=FAKE), -1, "exactly one"),
            (dict(c=None, q=FAKE), -1, "go together"), (dict(qs=FAKE), -1, "go together"),
            (dict(op=1, w1=None, c=None, q=FAKE, qs=FAKE), -1, "GATE_UP_SILU"), (dict(op=1), -1, "no w1"), (dict(w1=None), -1, "needs w1"),
            (dict(n=12), -1, "multiple of 8"), (dict(n=136, c=None, q=FAKE, qs=FAKE), -1, "multiple of 16"),
            (dict(k=40), -1, "multiple of 16"), (dict(w0=mw(2)), -1, "MOE_W_FP8_BLOCK"), (dict(w1=mw(2)), -1, "MOE_W_FP8_BLOCK"),
            (dict(E=257), -2, "256"), (dict(bs=48), -1, "block_size"), (dict(mp=16), -1, "max_pad"), (dict(P=15), -1, "multiple of top_k"),
            (dict(n=65536, k=65536 + 16), -2, "4 GiB"), (dict(op=1, w1=None, P=2**26, k=128, n=8), -2, "4 GiB"),
            (dict(ws=FAKE, wsb=8), -1, "workspace_bytes"), (dict(a=None), -1, "a is NULL"), (dict(sa=OFF), -1, "aligned"),
            (dict(c=None, q=FAKE, qs=OFF), -1, "aligned"), (dict(ids=None), -1, "sorted_ids"), (dict(off=None), -1, "expert_offsets"),
            (dict(w0=mw(3, scales=None)), -1, "scales is NULL")]:
        rc, msg = gemm(L, **kw)
        assert rc == code and word in msg, (kw, rc, msg)


def test_gemm_fp8_block_binding_refuses_mismatched_buffers():
    r = m.Routing.allocate(16, 2, 4, 16, "cpu")
    w = m.Fp8BlockWeight(u8(4, 144, 272), torch.zeros(4, 2, 3))
    sa = torch.zeros(8, 3)
    for kw, word in [(dict(a_scale=torch.zeros(8, 2)), "a_scale"), (dict(a_scale=torch.zeros(7, 3)), "a_scale"),
                     (dict(a=u8(7, 272)), "rows"), (dict(a=u8(8, 256)), "width must be K"),
                     (dict(out=bf(r.max_pad - 1, 144)), "out is"), (dict(q=u8(r.max_pad, 144)), "go together"),
                     (dict(q=u8(r.max_pad, 144), scale=torch.zeros(r.max_pad, 1)), "scale is"),
                     (dict(q=u8(r.max_pad, 128), scale=torch.zeros(r.max_pad, 2)), "out is"),
                     (dict(q=u8(r.max_pad, 144), scale=torch.zeros(r.max_pad, 2), out=bf(r.max_pad, 144)), "exclude"),
                     (dict(w0=m.Fp8BlockWeight(u8(4, 144, 272), torch.zeros(4, 2, 2)), a_scale=sa), "scales is")]:
        args = dict(op=0, a=u8(8, 272), a_scale=sa, w0=w, w1=w, routing=r)
        args.update(kw)
        if "w0" in kw:
            args["w1"] = args["w0"]
        with pytest.raises(ValueError, match=word):
            m.moe_grouped_gemm_fp8_block(**args)


def test_layer_refuses_combinations_it_has_no_path_for():
    w8 = m.Fp8BlockWeight(u8(4, 128, 128), torch.zeros(4, 1, 1))
    wb = m.Bf16Weight(bf(4, 128, 128))
    tabs = m.LoraTables(torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int64), torch.zeros(4), 4, 128, 128, 32)

    def layer(w, **kw):
        return m.MoeLayer(4, 128, 128, 2, 16, w, w, w, **kw)
    for w, kw, word in [(wb, dict(lora=tabs, few_tokens=True), "few_tokens"), (wb, dict(lora_up=tabs, few_tokens=True), "few_tokens"),
                        (w8, dict(lora_gate=tabs), "fp8"), (wb, dict(hs_codes=True), "hs_codes"),
                        (w8, dict(hs_codes=True, lora=tabs), "hs_codes")]:
        with pytest.raises(ValueError, match=word):
            layer(w, **kw)
    assert layer(w8, lora=tabs).fp8_block and layer(w8, hs_codes=True).hs_codes
