"""Training operators, CPU side: the library exports what training/moe_training.h declares, the C ABI, the
binding and the layer refuse invalid calls before anything is enqueued, and the oracle's functions are
pinned to published vectors, to torch's autograd and to differences."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import mixture_experts_routed_route_amd as m
import oracle
from _util import ROOT
from mixture_experts_routed_route_amd._lib import MoeWeight

HEADER = os.path.join(ROOT, "include", "training", "moe_training.h")


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
    assert names == set(_lib.TRAINING_SIGNATURES)
    for n in names:
        assert hasattr(L, n), f"{n} not exported"


# ------------------------------------------------------------------ refusals of the C ABI
F = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails validation or has nothing to do
OFF = ctypes.c_void_p((1 << 20) + 8)
W = ctypes.byref(MoeWeight(0, 0, 1 << 20, None, None))
W4 = ctypes.byref(MoeWeight(1, 128, 1 << 20, 1 << 20, 1 << 20))
MP = 2 * 8 + 4 * 16  # padded rows of 8 tokens, 2 of 4 experts, blocks of 16 (at least 76, in whole blocks)


def drop(rows=4, n=64, p=0.1, rng=F, g=F, u=F, out=F, ids=None, pairs=4):
    return "moe_silu_mul_dropout", (g, u, out, ids, pairs, rows, n, p, rng, None)


def back(rows=4, n=64, p=0.1, rng=F, d=F, w=F, ids=None, pairs=4, dg=F, du=ctypes.c_void_p(2 << 20),
         hw=ctypes.c_void_p(3 << 20), dw=F):
    return "moe_silu_mul_backward", (F, F, d, w, ids, pairs, rows, n, p, rng, dg, du, hw, dw, None)


def dgrad(dy=F, w0=W, dy1=None, w1=None, dx=F, ids=F, off=F, pairs=16, k=2, E=4, n=64, kk=64, bs=16, mp=MP, ws=None, nws=0):
    return "moe_grouped_gemm_dgrad", (dy, w0, dy1, w1, dx, ids, off, pairs, k, E, n, kk, bs, mp, 0, ws, nws, None)


def wgrad(dy=F, x=F, dw=F, base=None, ids=F, off=F, pairs=16, k=2, E=4, n=64, kk=64, bs=16, mp=MP, ws=None, nws=0):
    return "moe_grouped_gemm_wgrad", (dy, x, dw, base, 0, ids, off, pairs, k, E, n, kk, bs, mp, 0, 0, ws, nws, None)


def rback(ids=F, w=F, dw=F, logits=None, T=4, E=8, k=2, out=F):
    return "moe_route_backward", (ids, w, dw, logits, T, E, k, out, None)


INVALID = [
    (drop(n=20), "n 20"), (drop(n=0), "n 0"), (drop(rows=-1), "rows"), (drop(p=1.0), "p_drop"), (drop(p=-0.1), "p_drop"),
    (drop(p=float("nan")), "p_drop"), (drop(rng=None), "rng"), (drop(g=None), "gate"), (drop(out=OFF), "out"),
    (drop(ids=OFF), "sorted_ids"), (drop(pairs=-1), "num_pairs"),
    (back(n=12), "n 12"), (back(rows=5), "num_pairs 4 < rows 5"), (back(p=1.5), "p_drop"), (back(rng=None), "rng"),
    (back(d=None), "d is NULL"), (back(w=None), "topk_w"), (back(du=F), "one buffer"), (back(hw=F), "one buffer"),
    (back(dw=OFF), "d_topk_w"), (back(dg=None), "d_gate"),
    (dgrad(pairs=15), "multiple of top_k"), (dgrad(k=0), "top_k"), (dgrad(E=0), "num_experts"), (dgrad(n=60), "n 60"),
    (dgrad(kk=4), "k 4"), (dgrad(bs=24), "block_size"), (dgrad(mp=MP - 16), "max_pad"), (dgrad(mp=MP + 8), "max_pad"),
    (dgrad(w0=None), "w0"), (dgrad(dy1=F), "go together"), (dgrad(w1=W), "go together"), (dgrad(dy=None), "dy0"),
    (dgrad(dx=OFF), "dx"), (dgrad(ids=None), "sorted_ids"), (dgrad(off=None), "expert_offsets"),
    (dgrad(ws=F, nws=64), "workspace_bytes"), (dgrad(ws=OFF, nws=1 << 40), "workspace"), (dgrad(pairs=-2), "num_pairs"),
    (wgrad(pairs=15), "multiple of top_k"), (wgrad(n=4), "n 4"), (wgrad(kk=100), "k 100"), (wgrad(dw=None), "dw"),
    (wgrad(base=OFF), "base"), (wgrad(dy=None), "dy"), (wgrad(x=OFF), "x"), (wgrad(mp=0), "max_pad"),
    (wgrad(ws=F, nws=64), "workspace_bytes"),
    (rback(T=-1), "num_tokens"), (rback(E=0), "num_experts"), (rback(k=0), "top_k"), (rback(ids=None), "topk_ids"),
    (rback(logits=OFF), "logits"), (rback(out=None), "d_logits"),
]
UNSUPPORTED = [
    (drop(rows=1 << 30, n=64), "2\\^35"), (back(rows=1 << 24, pairs=1 << 24), "2\\^24"), (dgrad(E=257, mp=16 + 257 * 16), "257"),
    (dgrad(w0=W4), "bf16 weights"), (dgrad(dy1=F, w1=W4), "bf16 weights"), (dgrad(n=(1 << 20) + 8), "2\\^20"),
    (wgrad(E=257, mp=16 + 257 * 16), "257"), (wgrad(n=1 << 20, kk=1 << 20, E=32, mp=16 + 32 * 16), "2\\^28"),
    (rback(E=257), "257"), (rback(k=300), "300"),
]


@pytest.mark.parametrize("call,what", INVALID)
def test_invalid(L, call, what):
    rc = getattr(L, call[0])(*call[1])
    assert rc == -1 and re.search(what, L.moe_last_error().decode()), L.moe_last_error()


F2 = ctypes.c_void_p(2 << 20)
FAR = (1 << 31) - 1024   # a multiple of every block size; the rows past a span's end would pass 32 bits


@pytest.mark.parametrize("call", [dgrad(dx=F2, mp=FAR), wgrad(dw=F2, mp=FAR)])
def test_rows_past_32_bits(L, call):
    test_unsupported(L, call, "max_pad")


@pytest.mark.parametrize("call,what", [
    (dgrad(), "dx is one buffer"), (dgrad(dx=F2, dy1=F2, w1=W), "dx is one buffer"),
    (wgrad(dw=F2, dy=F2), "dw is one buffer"), (wgrad(dw=F2, x=F2), "dw is one buffer")])
def test_results_over_operands(L, call, what):
    """Rows are read for one tile after another tile was written: refused."""
    test_invalid(L, call, what)


@pytest.mark.parametrize("call,what", UNSUPPORTED)
def test_unsupported(L, call, what):
    rc = getattr(L, call[0])(*call[1])
    assert rc == -2 and re.search(what, L.moe_last_error().decode()), L.moe_last_error()


@pytest.mark.parametrize("call", [drop(rows=0, g=None, u=None, out=None), back(rows=0, pairs=0, d=None, dg=None),
                                  drop(ids=F, pairs=0, rng=None), back(ids=F, pairs=0, w=None, dw=None),
                                  dgrad(pairs=0, dy=None, dx=None), rback(T=0, ids=None)])
def test_nothing_to_do(L, call):
    assert getattr(L, call[0])(*call[1]) == 0


# ------------------------------------------------------------------ refusals of the binding (CPU tensors)
T, H, I, E, K, BS = 8, 64, 32, 4, 2, 16


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def routing():
    return m.Routing.allocate(T * K, K, E, BS, "cpu")


R = routing()
RP = R.max_pad
RNG = torch.zeros(2, dtype=torch.int64)
WT = lambda *s: m.Bf16Weight(bf(*s))
BINDING = [
    (lambda: m.moe_silu_mul_dropout(bf(RP, I), bf(RP, I + 8), R), "up is"),
    (lambda: m.moe_silu_mul_dropout(bf(RP, I), bf(RP, I), R, out=bf(RP - 1, I)), "out is"),
    (lambda: m.moe_silu_mul_dropout(bf(RP + 1, I), bf(RP + 1, I), R), "sorted_ids"),
    (lambda: m.moe_silu_mul_dropout(bf(RP, I), bf(RP, I), R, p=0.5), "needs rng"),
    (lambda: m.moe_silu_mul_dropout(bf(RP, I), bf(RP, I), R, p=1.0, rng=RNG), "needs \\[0, 1\\)"),
    (lambda: m.moe_silu_mul_dropout(bf(RP, I), bf(RP, I), R, p=0.5, rng=RNG[:1]), "shape \\(2,\\)"),
    (lambda: m.moe_silu_mul_dropout(bf(RP), bf(RP), R), "rows, n"),
    (lambda: m.moe_silu_mul_backward(bf(RP, I), bf(RP, I), bf(RP, I - 8), torch.zeros(T, K), R), "d is"),
    (lambda: m.moe_silu_mul_backward(bf(RP, I), bf(RP, I), bf(RP, I), torch.zeros(T - 1, K), R), "topk_w"),
    (lambda: m.moe_silu_mul_backward(bf(RP, I), bf(RP, I), bf(RP, I), torch.zeros(T, K), R, d_topk_w=torch.zeros(1)), "d_topk_w"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP, I), WT(E - 1, I, H), R), "experts"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP, I), WT(E, I + 8, H), R), "width"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP - 1, I), WT(E, I, H), R), "rows"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(T - 1, I), WT(E, I, H), R, by_token=True), "rows"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP, I), WT(E, I, H), R, out=bf(RP - 1, H)), "out is"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP, I), WT(E, I, H), R, dy1=bf(RP, I)), "go together"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP, I), WT(E, I, H), R, dy1=bf(RP, I), w1=WT(E, I, H + 8)), "one shape"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP, I), m.Fp8Weight(torch.zeros(E, I, H, dtype=torch.uint8), torch.zeros(E, I)), R), "bf16 weights"),
    (lambda: m.moe_grouped_gemm_wgrad(bf(RP - 1, I), bf(T, H), R, x_by_token=True), "rows"),
    (lambda: m.moe_grouped_gemm_wgrad(bf(RP, I), bf(T - 1, H), R, x_by_token=True), "rows"),
    (lambda: m.moe_grouped_gemm_wgrad(bf(RP, I), bf(RP, H), R, out=bf(E, H, I)), "out is not"),
    (lambda: m.moe_grouped_gemm_wgrad(bf(RP, I), bf(RP, H), R, base=bf(E, I, H - 8), out=bf(E, I, H)), "base is not"),
    (lambda: m.moe_grouped_gemm_wgrad(bf(RP, I), bf(RP, H), R, out=torch.zeros(E, I, H, dtype=torch.float16)), "float32"),
    (lambda: m.moe_grouped_gemm_wgrad(bf(I), bf(RP, H), R), "two dimensions"),
    (lambda: m.moe_route_backward(torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K), torch.zeros(T, K + 1), E), "d_topk_w"),
    (lambda: m.moe_route_backward(torch.zeros(T, K, dtype=torch.int32), torch.zeros(T, K), torch.zeros(T, K), E,
                                  logits=torch.zeros(T, E + 1)), "logits"),
    (lambda: m.moe_route_backward(torch.zeros(T * K, dtype=torch.int32), torch.zeros(T, K), torch.zeros(T, K), E), "T, k"),
    # and with good shapes the last refusal: not on a HIP device
    (lambda: m.moe_silu_mul_dropout(bf(RP, I), bf(RP, I), R), "HIP device"),
    (lambda: m.moe_grouped_gemm_wgrad(bf(RP, I), bf(RP, H), R), "HIP device"),
    (lambda: m.moe_grouped_gemm_dgrad(bf(RP, I), WT(E, I, H), R), "HIP device"),
]


@pytest.mark.parametrize("call,what", BINDING)
def test_binding_refuses(L, call, what):
    with pytest.raises(ValueError, match=what):
        call()


def layer(**kw):
    return m.MoeLayer(E, H, I, K, BS, WT(E, I, H), WT(E, I, H), WT(E, H, I), **kw)


def test_layer_refuses(L):
    f8 = m.Fp8Weight(torch.zeros(E, I, H, dtype=torch.uint8), torch.zeros(E, I))
    with pytest.raises(ValueError, match="bf16"):
        m.MoeLayer(E, H, I, K, BS, f8, f8, m.Fp8Weight(torch.zeros(E, H, I, dtype=torch.uint8), torch.zeros(E, H))).train_plan(T, "cpu")
    with pytest.raises(ValueError, match="LoRA"):
        layer(lora=object()).train_plan(T, "cpu")
    with pytest.raises(ValueError, match="dropout"):
        layer().train_plan(T, "cpu", dropout=1.0)
    b = layer().train_plan(T, "cpu")
    with pytest.raises(ValueError, match="train_forward"):
        layer().train_backward(bf(T, H), bf(T, H), b)
    b.forward_done = True
    with pytest.raises(ValueError, match="logits"):
        layer(renormalize=False).train_backward(bf(T, H), bf(T, H), b)
    with pytest.raises(ValueError, match="accumulate"):
        layer().train_backward(bf(T, H), bf(T, H), b, accumulate=True)
    with pytest.raises(ValueError, match="d_out"):
        layer().train_backward(bf(T - 1, H), bf(T, H), b)
    for wrong in ((bf(E, I, H), bf(E, I, H), bf(E, I, H)), (bf(E, I, H), bf(E, I, H).half(), bf(E, H, I)),
                  (bf(E, H, I).transpose(1, 2), bf(E, I, H), bf(E, H, I))):   # before anything is added to the others
        with pytest.raises(ValueError, match="grads"):
            layer().train_backward(bf(T, H), bf(T, H), b, grads=wrong, accumulate=True)
    with pytest.raises(ValueError, match="contiguous bfloat16"):
        layer().train_backward(bf(T, H).float(), bf(T, H), b)
    assert b.forward_done


# ------------------------------------------------------------------ the oracle
def test_philox_vectors():
    """Known answers that the generator's authors publish (kat_vectors of Random123)."""
    ones = 2**32 - 1
    pi = [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]
    for c, k, want in [((0,) * 4, (0,) * 2, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
                       ((ones,) * 4, (ones,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
                       (*pi, (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        assert tuple(int(v) for v in oracle.philox4x32(c, k)) == want


def test_dropout_factors():
    f = oracle.dropout_factors(np.arange(400), 203, 0.3, 77, 5)
    p = round(0.3 * 65536) / 65536
    assert set(np.unique(f)) == {0.0, 1 / (1 - p)}
    assert abs((f == 0).mean() - p) < 5 * np.sqrt(p * (1 - p) / f.size)
    # each (pair, column) alone decides: other pairs, widths and orders give the same values
    assert np.array_equal(oracle.dropout_factors([7, 3], 50, 0.3, 77, 5), f[[7, 3], :50])
    assert not np.array_equal(oracle.dropout_factors([7], 203, 0.3, 77, 6), f[[7]])
    assert np.all(oracle.dropout_factors([1], 9, 0.0, 1, 1) == 1)


def small(seed, T=5, H=6, I=8, E=3, k=2):
    g = np.random.default_rng(seed)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    return (g.standard_normal((T, H)), g.standard_normal((E, I, H)), g.standard_normal((E, I, H)),
            g.standard_normal((E, H, I)), ids, g.uniform(0.1, 1, (T, k)), g.integers(0, 2, (T * k, I)) * 1.5,
            g.standard_normal((T, H)))


def test_layer_gradients_against_differences():
    x, wg, wu, wd, ids, w, f, d_out = small(1)
    ids[0, 1] = -1   # a pair without an expert
    out, *grads = oracle.train_layer(x, wg, wu, wd, ids, w, f, d_out)
    args = [x, w, wg, wu, wd]
    loss = lambda: (oracle.train_layer(x, wg, wu, wd, ids, w, f, d_out)[0] * d_out).sum()
    step = 1e-6
    rng = np.random.default_rng(0)
    for a, grad in zip(args, grads):
        for i in rng.choice(a.size, min(a.size, 25), replace=False):
            at = np.unravel_index(i, a.shape)
            keep = a[at]
            a[at] = keep + step
            up = loss()
            a[at] = keep - step
            slope = (up - loss()) / (2 * step)
            a[at] = keep
            assert abs(slope - grad[at]) < 1e-6 * (1 + abs(slope))


def test_operators_make_the_layer():
    """The grouped operators, chained as the header says, give the gradients of the token-by-token layer."""
    x, wg, wu, wd, ids, w, f, d_out = small(2, T=17)
    k, Ec = ids.shape[1], len(wg)
    al = oracle.align(ids.astype(np.int32), Ec, 16)
    sid, off, P = al["sorted_ids"], al["offsets"], ids.size
    real = (sid >= 0) & (sid < P)
    p = np.where(real, sid, 0)
    tok, ex = p // k, ids.reshape(-1)[p]
    g = np.einsum("rih,rh->ri", wg[ex], x[tok])
    u = np.einsum("rih,rh->ri", wu[ex], x[tok])
    d, _ = oracle.grouped_dgrad([d_out], [wd], sid, off, P, k, True)
    dg, du, hw, dw = oracle.silu_mul_backward(g, u, d, w.reshape(-1)[p], f[p])
    d_wd, _ = oracle.grouped_wgrad(d_out, hw, sid, off, P, k, True, False)
    d_wg, _ = oracle.grouped_wgrad(dg, x, sid, off, P, k, False, True)
    d_wu, _ = oracle.grouped_wgrad(du, x, sid, off, P, k, False, True)
    rows, _ = oracle.grouped_dgrad([dg, du], [wg, wu], sid, off, P, k, False)
    d_x = np.zeros_like(x)
    np.add.at(d_x, tok[real], rows[real])
    d_w = np.zeros(P)
    d_w[p[real]] = dw[real]
    want = oracle.train_layer(x, wg, wu, wd, ids, w, f, d_out)
    for a, b in zip((d_x, d_w.reshape(w.shape), d_wg, d_wu, d_wd), want[1:]):
        np.testing.assert_allclose(a, b, rtol=1e-10, atol=1e-10)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_against_autograd(renormalize):
    g = np.random.default_rng(3)
    lg = torch.tensor(g.standard_normal((9, 7)), requires_grad=True)
    ids = torch.argsort(lg.detach(), dim=1, descending=True)[:, :3]
    w = torch.softmax(lg, 1).gather(1, ids)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    dw = torch.tensor(g.standard_normal((9, 3)))
    (w * dw).sum().backward()
    got = oracle.route_backward(ids.numpy(), w.detach().numpy(), dw.numpy(), 7, None if renormalize else lg.detach().numpy())
    np.testing.assert_allclose(got, lg.grad.numpy(), rtol=1e-12, atol=1e-14)
