"""A whole training step of the layer: its chain bit for bit, its gradients against the token-by-token fp64
layer, and the step in graphs and over batches.

Bars.  The step rounds to bf16 at g, u, h, Ys and out, and at d, dg, du, w h, the pairs' dx and the results: each
2^-8 of a value at most, independent of the others.  A gradient's rounding noise is then a few times 2^-8 of its
terms, added up at random over them; 2e-2 of the tensor's norm (row by row for d_x, expert by expert for the
weights) is five such roundings, the bar of the forward layer.

d_w is no sum over many independent rows but one dot product sum_i d_i h_i a pair, whose terms may cancel, so its bar
is of the terms: d_i, g_i and u_i are rounded by 2^-8 of themselves; h = SiLU(g) u moves with u one to one, and with g
by its relative slope 1 + g (1 - sigmoid(g)), at most 1.3 for g > 0 and max(1, |g|) below.  So the error is at most
2^-8 sum_i |d_i h_i| (2 + 1.3 + |g_i|), and 2% more for products of two roundings and the fp32 sums before them."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def make(m, T, H, I, E, k, bs, seed=0, renormalize=True):
    g = torch.Generator().manual_seed(seed)
    bf = lambda s, *shape: (s * torch.randn(shape, generator=g)).bfloat16().cuda()
    wg, wu, wd = bf(H ** -0.5, E, I, H), bf(H ** -0.5, E, I, H), bf(I ** -0.5, E, H, I)
    layer = m.MoeLayer(E, H, I, k, bs, m.Bf16Weight(wg), m.Bf16Weight(wu), m.Bf16Weight(wd), renormalize=renormalize)
    return layer, torch.randn((T, E), generator=g).cuda(), bf(1.0, T, H), bf(1.0, T, H)


def close(got, want, axes):
    got = f64(got)
    err = np.sqrt(((got - want) ** 2).sum(axis=axes))
    size = np.sqrt((want ** 2).sum(axis=axes))
    assert np.all(err <= 2e-2 * size), (err / np.maximum(size, 1e-300)).max()


CASES = [(1, 64, 32, 4, 2, 16, 0.0, True), (1, 64, 32, 4, 1, 16, 0.5, False), (23, 72, 104, 5, 2, 16, 0.0, True),
         (64, 256, 128, 8, 2, 16, 0.4, True), (96, 136, 264, 6, 3, 32, 0.1, False), (200, 264, 72, 3, 1, 128, 0.0, False)]


@pytest.mark.parametrize("T,H,I,E,k,bs,p,renormalize", CASES)
def test_step_against_fp64(m, T, H, I, E, k, bs, p, renormalize):
    print(f"step T={T} H={H} I={I} E={E} k={k} bs={bs} p={p} renormalize={renormalize}", flush=True)
    layer, logits, x, d_out = make(m, T, H, I, E, k, bs, T, renormalize)
    b = layer.train_plan(T, "cuda", dropout=p, seed=11)
    b.rng[1] = 4
    out = layer.train_forward(logits, x, b).clone()
    d_x, d_l, grads = layer.train_backward(d_out, x, b, None if renormalize else logits)
    ids, w = b.ids.cpu().numpy(), f64(b.w)
    f = oracle.dropout_factors(np.arange(T * k), I, p, 11, 4)
    want = oracle.train_layer(f64(x), *(f64(v.w) for v in (layer.gate, layer.up, layer.down)), ids, w, f, f64(d_out))
    close(out, want[0], 1)
    close(d_x, want[1], 1)
    ex, tok = ids.reshape(-1), np.arange(T * k) // k
    g, u = (np.einsum("rih,rh->ri", f64(v.w)[ex], f64(x)[tok]) for v in (layer.gate, layer.up))
    terms = np.abs(g / (1 + np.exp(-g)) * u * f * np.einsum("rhi,rh->ri", f64(layer.down.w)[ex], f64(d_out)[tok]))
    bar = (1.02 * 2.0 ** -8 * terms * (3.3 + np.abs(g))).sum(1).reshape(T, k)
    assert np.all(np.abs(f64(b.d_w) - want[2]) <= bar)
    for got, ref in zip(grads, want[3:]):
        close(got, ref, (1, 2))
        used = np.isin(np.arange(E), ids)
        assert not f64(got)[~used].any()
    ref = oracle.route_backward(ids, w, f64(b.d_w), E, None if renormalize else f64(logits))
    np.testing.assert_allclose(f64(d_l), ref, rtol=1e-6, atol=1e-6 * np.abs(f64(b.d_w)).max())


def test_step_is_its_chain(m):
    T, H, I, E, k, bs = 77, 264, 136, 6, 2, 16
    layer, logits, x, d_out = make(m, T, H, I, E, k, bs)
    b = layer.train_plan(T, "cuda", dropout=0.2, seed=5)
    out = layer.train_forward(logits, x, b).clone()
    d_x, d_l, grads = layer.train_backward(d_out, x, b)
    ids, w = m.moe_route(logits, k)
    r = m.moe_align(ids, E, bs)
    real = torch.nonzero(r.sorted_ids < T * k).reshape(-1)
    ws, rng = m.gemm_workspace("cuda"), torch.tensor([5, 0]).cuda()
    g = m.moe_grouped_gemm(m.MOE_OP_GATHER, x, layer.gate, None, r, workspace=ws)
    u = m.moe_grouped_gemm(m.MOE_OP_GATHER, x, layer.up, None, r, workspace=ws)
    h = m.moe_silu_mul_dropout(g, u, r, 0.2, rng)
    ys = m.moe_grouped_gemm(m.MOE_OP_DOWN, h, layer.down, None, r, workspace=ws)
    assert torch.equal(m.moe_combine(ys, r.inv_sorted, w), out)
    d = m.moe_grouped_gemm_dgrad(d_out, layer.down, r, by_token=True, workspace=ws)
    dg, du, hw, dw = m.moe_silu_mul_backward(g, u, d, w, r, 0.2, rng)
    want = (m.moe_grouped_gemm_wgrad(dg, x, r, x_by_token=True, workspace=ws),
            m.moe_grouped_gemm_wgrad(du, x, r, x_by_token=True, workspace=ws),
            m.moe_grouped_gemm_wgrad(d_out, hw, r, dy_by_token=True, workspace=ws))
    assert all(torch.equal(a, c) for a, c in zip(grads, want))
    dxs = m.moe_grouped_gemm_dgrad(dg, layer.gate, r, dy1=du, w1=layer.up, workspace=ws)
    assert torch.equal(m.moe_combine(dxs, r.inv_sorted, torch.ones_like(w)), d_x)
    assert torch.equal(m.moe_route_backward(ids, w, dw, E), d_l)
    assert torch.equal(b.ys[real], dxs[real])


def test_without_dropout_the_forward_is_the_unfused_path(m):
    layer, logits, x, _ = make(m, 50, 128, 72, 4, 2, 16)
    b = layer.train_plan(50, "cuda")
    f = layer.plan(50, "cuda")
    out = layer.train_forward(logits, x, b)
    m.moe_route_align(logits, 2, True, 16, f.ids, f.w, f.routing)
    g = m.moe_grouped_gemm(m.MOE_OP_GATHER, x, layer.gate, None, f.routing, workspace=f.ws)
    u = m.moe_grouped_gemm(m.MOE_OP_GATHER, x, layer.up, None, f.routing, workspace=f.ws)
    layer_out = m.moe_combine(m.moe_grouped_gemm(m.MOE_OP_DOWN, m.moe_silu_mul(g, u, f.hs, f.routing), layer.down, None,
                                                 f.routing, out=f.ys, workspace=f.ws), f.routing.inv_sorted, f.w)
    assert torch.equal(out, layer_out)


def test_accumulation_over_batches(m):
    """fp32 sums over three batches are the batches' fp32 gradients, added one after the other."""
    layer, logits, x, d_out = make(m, 40, 72, 136, 5, 2, 16)
    b = layer.train_plan(40, "cuda", dropout=0.1)
    shapes = [(5, 136, 72), (5, 136, 72), (5, 72, 136)]
    total = tuple(torch.full(s, float("nan"), device="cuda") for s in shapes)
    want = [torch.zeros(s, device="cuda") for s in shapes]
    for step in range(3):
        one = tuple(torch.empty(s, device="cuda") for s in shapes)
        b.rng[1] = step
        layer.train_forward(logits.roll(step, 1), x, b)
        layer.train_backward(d_out, x, b, grads=one)
        layer.train_forward(logits.roll(step, 1), x, b)
        layer.train_backward(d_out, x, b, grads=total, accumulate=step > 0)
        for a, c in zip(want, one):
            a += c
    for a, c in zip(want, total):
        assert torch.equal(a, c)


def test_backward_runs_once_for_each_forward(m):
    layer, logits, x, d_out = make(m, 8, 64, 32, 4, 2, 16)
    b = layer.train_plan(8, "cuda")
    layer.train_forward(logits, x, b)
    layer.train_backward(d_out, x, b)
    with pytest.raises(ValueError, match="train_forward"):
        layer.train_backward(d_out, x, b)


def test_step_in_a_graph(m):
    """A captured step, replayed with other inputs, offsets and eager work in between, is the eager step."""
    layer, logits, x, d_out = make(m, 130, 264, 136, 6, 2, 16)
    b = layer.train_plan(130, "cuda", dropout=0.3, seed=9)
    e = layer.train_plan(130, "cuda", dropout=0.3, seed=9)
    grads = tuple(torch.empty_like(w.w) for w in (layer.gate, layer.up, layer.down))

    def step():
        layer.train_forward(logits, x, b)
        layer.train_backward(d_out, x, b, grads=grads)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        b.rng[1] = i
        e.rng[1] = i
        logits.copy_(logits.roll(1, 1))
        x.mul_(-1)
        graph.replay()
        out = layer.train_forward(logits, x, e)
        got = layer.train_backward(d_out, x, e)
        torch.cuda.synchronize()
        assert torch.equal(out, b.out) and torch.equal(got[0], b.d_x) and torch.equal(got[1], b.d_logits)
        assert all(torch.equal(p, q) for p, q in zip(got[2], grads))


def test_directional_difference(m):
    """The loss <out, d_out> along one direction of all inputs, by a central difference of the fp64 layer at the
    GPU's routing, is the sum of the GPU's gradients along it."""
    T, H, I, E, k = 24, 72, 40, 4, 2
    layer, logits, x, d_out = make(m, T, H, I, E, k, 16, seed=3)
    b = layer.train_plan(T, "cuda")
    layer.train_forward(logits, x, b)
    d_x, d_l, (dg, du, dd) = layer.train_backward(d_out, x, b)
    ids = b.ids.cpu().numpy()
    rng = np.random.default_rng(0)
    at = [f64(v) for v in (x, layer.gate.w, layer.up.w, layer.down.w, logits)]
    along = [rng.standard_normal(v.shape) * np.abs(v).mean() for v in at]

    def loss(s):
        X, wg, wu, wd, lg = (v + s * a for v, a in zip(at, along))
        p = np.exp(np.take_along_axis(lg, ids, 1))
        w = p / p.sum(1, keepdims=True)
        return (oracle.train_layer(X, wg, wu, wd, ids, w, np.ones((T * k, I)), f64(d_out))[0] * f64(d_out)).sum()
    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    parts = [(f64(v) * a).sum() for v, a in zip((d_x, dg, du, dd, d_l), along)]
    noise = np.sqrt(sum(((f64(v) * a) ** 2).sum() for v, a in zip((d_x, dg, du, dd, d_l), along)))
    assert abs(sum(parts) - slope) <= 2e-2 * noise + 1e-3 * abs(slope)


def test_no_tokens(m):
    layer, *_ = make(m, 4, 64, 32, 4, 2, 16)
    b = layer.train_plan(0, "cuda")
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert layer.train_forward(torch.empty((0, 4), device="cuda"), z, b).shape == (0, 64)
    d_x, d_l, grads = layer.train_backward(z, z, b)
    assert d_x.shape == (0, 64) and d_l.shape == (0, 4) and not any(g.any() for g in grads)
