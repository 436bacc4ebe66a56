"""SiLU * up with dropout, its backward and the gradient of the router's logits, against the fp64 oracle.

Bars.  Outputs are one rounding away from fp32 values: 2^-8 of themselves in bf16.  The fp32 values use
a hardware exponential and reciprocal: exp(-g) is exp2(-g log2 e), whose argument is rounded (|g| log2 e 2^-24
relative, 2^-19 for |g| <= 20) and whose result is good to a few ulps, and a handful of products of 2^-24
each; 2^-17 of every term covers them.  d_gate is a sum of two terms that may cancel, so its slack is taken of
the terms.  d_topk_w is a sum of n products in fp32: n 2^-24 of the sum of magnitudes beside the terms' own slack.
d_logits is computed in fp64 from the fp32 inputs and rounded once: 2^-24 of itself, and 2^-50 of its terms."""
import numpy as np
import pytest
import torch

import oracle
from _util import bf16_dev

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -17
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def make(m, T, k, E, bs, n, seed, drop_ids=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.argsort(torch.rand((T, E), generator=g), dim=1)[:, :k].int()
    if drop_ids and T:
        ids[::3, 0] = -1
        ids[1::4, k - 1] = E + 2
    r = m.moe_align(ids.cuda().contiguous(), E, bs)
    rows = lambda s: (s * torch.randn((r.max_pad, n), generator=g)).bfloat16().cuda()
    sid = r.sorted_ids.cpu().numpy()
    real = np.nonzero((sid >= 0) & (sid < T * k))[0]
    return r, ids, rows(2.0), rows(1.0), rows(0.1), torch.rand((T, k), generator=g).cuda(), real, sid[real]


SHAPES = [  # T, k, E, bs, n
    (1, 1, 1, 16, 8), (3, 2, 4, 16, 24), (64, 2, 8, 16, 128), (37, 3, 5, 32, 520), (50, 2, 8, 64, 768), (20, 6, 64, 16, 1408),
    (9, 1, 2, 128, 2048), (9, 2, 3, 16, 2056), (6, 2, 8, 16, 14336), (130, 8, 128, 16, 104)]
SEED, OFFSET = 0x1234567890ABCDEF, (3 << 32) + 17


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.75, 0.99999])
def test_dropout_forward_and_backward(m, shape, p):
    T, k, E, bs, n = shape
    print(f"dropout {shape} p={p}", flush=True)
    r, ids, g, u, d, w, real, pairs = make(m, T, k, E, bs, n, n + T, drop_ids=True)
    rng = torch.tensor([SEED, OFFSET]).cuda()
    f = oracle.dropout_factors(pairs, n, p, SEED, OFFSET)
    G, U, D, Wt = f64(g)[real], f64(u)[real], f64(d)[real], f64(w).reshape(-1)[pairs]
    mark = torch.full_like(g, 7.5)
    h = m.moe_silu_mul_dropout(g, u, r, p, rng, out=mark.clone())
    want = oracle.silu_mul_dropout(G, U, f)
    assert np.all(np.abs(f64(h)[real] - want) <= (HALF + SLACK) * np.abs(want))
    assert np.array_equal(f64(h)[real] == 0, want == 0) or p == 0
    rest = np.setdiff1d(np.arange(r.max_pad), real)
    assert np.all(f64(h)[rest] == 7.5)

    dw0 = torch.full((T, k), -3.0).cuda()
    dg, du, hw, dw = m.moe_silu_mul_backward(g, u, d, w, r, p, rng, d_gate=mark.clone(), d_up=mark.clone(),
                                             h_weighted=mark.clone(), d_topk_w=dw0)
    wdg, wdu, whw, wdw = oracle.silu_mul_backward(G, U, D, Wt, f)
    s = 1 / (1 + np.exp(-G))
    terms = np.abs(Wt[:, None] * D * f * U) * (s + np.abs(G) * s * (1 - s))
    assert np.all(np.abs(f64(dg)[real] - wdg) <= HALF * np.abs(wdg) + (SLACK + HALF * SLACK) * terms)
    for got, ref in ((du, wdu), (hw, whw)):
        assert np.all(np.abs(f64(got)[real] - ref) <= (HALF + SLACK) * np.abs(ref))
    size = np.abs(D * whw / Wt[:, None]).sum(1)
    assert np.all(np.abs(f64(dw).reshape(-1)[pairs] - wdw) <= (SLACK + n * 2.0 ** -24) * size)
    for t in (dg, du, hw):
        assert np.all(f64(t)[rest] == 7.5)
    lost = np.setdiff1d(np.arange(T * k), pairs)
    assert np.all(f64(dw).reshape(-1)[lost] == -3.0)

    # in place, any output on any input: the same bits
    for a, b, c in ((0, 1, 2), (2, 0, 1), (1, 2, 0)):
        x = [g.clone(), u.clone(), d.clone()]
        got = m.moe_silu_mul_backward(*x, w, r, p, rng, d_gate=x[a], d_up=x[b], h_weighted=x[c], d_topk_w=dw0.clone())
        for one, two in zip(got[:3], (dg, du, hw)):
            assert torch.equal(one[real], two[real])
        assert torch.equal(got[3], dw)
    x = g.clone()
    assert torch.equal(m.moe_silu_mul_dropout(x, u, r, p, rng, out=x)[real], h[real])
    # allocated outputs: the weights' gradient of pairs without an expert is zero
    assert np.all(f64(m.moe_silu_mul_backward(g, u, d, w, r, p, rng)[3]).reshape(-1)[lost] == 0)


def test_without_routing_rows_are_pairs(m):
    g = torch.Generator().manual_seed(5)
    rows = lambda: torch.randn((33, 264), generator=g).bfloat16().cuda()
    G, U, D, w = rows(), rows(), rows(), torch.rand(33, generator=g).cuda()
    rng = torch.tensor([-5, -9]).cuda()   # all 64 bits of both count
    f = oracle.dropout_factors(np.arange(33), 264, 0.4, -5, -9)
    h = m.moe_silu_mul_dropout(G, U, p=0.4, rng=rng)
    want = oracle.silu_mul_dropout(f64(G), f64(U), f)
    assert np.all(np.abs(f64(h) - want) <= (HALF + SLACK) * np.abs(want))
    dw = m.moe_silu_mul_backward(G, U, D, w, p=0.4, rng=rng)[3]
    ref = oracle.silu_mul_backward(f64(G), f64(U), f64(D), f64(w), f)[3]
    size = np.abs(f64(D) * want).sum(1)
    assert np.all(np.abs(f64(dw) - ref) <= (SLACK + 264 * 2.0 ** -24) * size)


def test_masks_of_steps_and_pairs(m):
    """The share that is dropped, and that offsets, seeds and pairs have masks of their own."""
    one = torch.ones((64, 4096), dtype=torch.bfloat16, device="cuda")
    mask = lambda s, o: m.moe_silu_mul_dropout(one, one, p=0.25, rng=torch.tensor([s, o]).cuda()) != 0
    a = mask(1, 0)
    n = a.numel()
    assert abs(a.float().mean().item() - 0.75) < 5 * np.sqrt(0.75 * 0.25 / n)
    assert torch.equal(a, mask(1, 0))
    for other in (mask(1, 1), mask(2, 0), mask(1, 1 << 32), mask(1 + (1 << 32), 0), a.roll(1, 0), a.roll(1, 1), a.roll(8, 1)):
        same = (a == other).float().mean().item()
        assert abs(same - (0.75 ** 2 + 0.25 ** 2)) < 0.01


def test_extreme_values(m):
    """Large gates: SiLU saturates to 0 or g, its slope to 0 or 1, and nothing becomes NaN; a NaN stays in its
    own column of the rows, and a dropped one is gone."""
    g = torch.tensor([[-1e4, -100.0, -40.0, 0.0, 40.0, 100.0, 1e4, 3e38]]).bfloat16().cuda()
    u, d, w = torch.full_like(g, 2.0), torch.full_like(g, 0.5), torch.ones(1).cuda()
    h = m.moe_silu_mul_dropout(g, u)
    assert torch.equal(h[0, 3:7], (2 * g)[0, 3:7]) and torch.isfinite(h[0, :7]).all() and h[0, :2].abs().max() < 1e-30
    dg, du, hw, dw = m.moe_silu_mul_backward(g[:, :8].contiguous(), u, d, w)
    assert torch.isfinite(dg[0, :7]).all()
    assert torch.equal(dg[0, [0, 3, 5, 6]].float().cpu(), torch.tensor([0.0, 0.5, 1.0, 1.0]))
    n = torch.ones((1, 16), dtype=torch.bfloat16, device="cuda")
    n[0, 5] = float("nan")
    out = m.moe_silu_mul_dropout(n, torch.ones_like(n))
    assert torch.isnan(out).nonzero().tolist() == [[0, 5]]
    # p near 1: 16 bits at most 65535 are dropped, 1 in 65536 kept
    rng = torch.tensor([0, 0]).cuda()
    assert not torch.isnan(m.moe_silu_mul_dropout(n, torch.ones_like(n), p=0.9999999, rng=rng)).any()


def test_no_rows(m):
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert m.moe_silu_mul_dropout(z, z).shape == (0, 64)
    assert m.moe_silu_mul_backward(z, z, z, torch.empty(0, device="cuda"))[3].shape == (0,)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 4, 2), (5, 64, 6), (7, 63, 1), (9, 65, 8), (11, 128, 8), (4, 200, 200),
                                   (6, 256, 8), (3, 256, 256), (1030, 8, 2)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward(m, T, E, k, renormalize):
    print(f"route_backward T={T} E={E} k={k} renormalize={renormalize}", flush=True)
    g = torch.Generator().manual_seed(T + E)
    lg = torch.randn((T, E), generator=g).cuda()
    ids, w = m.moe_route(lg, k, renormalize)
    dw = torch.randn((T, k), generator=g).cuda()
    ids = ids.clone()
    if T > 2:   # ids without an expert, whose gradient may hold anything, and an id that comes twice
        ids[1, 0], dw[1, 0] = -1, float("nan")
        ids[2, k - 1], dw[2, k - 1] = E, float("inf")
        if k > 1:
            ids[0, 1] = ids[0, 0]
    got = f64(m.moe_route_backward(ids, w, dw, E, None if renormalize else lg))
    I, Wt, D = ids.cpu().numpy(), f64(w), f64(dw)
    D = np.where((I >= 0) & (I < E), D, 0)
    want = oracle.route_backward(I, Wt, D, E, None if renormalize else f64(lg))
    size = np.abs(D).max(1, keepdims=True) * (1 + np.abs(Wt).sum(1, keepdims=True)) * k
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -50 * size)
    if renormalize and k == 1 and T <= 2:
        assert np.all(got == 0)


def test_streams_and_graph(m):
    """A captured chain replays with the numbers that its buffers hold then; another stream's calls alike."""
    r, ids, g, u, d, w, real, pairs = make(m, 40, 2, 8, 16, 264, 1)
    rng = torch.tensor([3, 0]).cuda()
    h, dg, du, hw = (torch.zeros_like(g) for _ in range(4))
    dw, dl = torch.zeros((40, 2), device="cuda"), torch.zeros((40, 8), device="cuda")
    did = ids.cuda()

    def chain(h, dg, du, hw, dw, dl):
        m.moe_silu_mul_dropout(g, u, r, 0.3, rng, out=h)
        m.moe_silu_mul_backward(g, u, d, w, r, 0.3, rng, d_gate=dg, d_up=du, h_weighted=hw, d_topk_w=dw)
        m.moe_route_backward(did, w, dw, 8, out=dl)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(h, dg, du, hw, dw, dl)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(h, dg, du, hw, dw, dl)
    for step in range(4):
        rng[1] = step
        d.mul_(-1.5)
        outs = [torch.zeros_like(t) for t in (h, dg, du, hw, dw, dl)]
        chain(*outs)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((h, dg, du, hw, dw, dl), outs):
            assert torch.equal(a, b)
