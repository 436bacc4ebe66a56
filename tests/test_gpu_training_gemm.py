"""Grouped products for input and weight gradients against the fp64 oracle.

Bars.  The products of bf16 values are exact in fp32; a sum of n of them, added in fp32 in any order, is off by
at most n 2^-24 of the sum of magnitudes S (2 n 2^-24 is allowed: the matrix instruction may cut where an addition
rounds), and the result is rounded once: 2^-8 of itself in bf16, 2^-24 in fp32, where adding base rounds once
more.  One product left out or taken twice is off by about S / n, far outside at these n."""
import numpy as np
import pytest
import torch

import oracle
from _util import bf16_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def ws(m):
    """One workspace for every call here: each has to leave it as it found it."""
    w = m.gemm_workspace("cuda")
    yield w
    assert not w[:4096].any()


def f64(t):
    return t.detach().cpu().double().numpy()


def route(m, g, T, k, E, bs, how):
    if how == "one":         # every token's first choice is expert E - 1
        ids = torch.argsort(torch.rand((T, E), generator=g), dim=1)[:, :k]
        ids = torch.where(ids == E - 1, ids[:, :1], ids)
        ids[:, 0] = E - 1
    else:
        ids = torch.argsort(torch.rand((T, E), generator=g), dim=1)[:, :k]
    if how == "dropped":     # pairs without an expert
        ids[::2, 0] = -1
        ids[1::3, k - 1] = E + 5
    return m.moe_align(ids.int().cuda().contiguous(), E, bs)


def operand(g, r, T, width, by_token):
    """bf16 rows; sorted rows without a pair hold NaN."""
    x = torch.randn((T if by_token else r.max_pad, width), generator=g).bfloat16().cuda()
    if not by_token:
        sid = r.sorted_ids.long()
        x[(sid < 0) | (sid >= r.num_pairs)] = float("nan")
    return x


def host(r):
    return r.sorted_ids.cpu().numpy(), r.offsets.cpu().numpy()


# T, k, E, bs, N, K: one value of everything; sizes on both sides of the 64-deep stage and the 256-wide tile;
# experts without rows, one expert with all of them; a contraction of many stages over few tiles
SHAPES = [(1, 1, 1, 16, 8, 8), (2, 2, 3, 16, 16, 24), (5, 1, 2, 32, 64, 256), (9, 2, 4, 16, 72, 264), (33, 3, 7, 16, 200, 40),
          (40, 2, 64, 16, 56, 520), (64, 2, 8, 16, 256, 128), (70, 8, 8, 128, 264, 248), (100, 1, 1, 64, 128, 1032),
          (300, 2, 3, 64, 520, 264), (700, 1, 2, 128, 40, 264), (257, 2, 256, 16, 24, 16), (1500, 2, 2, 64, 264, 520),
          (4100, 1, 1, 16, 16, 264)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("by_token", [False, True])
def test_dgrad(m, ws, shape, pair, by_token):
    T, k, E, bs, N, K = shape
    for how in ("spread", "one", "dropped"):
        if how == "one" and k > 1 and E <= k:
            continue
        print(f"dgrad {shape} pair={pair} by_token={by_token} {how}", flush=True)
        g = torch.Generator().manual_seed(N + K + T)
        r = route(m, g, T, k, E, bs, how)
        dys = [operand(g, r, T, N, by_token) for _ in range(1 + pair)]
        Ws = [torch.randn((E, N, K), generator=g).bfloat16().cuda() for _ in range(1 + pair)]
        sid, off = host(r)
        want, size = oracle.grouped_dgrad([np.nan_to_num(f64(t)) for t in dys], [f64(w) for w in Ws], sid, off, T * k, k, by_token)
        args = dict(dy1=dys[1], w1=m.Bf16Weight(Ws[1])) if pair else {}
        real = (sid >= 0) & (sid < T * k)
        for space in (None, ws):
            out = torch.full((r.max_pad, K), 7.5, dtype=torch.bfloat16, device="cuda")
            m.moe_grouped_gemm_dgrad(dys[0], m.Bf16Weight(Ws[0]), r, by_token=by_token, out=out, workspace=space, **args)
            got = f64(out)
            n = N * (1 + pair)
            err = np.abs(got - want)[real] - (2.0 ** -8 * np.abs(want) + 2 * n * 2.0 ** -24 * size)[real]
            assert np.all(err <= 0), f"workspace={space is not None}: {err.max()}"
            assert np.all(got[~real] == 7.5)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dy_by_token,x_by_token", [(False, False), (True, False), (False, True), (True, True)])
def test_wgrad(m, ws, shape, dy_by_token, x_by_token):
    T, k, E, bs, N, K = shape
    for how in ("spread", "one", "dropped"):
        if how == "one" and k > 1 and E <= k:
            continue
        print(f"wgrad {shape} by_token={dy_by_token},{x_by_token} {how}", flush=True)
        g = torch.Generator().manual_seed(N + K + T)
        r = route(m, g, T, k, E, bs, how)
        dy, x = operand(g, r, T, N, dy_by_token), operand(g, r, T, K, x_by_token)
        sid, off = host(r)
        want, size = oracle.grouped_wgrad(np.nan_to_num(f64(dy)), np.nan_to_num(f64(x)), sid, off, T * k, k, dy_by_token, x_by_token)
        n = r.counts.max().item() + 1
        for dtype, half in ((torch.bfloat16, 2.0 ** -8), (torch.float32, 2.0 ** -24)):
            old = torch.randn((E, N, K), generator=g).to(dtype).cuda()
            for space in (None, ws):
                out = torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda")
                for base in (None, old):
                    got = f64(m.moe_grouped_gemm_wgrad(dy, x, r, dy_by_token, x_by_token, base=base, out=out, workspace=space))
                    ref = want if base is None else want + f64(base)
                    slack = 2 * n * 2.0 ** -24 * size + (0 if base is None else 2.0 ** -24 * np.abs(ref))
                    err = np.abs(got - ref) - (half * np.abs(ref) + slack)
                    assert np.all(err <= 0), f"{dtype} base={base is not None} workspace={space is not None}: {err.max()}"
                into = old.clone()
                m.moe_grouped_gemm_wgrad(dy, x, r, dy_by_token, x_by_token, base=into, out=into, workspace=space)
                assert torch.equal(into, out)


def test_no_pairs(m, ws):
    r = m.moe_align(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4, 16)
    z = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda")
    base = torch.randn((4, 264, 40), device="cuda")
    for space in (None, ws):
        assert not m.moe_grouped_gemm_wgrad(z(0, 264), z(0, 40), r, True, True, out=z(4, 264, 40), workspace=space).any()
        assert torch.equal(m.moe_grouped_gemm_wgrad(z(0, 264), z(0, 40), r, True, True, base=base, workspace=space), base)
        out = z(r.max_pad, 40)
        m.moe_grouped_gemm_dgrad(z(0, 264), m.Bf16Weight(z(4, 264, 40)), r, by_token=True, out=out, workspace=space)
        assert torch.isnan(out).all()


def test_nan_stays_in_its_expert(m, ws):
    """A NaN or infinity in one expert's rows or weights reaches that expert's results only."""
    g = torch.Generator().manual_seed(1)
    r = m.moe_align(torch.arange(96, dtype=torch.int32).remainder(3).view(96, 1).cuda(), 3, 16)   # 32 rows each
    dy, x = torch.randn((96, 72), generator=g).bfloat16().cuda(), torch.randn((96, 264), generator=g).bfloat16().cuda()
    dy[1, 5], dy[4, 6] = float("nan"), float("inf")    # tokens of expert 1
    dw = m.moe_grouped_gemm_wgrad(dy, x, r, True, True, workspace=ws)
    bad = ~torch.isfinite(dw)
    assert bad[1, 5].all() and bad[1, 6].all() and bad.sum() == 2 * 264
    w = torch.randn((3, 72, 264), generator=g).bfloat16().cuda()
    w[2] = float("nan")
    dx = m.moe_grouped_gemm_dgrad(dy.nan_to_num(0, 0), m.Bf16Weight(w), r, by_token=True, workspace=ws)
    assert torch.isfinite(dx[:64]).all() and torch.isnan(dx[64:96]).all()


@pytest.mark.parametrize("seed", range(3))
def test_repeats_and_streams(m, seed):
    """Bit for bit the same on every run, on two streams at once with a workspace each, and in replayed graphs."""
    g = torch.Generator().manual_seed(seed)
    r = route(m, g, 600, 2, 5, 64, "spread")
    dy, x = operand(g, r, 600, 328, True), operand(g, r, 600, 520, False)
    w = m.Bf16Weight(torch.randn((5, 328, 520), generator=g).bfloat16().cuda())
    spaces = [m.gemm_workspace("cuda") for _ in range(2)]

    def both(space):
        dx = torch.zeros((r.max_pad, 520), dtype=torch.bfloat16, device="cuda")
        m.moe_grouped_gemm_dgrad(dy, w, r, by_token=True, out=dx, workspace=space)
        return dx, m.moe_grouped_gemm_wgrad(dy, x, r, True, False, workspace=space)
    first = both(spaces[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for s, space in zip(streams, spaces):
            with torch.cuda.stream(s):
                got.append(both(space))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both(spaces[0])
    for _ in range(3):
        graph.replay()
        both(spaces[0])
        torch.cuda.synchronize()
        got.append(tuple(t.clone() for t in kept))
    for one in got:
        assert all(torch.equal(a, b) for a, b in zip(one, first))


def test_long_rows(m, ws):
    """Row offsets past 2^31 bytes and elements past 2^32 bytes of one operand."""
    T, N, K = 140_000, 8192, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = torch.randn((T, N), generator=g, device="cuda", dtype=torch.bfloat16)   # 2.3 GB
    dy[-3:] *= 8
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ids[-70:] = 1
    r = m.moe_align(ids, 2, 16)
    x = torch.randn((T, K), generator=g, device="cuda", dtype=torch.bfloat16)
    dw = m.moe_grouped_gemm_wgrad(dy, x, r, True, True, out=torch.empty((2, N, K), device="cuda"), workspace=ws)
    for e, part in ((0, slice(0, T - 70)), (1, slice(T - 70, T))):
        want = torch.zeros((N, K), dtype=torch.float64, device="cuda")
        size = torch.zeros_like(want)
        for lo in range(0, len(range(*part.indices(T))), 20_000):
            a, b = dy[part][lo:lo + 20_000].double(), x[part][lo:lo + 20_000].double()
            want += a.t() @ b
            size += a.abs().t() @ b.abs()
        assert ((dw[e] - want).abs() <= 2 * T * 2.0 ** -24 * size + 2.0 ** -24 * want.abs()).all()
        assert (dw[e] - want).abs().max() <= 1e-4 * want.abs().max()
    w = torch.randn((2, N, K), generator=g, device="cuda", dtype=torch.bfloat16)
    dx = m.moe_grouped_gemm_dgrad(dy, m.Bf16Weight(w), r, by_token=True, workspace=ws)
    for row, tok, e in ((0, 0, 0), (T - 71, T - 71, 0), (r.offsets[1].item(), T - 70, 1), (r.offsets[1].item() + 69, T - 1, 1)):
        want = dy[tok].double() @ w[e].double()
        size = dy[tok].double().abs() @ w[e].double().abs()
        assert ((dx[row] - want).abs() <= 2.0 ** -8 * want.abs() + 2 * N * 2.0 ** -24 * size).all()


@pytest.mark.slow
@pytest.mark.parametrize("T,N,K,E,k,bs", [(4096, 1408, 4096, 64, 6, 64), (2048, 768, 2048, 128, 8, 64), (4096, 4096, 1408, 8, 2, 64)])
def test_large(m, ws, T, N, K, E, k, bs):
    """Many tiles per workgroup: every expert against fp64 on the device."""
    g = torch.Generator(device="cuda").manual_seed(N)
    logits = torch.randn((T, E), generator=g, device="cuda") - 1.26 * torch.log(torch.arange(1, E + 1, device="cuda").float())
    ids = torch.argsort(logits, dim=1, descending=True)[:, :k].int().contiguous()
    r = m.moe_align(ids, E, bs)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    dy, dy1, x, w, w1 = normal(r.max_pad, N), normal(r.max_pad, N), normal(T, K), normal(E, N, K), normal(E, N, K)
    off, cnt = r.offsets.tolist(), r.counts.tolist()
    for space in (None, ws):
        dx = m.moe_grouped_gemm_dgrad(dy, m.Bf16Weight(w), r, dy1=dy1, w1=m.Bf16Weight(w1), workspace=space)
        dw = m.moe_grouped_gemm_wgrad(dy, x, r, False, True, workspace=space)
        df = m.moe_grouped_gemm_wgrad(dy, x, r, False, True, out=torch.empty((E, N, K), device="cuda"), workspace=space)
        for e in range(E):
            rows = slice(off[e], off[e] + cnt[e])
            a, a1, b, b1 = (t.double() for t in (dy[rows], dy1[rows], w[e], w1[e]))
            want, size = a @ b + a1 @ b1, a.abs() @ b.abs() + a1.abs() @ b1.abs()
            assert ((dx[rows] - want).abs() <= 2.0 ** -8 * want.abs() + 4 * N * 2.0 ** -24 * size).all()
            xe = x[torch.div(r.sorted_ids[rows].long(), k, rounding_mode="floor")].double()
            want, size = a.t() @ xe, a.abs().t() @ xe.abs()
            assert ((dw[e] - want).abs() <= 2.0 ** -8 * want.abs() + 2 * cnt[e] * 2.0 ** -24 * size).all()
            assert ((df[e] - want).abs() <= 2.0 ** -24 * want.abs() + 2 * cnt[e] * 2.0 ** -24 * size).all()
