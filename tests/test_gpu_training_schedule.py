"""Grouped gradient products: the lists of tiles that workgroups run and where operands end, at sizes that the plain
sweeps of types and layouts do not reach.  The bars are those of the sums of exact products: n terms added in fp32 in
any order are off by at most 2 n 2^-24 of their sum of magnitudes, and a rounding to bf16 by 2^-8 of the value (fp32
results: 2^-24, and once more where base is added)."""
import pytest
import torch

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
    w = m.gemm_workspace("cuda")
    yield w
    assert not w[:4096].any()


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def aligned(m, counts, bs, g):
    """A routing that gives expert e counts[e] tokens (one choice each), in random order."""
    ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).int()
    ids = ids[torch.randperm(len(ids), generator=g)]
    return m.moe_align(ids.view(-1, 1).cuda(), len(counts), bs)


def spans(r):
    off, cnt = r.offsets.tolist(), r.counts.tolist()
    return [(e, slice(off[e], off[e] + cnt[e]), r.sorted_ids[off[e]:off[e] + cnt[e]].long()) for e in range(r.num_experts)]


def check_dgrad(dx, r, pairs, columns=slice(None)):
    """pairs: (dy by token, w) each."""
    n = sum(dy.shape[1] for dy, _ in pairs)
    for e, rows, tok in spans(r):
        if len(tok) == 0:
            continue
        want = sum(dy[tok].double() @ w[e][:, columns].double() for dy, w in pairs)
        size = sum(dy[tok].double().abs() @ w[e][:, columns].double().abs() for dy, w in pairs)
        err = (dx[rows][:, columns].double() - want).abs() - (2.0 ** -8 * want.abs() + 2 * n * 2.0 ** -24 * size)
        assert (err <= 0).all(), (e, err.max().item())


def check_wgrad(dw, r, dy, x, base=None, rows_n=slice(None), columns=slice(None)):
    half = 2.0 ** -8 if dw.dtype is torch.bfloat16 else 2.0 ** -24
    for e, _, tok in spans(r):
        a, b = dy[tok][:, rows_n].double(), x[tok][:, columns].double()
        want, size = a.t() @ b, a.abs().t() @ b.abs()
        slack = 2 * (len(tok) + 1) * 2.0 ** -24 * size
        if base is not None:
            want = want + base[e][rows_n, columns].double()
            slack = slack + 2.0 ** -24 * want.abs()
        err = (dw[e][rows_n, columns].double() - want).abs() - (half * want.abs() + slack)
        assert (err <= 0).all(), (e, err.max().item())


def test_lists_longer_than_the_table(m, ws):
    """129 column tiles for 256 experts: 130 tiles per workgroup, two more than are located in advance."""
    g = torch.Generator().manual_seed(0)
    d = torch.Generator(device="cuda").manual_seed(0)
    E, N, K = 256, 8, 129 * 256 + 8
    r = aligned(m, [9] * E, 16, g)
    dy, x, w = normal(d, 9 * E, N), normal(d, 9 * E, K), normal(d, E, N, K)
    for space in (None, ws):
        print(f"long lists, workspace={space is not None}", flush=True)
        dx = m.moe_grouped_gemm_dgrad(dy, m.Bf16Weight(w), r, by_token=True, workspace=space)
        check_dgrad(dx, r, [(dy, w)])
        dw = m.moe_grouped_gemm_wgrad(dy, x, r, True, True, workspace=space)
        check_wgrad(dw, r, dy, x)


@pytest.mark.parametrize("N", [8, 32, 40, 64, 72, 136])
def test_tiles_of_few_halves(m, ws, N):
    """Contractions of 1 to 5 slots in a row of many tiles, whole, half and quarter ones, with and without a pair."""
    g = torch.Generator().manual_seed(N)
    d = torch.Generator(device="cuda").manual_seed(N)
    counts = [0, 300, 1, 256, 64, 65, 0, 128, 129, 513, 31, 33, 96, 0, 160, 255] * 3
    r = aligned(m, counts, 16, g)
    T, E, K = sum(counts), len(counts), 1112
    dys, w = [normal(d, T, N) for _ in range(2)], [normal(d, E, N, K) for _ in range(2)]
    for n in (1, 2):
        print(f"short dgrad N={N} pairs={n}", flush=True)
        args = dict(dy1=dys[1], w1=m.Bf16Weight(w[1])) if n == 2 else {}
        dx = m.moe_grouped_gemm_dgrad(dys[0], m.Bf16Weight(w[0]), r, by_token=True, workspace=ws, **args)
        check_dgrad(dx, r, list(zip(dys, w))[:n])


@pytest.mark.parametrize("N,K", [(520, 520), (72, 1032), (2056, 136), (264, 264)])
@pytest.mark.parametrize("counts", [[0] * 20 + [2100, 1, 33] + [0] * 20 + [40, 700], [30, 31, 32, 33, 64, 65, 100, 129] * 8,
                                    [1500] + [0] * 63, [17 * e % 97 for e in range(128)]])
def test_experts_of_unequal_length(m, ws, N, K, counts):
    """Tiles dealt in turn and levelled over the workgroups; experts without rows get base, or zeros."""
    g = torch.Generator().manual_seed(N)
    d = torch.Generator(device="cuda").manual_seed(N)
    r = aligned(m, counts, 32, g)
    T, E = sum(counts), len(counts)
    dy, x = normal(d, T, N), normal(d, T, K)
    for dtype in (torch.bfloat16, torch.float32):
        print(f"unequal N={N} K={K} E={E} {dtype}", flush=True)
        out = torch.full((E, N, K), float("nan"), dtype=dtype, device="cuda")
        for space in (None, ws):
            check_wgrad(m.moe_grouped_gemm_wgrad(dy, x, r, True, True, out=out, workspace=space), r, dy, x)
            base = normal(d, E, N, K).to(dtype)
            check_wgrad(m.moe_grouped_gemm_wgrad(dy, x, r, True, True, base=base, workspace=space), r, dy, x, base)


@pytest.mark.parametrize("N,K,counts", [(2056, 264, [100]), (4104, 40, [7, 0, 20]), (8200, 520, [260]), (14336, 8, [1]),
                                        (520, 264, [30] * 5), (1000, 72, [3] * 60)])
def test_long_contractions_of_few_tiles(m, ws, N, K, counts):
    """dgrad: the sum over N divided among workgroups, over the border of the pairs and up to an end inside a slot;
    with the operands exchanged, long sums over rows."""
    g = torch.Generator().manual_seed(N)
    d = torch.Generator(device="cuda").manual_seed(N)
    r = aligned(m, counts, 16, g)
    T, E = sum(counts), len(counts)
    dys, w = [normal(d, T, N) for _ in range(2)], [normal(d, E, N, K) for _ in range(2)]
    print(f"few tiles N={N} K={K} E={E}", flush=True)
    for n in (1, 2):
        args = dict(dy1=dys[1], w1=m.Bf16Weight(w[1])) if n == 2 else {}
        dx = m.moe_grouped_gemm_dgrad(dys[0], m.Bf16Weight(w[0]), r, by_token=True, workspace=ws, **args)
        check_dgrad(dx, r, list(zip(dys, w))[:n])
        again = m.moe_grouped_gemm_dgrad(dys[0], m.Bf16Weight(w[0]), r, by_token=True, workspace=ws, **args)
        assert all(torch.equal(dx[rows], again[rows]) for _, rows, _ in spans(r))
    rows = [N] + [N // 3 + 1] * (E - 1)
    r = aligned(m, rows, 16, g)
    dy, x = normal(d, sum(rows), 72), normal(d, sum(rows), K)
    base = torch.randn((E, 72, K), generator=d, device="cuda")
    check_wgrad(m.moe_grouped_gemm_wgrad(dy, x, r, True, True, base=base, workspace=ws), r, dy, x, base)


def test_workspace_of_the_forward_products(m):
    """One workspace for forward and gradient products in turn, each of which leaves its counters at zero."""
    g = torch.Generator().manual_seed(4)
    d = torch.Generator(device="cuda").manual_seed(4)
    counts = [40, 0, 300, 9]
    r = aligned(m, counts, 16, g)
    T, N, K = sum(counts), 2048, 1024
    x, dy, w = normal(d, T, K), normal(d, T, N), m.Bf16Weight(normal(d, 4, N, K))
    shared = m.gemm_workspace("cuda")

    def calls(space):
        return [m.moe_grouped_gemm(m.MOE_OP_GATHER, x, w, None, r, workspace=space()),
                m.moe_grouped_gemm_dgrad(dy, w, r, by_token=True, workspace=space()),
                m.moe_grouped_gemm(m.MOE_OP_GATHER, x, w, None, r, workspace=space()),
                m.moe_grouped_gemm_wgrad(dy, x, r, True, True, workspace=space())]
    want = calls(lambda: m.gemm_workspace("cuda"))
    for _ in range(3):
        got = calls(lambda: shared)
        for i, (a, b) in enumerate(zip(got, want)):
            real = [s for _, s, _ in spans(r)] if i < 3 else [slice(None)]
            assert all(torch.equal(a[s], b[s]) for s in real)
        assert not shared[:4096].any()


def test_weights_past_32_bits(m, ws):
    """Experts' matrices and gradients of 2^31 bytes each and offsets past 2^32 bytes and elements."""
    g = torch.Generator().manual_seed(5)
    d = torch.Generator(device="cuda").manual_seed(5)
    E, N, K = 5, 16384, 65544
    counts = [3, 0, 20, 0, 17]
    r = aligned(m, counts, 16, g)
    T = sum(counts)
    dy, x = normal(d, T, N), normal(d, T, K)
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")   # 10.7 GB
    for e in range(E):
        w[e].normal_(generator=d)
    print("large weights: dgrad", flush=True)
    dx = m.moe_grouped_gemm_dgrad(dy, m.Bf16Weight(w), r, by_token=True, workspace=ws)
    for cols in (slice(0, 520), slice(32700, 33300), slice(K - 300, K)):
        check_dgrad(dx, r, [(dy, w)], cols)
    print("large weights: wgrad", flush=True)
    out = w.fill_(float("nan"))
    m.moe_grouped_gemm_wgrad(dy, x, r, True, True, out=out, workspace=ws)
    for rows_n in (slice(0, 300), slice(8100, 8300), slice(N - 300, N)):
        for cols in (slice(0, 300), slice(32700, 33300), slice(K - 300, K)):
            check_wgrad(out, r, dy, x, None, rows_n, cols)
    assert not any(out[e].isnan().any() for e in range(E)) and not out[1].any() and not out[3].any()
