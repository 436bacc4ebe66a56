"""Block-scaled fp8 grouped GEMMs against the fp64 definition: both tile heights, ragged widths, sparse
and skewed experts, split tails, codes out, and the chain norm -> gate/up -> down -> combine.

Bars.  The products of two E4M3 codes are exact and a sum of n of them in fp32 is off by at most
n 2^-24 of the sum of their magnitudes (n = K plus a scaled sum per block of 128).  With bf16 out the
fp8 MFMA forms them, which rounds the sum of neighbouring products at about 2^-14 of the largest
(measured against fp64: at most 2^-12.7 of the sum of magnitudes for four products, less for more;
unbiased): 2^-12.5 of the magnitudes in its place.  bf16 out rounds by 2^-8 of itself; SiLU's exponential
and reciprocal by 2^-20 of h.  Codes stand for h within half a step
(2^-4 of it, 2^-10 of the scale below the normal range)."""
import numpy as np
import pytest
import torch

import oracle
from _util import bf16_dev, bf16_host, to_dev
from moe_synth import f32_to_bf16_bits

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
    return m.gemm_workspace("cuda")


def codes(rng, *shape):
    return (rng.integers(4 * 8, 11 * 8, shape) | (rng.integers(0, 2, shape) << 7)).astype(np.uint8)


def weight(rng, E, N, K):
    # scales spread over two powers of two, so a wrong block shows
    return {"codes": codes(rng, E, N, K), "scales": rng.uniform(0.001, 0.008, (E, -(-N // 128), -(-K // 128))).astype(np.float32)}


def dev_weight(m, w):
    return m.Fp8BlockWeight(to_dev(w["codes"]), to_dev(w["scales"]))


def routed(m, rng, T, E, k, bs, empty=()):
    """Routing of T tokens; ``empty`` experts get none, and some ids are out of range (dropped)."""
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[np.isin(ids, empty)] = -1
    return m.moe_align(to_dev(ids), E, bs), ids


def reference(w0, w1, a, sa, r, ids, k, down):
    """acc or h of every pair [P, N] in fp64 with its fp32 noise (sum of magnitudes)."""
    inv = r.inv_sorted.cpu().numpy()
    P = ids.size
    N, K = w0["codes"].shape[1:]
    A = oracle.e4m3_to_f64(a) * oracle.spread_blocks(sa.astype(np.float64), K)
    val, mag = np.zeros((P, N)), np.zeros((P, N))
    for e in range(w0["codes"].shape[0]):
        mine = np.flatnonzero((ids.reshape(-1) == e) & (inv[:P] >= 0))
        if not len(mine):
            continue
        x = A[inv[mine]] if down else A[mine // k]
        W = oracle.fp8_block_matrix(w0, e)
        g, gm = x @ W.T, np.abs(x) @ np.abs(W.T)
        if down:
            val[mine], mag[mine] = g, gm
            continue
        U = oracle.fp8_block_matrix(w1, e)
        u, um = x @ U.T, np.abs(x) @ np.abs(U.T)
        val[mine] = oracle.silu(g) * u
        mag[mine] = 1.1 * np.abs(u) * gm + np.abs(oracle.silu(g)) * um
    return val, mag, inv[:P]


def check_rows(got, ref, mag, inv, K):
    """bf16 rows of the real pairs; returns the row mask."""
    real = inv >= 0
    n = (K + K // 128 + 8) * 2.0 ** -24 + 2.0 ** -12.5
    o = got[inv[real]]
    bar = (2.0 ** -8 + 2.0 ** -20) * np.abs(ref[real]) + n * mag[real]
    worst = np.max(np.abs(o - ref[real]) / np.maximum(bar, 1e-300))
    print(f"  {real.sum()} rows, worst |diff|/bar {worst:.3f}", flush=True)
    assert worst <= 1.0


def check_codes(q, s, ref, mag, inv, K):
    real = inv >= 0
    n = (K + K // 128 + 8) * 2.0 ** -24
    h, noise = ref[real], n * mag[real] + 2.0 ** -20 * np.abs(ref[real])
    sg = s[inv[real]].astype(np.float64)
    amax = oracle.block_amax(h)
    want = np.where(amax > 0, np.maximum(amax, 2.0 ** -100) / 448.0, 1.0)
    assert np.all(np.abs(sg - want) <= 2.0 ** -22 * want + oracle.block_amax(noise) / 448.0)
    se = oracle.spread_blocks(sg, h.shape[1])
    v = oracle.e4m3_to_f64(q[inv[real]]) * se
    bar = (2.0 ** -4 + 2.0 ** -20) * np.abs(h) + 2.0 ** -10 * se + 2 * noise
    worst = np.max(np.abs(v - h) / np.maximum(bar, 1e-300))
    print(f"  {real.sum()} rows, worst code |diff|/bar {worst:.3f}", flush=True)
    assert worst <= 1.0


# name: T, E, k, bs, N, K, experts without tokens
SHAPES = {
    "tall": (300, 2, 1, 64, 256, 512, ()),          # 256-row tiles (experts average 128 rows or more)
    "tall_ragged": (333, 2, 1, 16, 400, 656, ()),   # N, K end inside a block; an expert's rows inside a tile
    "tall_wide_k": (290, 2, 1, 128, 136, 2064, ()),
    "short": (50, 4, 2, 16, 256, 512, ()),          # 128-row tiles
    "short_ragged": (37, 8, 2, 16, 400, 1040, (3,)),
    "short_one": (1, 8, 2, 16, 128, 256, ()),
    "tiny": (5, 3, 2, 16, 16, 16, ()),
    "many_experts": (64, 160, 8, 16, 144, 272, tuple(range(40, 60))),
    "all_dropped_but_one": (20, 4, 1, 32, 64, 144, (0, 1, 3)),
    # several tiles per workgroup (more tiles than compute units), 3 to 5 stages each: the next tile's
    # rows prepared inside the loop
    "multi_tall": (1500, 4, 1, 64, 6144 + 128, 400, ()),
    "multi_short": (900, 16, 1, 16, 6400, 512, ()),
    # split tail: few tiles with a long contraction
    "split_tall": (520, 3, 1, 64, 768, 4112, ()),
    "split_short": (200, 6, 2, 16, 512, 4096, ()),
}


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("use_ws", [False, True], ids=["", "ws"])
def test_gate_up(m, ws, name, use_ws):
    T, E, k, bs, N, K, empty = SHAPES[name]
    rng = np.random.default_rng(len(name) + T)
    print(f"gate_up {name} T={T} E={E} k={k} N={N} K={K} ws={use_ws}", flush=True)
    r, ids = routed(m, rng, T, E, k, bs, empty)
    w0, w1 = weight(rng, E, N, K), weight(rng, E, N, K)
    a, sa = codes(rng, T, K), rng.uniform(0.005, 0.08, (T, -(-K // 128))).astype(np.float32)
    d0, d1, da, ds = dev_weight(m, w0), dev_weight(m, w1), to_dev(a), to_dev(sa)
    work = ws if use_ws else None
    ref, mag, inv = reference(w0, w1, a, sa, r, ids, k, False)
    out = torch.full((r.max_pad, N), 9.0, dtype=torch.bfloat16, device="cuda")
    m.moe_grouped_gemm_fp8_block(0, da, ds, d0, d1, r, out=out, workspace=work)
    o = bf16_host(out)
    check_rows(o, ref, mag, inv, K)
    pad = np.ones(r.max_pad, bool)
    pad[inv[inv >= 0]] = False
    assert (o[pad] == 9.0).all(), "a row without a token was written"
    again = torch.full_like(out, 9.0)
    m.moe_grouped_gemm_fp8_block(0, da, ds, d0, d1, r, out=again, workspace=work)
    assert torch.equal(out, again)
    if N % 16 == 0:
        q = torch.full((r.max_pad, N), 0x33, dtype=torch.uint8, device="cuda")
        s = torch.full((r.max_pad, -(-N // 128)), -5.0, device="cuda")
        assert m.moe_grouped_gemm_fp8_block(0, da, ds, d0, d1, r, q=q, scale=s, workspace=work) is None
        qh, sh = q.cpu().numpy(), s.cpu().numpy()
        check_codes(qh, sh, ref, mag, inv, K)
        assert (qh[pad] == 0x33).all() and (sh[pad] == -5.0).all()


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("use_ws", [False, True], ids=["", "ws"])
def test_down(m, ws, name, use_ws):
    T, E, k, bs, N, K, empty = SHAPES[name]
    rng = np.random.default_rng(len(name) + T)
    print(f"down {name} T={T} E={E} k={k} N={N} K={K} ws={use_ws}", flush=True)
    r, ids = routed(m, rng, T, E, k, bs, empty)
    w0 = weight(rng, E, N, K)
    a, sa = codes(rng, r.max_pad, K), rng.uniform(0.005, 0.08, (r.max_pad, -(-K // 128))).astype(np.float32)
    ref, mag, inv = reference(w0, None, a, sa, r, ids, k, True)
    pad = np.ones(r.max_pad, bool)
    pad[inv[inv >= 0]] = False
    a[pad], sa[pad] = 0x7F, np.nan     # rows without a token hold anything
    out = torch.full((r.max_pad, N), 9.0, dtype=torch.bfloat16, device="cuda")
    m.moe_grouped_gemm_fp8_block(1, to_dev(a), to_dev(sa), dev_weight(m, w0), None, r, out=out,
                                 workspace=ws if use_ws else None)
    o = bf16_host(out)
    check_rows(o, ref, mag, inv, K)
    assert (o[pad] == 9.0).all()


def test_zero_blocks_and_rows(m):
    """A zero activation row gives zero codes with scale 1; a zero weight block adds nothing."""
    rng = np.random.default_rng(4)
    T, E, k, N, K = 20, 2, 1, 256, 384
    r, ids = routed(m, rng, T, E, k, 16)
    w0, w1 = weight(rng, E, N, K), weight(rng, E, N, K)
    w0["scales"][:, 1, 2] = 0.0
    w1["codes"][:, 128:, :] = 0
    a, sa = codes(rng, T, K), rng.uniform(0.01, 0.05, (T, 3)).astype(np.float32)
    a[7] = 0
    ref, mag, inv = reference(w0, w1, a, sa, r, ids, k, False)
    q = torch.zeros((r.max_pad, N), dtype=torch.uint8, device="cuda")
    s = torch.zeros((r.max_pad, 2), device="cuda")
    m.moe_grouped_gemm_fp8_block(0, to_dev(a), to_dev(sa), dev_weight(m, w0), dev_weight(m, w1), r, q=q, scale=s)
    qh, sh = q.cpu().numpy(), s.cpu().numpy()
    check_codes(qh, sh, ref, mag, inv, K)
    assert not (qh[inv[7]] & 0x7F).any() and (sh[inv[7]] == 1).all() and (sh[inv, 1] == 1).all()


def test_split_tail_shares_the_workspace_with_the_other_gemms(m, ws):
    """The block-scaled form leaves the shared workspace as the other grouped GEMMs need it."""
    rng = np.random.default_rng(6)
    T, E, k, N, K = 200, 6, 2, 512, 4096
    r, _ = routed(m, rng, T, E, k, 16)
    w = dev_weight(m, weight(rng, E, N, K))
    wb = m.Bf16Weight(torch.randn((E, N, K), device="cuda", dtype=torch.bfloat16) * 0.02)
    a, sa = to_dev(codes(rng, T, K)), to_dev(rng.uniform(0.01, 0.05, (T, K // 128)).astype(np.float32))
    x = torch.randn((T, K), device="cuda", dtype=torch.bfloat16)
    real = r.sorted_ids < T * k
    first = None
    for _ in range(3):
        o8 = m.moe_grouped_gemm_fp8_block(0, a, sa, w, w, r, workspace=ws)[real]
        ob = m.moe_grouped_gemm(0, x, wb, wb, r, workspace=ws)[real]
        first = first or (o8, ob)
        assert torch.equal(o8, first[0]) and torch.equal(ob, first[1])
    assert not ws[:4096].any()


def test_norm_gate_up_down_combine_chain(m, ws):
    """The operators as a layer runs them, captured in a graph and replayed: norm with block codes,
    routing, gate/up with codes out, down, combine; stage by stage against the definitions on the GPU's
    own inputs to each stage, and bit for bit the same on every replay."""
    rng = np.random.default_rng(11)
    T, H, I, E, k, bs = 96, 1024, 400, 8, 2, 16
    wg, wu, wd = weight(rng, E, I, H), weight(rng, E, I, H), weight(rng, E, H, I)
    dg, du, dd = (dev_weight(m, w) for w in (wg, wu, wd))
    xb = f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    rb = f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    nb = f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(H)).astype(np.float32))
    x, res, nw = bf16_dev(xb), bf16_dev(rb), bf16_dev(nb)
    logits = to_dev(rng.standard_normal((T, E)).astype(np.float32))
    h = torch.empty_like(x)
    xq, sx = torch.empty((T, H), dtype=torch.uint8, device="cuda"), torch.empty((T, 8), device="cuda")
    r = m.Routing.allocate(T * k, k, E, bs, "cuda")
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    hq, sh = torch.zeros((r.max_pad, I), dtype=torch.uint8, device="cuda"), torch.zeros((r.max_pad, 4), device="cuda")
    ys, out = torch.zeros((r.max_pad, H), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)

    def step():
        m.moe_rmsnorm(x, nw, 1e-6, residual=res, residual_out=h, q=xq, scale=sx)
        m.moe_route_align(logits, k, True, bs, ids, w, r)
        m.moe_grouped_gemm_fp8_block(0, xq, sx, dg, du, r, q=hq, scale=sh, workspace=ws)
        m.moe_grouped_gemm_fp8_block(1, hq, sh, dd, None, r, out=ys, workspace=ws)
        m.moe_combine(ys, r.inv_sorted, w, out=out)
    step()
    torch.cuda.synchronize()
    eager = [t.clone() for t in (h, xq, sx, hq, sh, ys, out)]
    hd, yd = oracle.rmsnorm(xb, nb, 1e-6, rb)
    assert np.array_equal(bf16_host(h), hd)
    v = oracle.e4m3_to_f64(xq.cpu().numpy()) * oracle.spread_blocks(sx.cpu().numpy().astype(np.float64), H)
    assert np.all(np.abs(v - yd) <= (2.0 ** -4 + 2e-5) * np.abs(yd) + 2.0 ** -10 * oracle.spread_blocks(sx.cpu().numpy(), H))
    idh = ids.cpu().numpy()
    ref, mag, inv = reference(wg, wu, xq.cpu().numpy(), sx.cpu().numpy(), r, idh, k, False)
    check_codes(hq.cpu().numpy(), sh.cpu().numpy(), ref, mag, inv, H)
    ref, mag, inv = reference(wd, None, hq.cpu().numpy(), sh.cpu().numpy(), r, idh, k, True)
    check_rows(bf16_host(ys), ref, mag, inv, I)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in (h, xq, sx, hq, sh, ys, out):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((h, xq, sx, hq, sh, ys, out), eager))
