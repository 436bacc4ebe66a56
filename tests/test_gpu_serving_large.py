"""The serving operators past 32-bit offsets and past one pass of their grids.  Rows are independent in
the norm and the quantisation, so slices of a large call equal calls on the slices bit for bit (those are
checked against fp64 elsewhere); products are checked on sampled rows with the bars of their own tests."""
import numpy as np
import pytest
import torch

import oracle
from _util import bf16_host
from test_gpu_fp8_block import check_codes, check_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


# more rows than one pass of the grid (2^20 workgroups of 4 rows or of one), and more than 2^31 elements
@pytest.mark.parametrize("rows,k", [(4 * 2 ** 20 + 7, 16), (2 ** 20 + 3, 2064)])
@pytest.mark.parametrize("out", ["row", "block"])
def test_rmsnorm_many_rows(m, rows, k, out):
    print(f"rmsnorm rows={rows} k={k} {out}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, k), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(k, generator=g, device="cuda", dtype=torch.bfloat16)
    shape = (lambda n: (n,)) if out == "row" else (lambda n: (n, -(-k // 128)))
    y, q, s = torch.empty_like(x), torch.empty((rows, k), dtype=torch.uint8, device="cuda"), torch.empty(shape(rows), device="cuda")
    m.moe_rmsnorm(x, w, residual=x, residual_out=x, y=y, q=q, scale=s)     # h = 2 x, in place
    for lo, hi in ((0, 5), (rows // 2, rows // 2 + 9), (2 ** 20 - 2, 2 ** 20 + 3), (rows - 6, rows)):
        part = x[lo:hi].clone()
        yp, qp, sp = torch.empty_like(part), torch.empty((hi - lo, k), dtype=torch.uint8, device="cuda"), torch.empty(shape(hi - lo), device="cuda")
        m.moe_rmsnorm(part, w, y=yp, q=qp, scale=sp)
        assert torch.equal(yp, y[lo:hi]) and torch.equal(qp, q[lo:hi]) and torch.equal(sp, s[lo:hi]), (lo, hi)


def test_quantize_block_many_rows(m):
    rows, k = 2 ** 20 + 3, 4112        # more than 2^32 elements, more rows than workgroups
    print(f"quantize rows={rows} k={k}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(k)
    x = torch.randn((rows, k), generator=g, device="cuda", dtype=torch.bfloat16)
    q, s = torch.empty((rows, k), dtype=torch.uint8, device="cuda"), torch.empty((rows, 33), device="cuda")
    m.moe_quantize_fp8_block(x, q, s)
    for lo, hi in ((0, 5), (2 ** 20 - 2, 2 ** 20 + 3)):
        part = x[lo:hi].clone()
        qp, sp = torch.empty((hi - lo, k), dtype=torch.uint8, device="cuda"), torch.empty((hi - lo, 33), device="cuda")
        m.moe_quantize_fp8_block(part, qp, sp)
        assert torch.equal(qp, q[lo:hi]) and torch.equal(sp, s[lo:hi])


@pytest.mark.parametrize("codes_out", [False, True])
def test_gate_up_output_past_4_gib(m, codes_out):
    T, E, k, N, K = 140000, 4, 2, 16384, 144      # 280 000 rows of 16384 columns
    print(f"gate_up T={T} N={N} K={K} codes={codes_out}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: (torch.randint(32, 88, s, generator=g, device="cuda", dtype=torch.uint8)
                      | (torch.randint(0, 2, s, generator=g, device="cuda", dtype=torch.uint8) << 7))
    uni = lambda lo, hi, *s: torch.rand(s, generator=g, device="cuda") * (hi - lo) + lo
    w0, w1 = (m.Fp8BlockWeight(rnd(E, N, K), uni(0.001, 0.008, E, N // 128, 2)) for _ in range(2))
    a, sa = rnd(T, K), uni(0.005, 0.08, T, 2)
    ids = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(64)]).int().repeat(-(-T // 64), 1)[:T].contiguous()
    r = m.moe_align(ids, E, 64)
    if codes_out:
        q, s = torch.empty((r.max_pad, N), dtype=torch.uint8, device="cuda"), torch.empty((r.max_pad, N // 128), device="cuda")
        m.moe_grouped_gemm_fp8_block(0, a, sa, w0, w1, r, q=q, scale=s)
    else:
        out = m.moe_grouped_gemm_fp8_block(0, a, sa, w0, w1, r)
    inv = r.inv_sorted[: T * k].cpu().numpy()
    order = np.argsort(inv)
    pairs = order[[0, 1, len(order) // 3, len(order) // 2, 2 * len(order) // 3, -2, -1]]
    idn = ids.cpu().numpy().reshape(-1)
    assert int(inv[pairs].max()) * N > 2 ** 32
    val, mag = np.zeros((len(pairs), N)), np.zeros((len(pairs), N))
    host = lambda w: {"codes": w.codes.cpu().numpy(), "scales": w.scales.cpu().numpy()}
    h0, h1 = host(w0), host(w1)
    A = oracle.e4m3_to_f64(a[pairs // k].cpu().numpy()) * oracle.spread_blocks(sa[pairs // k].cpu().numpy().astype(np.float64), K)
    for i, p in enumerate(pairs):
        W, U = oracle.fp8_block_matrix(h0, idn[p]), oracle.fp8_block_matrix(h1, idn[p])
        gt, u = W @ A[i], U @ A[i]
        val[i] = oracle.silu(gt) * u
        mag[i] = 1.1 * np.abs(u) * (np.abs(W) @ np.abs(A[i])) + np.abs(oracle.silu(gt)) * (np.abs(U) @ np.abs(A[i]))
    rows = torch.from_numpy(inv[pairs].astype(np.int64)).cuda()
    here = np.arange(len(pairs))
    if codes_out:
        check_codes(q[rows].cpu().numpy(), s[rows].cpu().numpy(), val, mag, here, K)
    else:
        check_rows(bf16_host(out[rows]), val, mag, here, K)


@pytest.mark.parametrize("T", [2, 20])
def test_few_tokens_weights_past_4_gib(m, T):
    E, k, H, I = 220, 2, 4096, 2560               # 4.6 GB a projection
    print(f"few tokens E={E} H={H} I={I} T={T}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(T)
    ws = []
    for n, c in ((I, H), (I, H), (H, I)):
        w = torch.empty((E, n, c), dtype=torch.bfloat16, device="cuda")
        for e in range(E):
            w[e] = 0.02 * torch.randn((n, c), generator=g, device="cuda")
        ws.append(m.Bf16Weight(w))
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits[:, E - 1] = 9.0                        # the last expert for every token
    out, ids, w = m.moe_few_tokens(m.few_tokens_plan(*ws, k, T), logits, x)
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            gt, u = ws[0].w[e].double() @ x[t].double(), ws[1].w[e].double() @ x[t].double()
            want[t] += w[t, j].double() * (ws[2].w[e].double() @ (gt / (1 + torch.exp(-gt)) * u))
    assert (ids == E - 1).any(1).all()
    err = ((out.double() - want).norm(dim=1) / want.norm(dim=1)).max().item()
    print(f"  worst row {err:.2e}", flush=True)
    assert err <= 2.0 ** -8                       # out's rounding, half a step of each element
