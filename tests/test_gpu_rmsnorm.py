"""Residual addition + root-mean-square norm + E4M3 output, and block quantisation, against the fp64
oracle.

Bars.  h is the correctly rounded sum: exact.  y differs from the fp64 value by one rounding to bf16
(2^-8 of itself) and by fp32 arithmetic: the sum of squares of positive terms, at most 40 sequential
fp32 additions deep per lane plus the reduction here (k / 256 * 8 for the widest row: 4096 + 16 roundings of 2^-24
each, 2.5e-4 as a worst case at k = 131072, halved by the square root), and five more roundings;
1.5e-4 covers it.  A code stands for its value within half a step (2^-4 of it, or 2^-10 of the scale
for subnormal codes), beside the same fp32 slack, and its scale is within that slack.  Block
quantisation of bf16 rows is decided in fp32 on both sides: bit-exact."""
import numpy as np
import pytest
import torch

import oracle
from _util import bf16_dev, bf16_host, bits_host
from moe_synth import f32_to_bf16_bits

pytestmark = pytest.mark.gpu
SLACK = 1.5e-4


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


def rows_of(rng, rows, k, std=1.0):
    return f32_to_bf16_bits((std * rng.standard_normal((rows, k))).astype(np.float32))


def check_codes(q, scale, y, block):
    """Codes and scales of exact values y."""
    amax = oracle.block_amax(y) if block else np.abs(y).max(axis=1, keepdims=True)
    s = scale.cpu().numpy().astype(np.float64).reshape(amax.shape)
    want = np.where(amax > 0, np.maximum(amax, 2.0 ** -100) / 448.0, 1.0)
    assert np.all(np.abs(s - want) <= SLACK * want)
    se = oracle.spread_blocks(s, y.shape[1]) if block else s
    v = oracle.e4m3_to_f64(q.cpu().numpy()) * se
    assert np.all(np.abs(v - y) <= (2.0 ** -4 + SLACK) * np.abs(y) + 2.0 ** -10 * se)


# widths: one per kernel form (1, 2 and 4 chunks a lane on one wave; 2, 4 and 8 on four; the two-pass
# form), on both sides of each border, and widths that end inside a block of 128
WIDTHS = [16, 64, 496, 512, 528, 1024, 1040, 2048, 2064, 4096, 4112, 5136, 8192, 8208, 16384, 16400, 131072]


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("out", ["bf16", "row", "block"])
def test_rmsnorm_widths(m, k, out):
    rows = 5 if k <= 16400 else 2
    rng = np.random.default_rng(k)
    xb, rb, wb = rows_of(rng, rows, k), rows_of(rng, rows, k, 2.0), rows_of(rng, 1, k)[0]
    print(f"rmsnorm rows={rows} k={k} out={out}", flush=True)
    h, y = oracle.rmsnorm(xb, wb, 1e-6, rb)
    x, r, w = bf16_dev(xb), bf16_dev(rb), bf16_dev(wb)
    yo = torch.full_like(x, 7.0)
    q = scale = None
    if out != "bf16":
        q = torch.full((rows, k), 0x55, dtype=torch.uint8, device="cuda")
        scale = torch.full((rows,) if out == "row" else (rows, -(-k // 128)), -1.0, device="cuda")
    m.moe_rmsnorm(x, w, 1e-6, residual=r, y=yo, q=q, scale=scale)   # r takes h in place
    assert np.array_equal(bf16_host(r), h)
    assert np.all(np.abs(bf16_host(yo) - y) <= (2.0 ** -8 + SLACK) * np.abs(y))
    if q is not None:
        check_codes(q, scale, y, out == "block")


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 63, 1000])
def test_rmsnorm_row_counts_without_residual(m, rows):
    rng = np.random.default_rng(rows)
    k = 640
    xb, wb = rows_of(rng, rows, k), rows_of(rng, 1, k)[0]
    _, y = oracle.rmsnorm(xb, wb, 1e-5)
    got = m.moe_rmsnorm(bf16_dev(xb), bf16_dev(wb), 1e-5)
    assert np.all(np.abs(bf16_host(got) - y) <= (2.0 ** -8 + SLACK) * np.abs(y))
    q, s = torch.empty((rows, k), dtype=torch.uint8, device="cuda"), torch.empty((rows, 5), device="cuda")
    assert m.moe_rmsnorm(bf16_dev(xb), bf16_dev(wb), 1e-5, q=q, scale=s) is None
    check_codes(q, s, y, True)


@pytest.mark.parametrize("k", [256, 4096, 20000])
def test_rmsnorm_buffers_that_coincide(m, k):
    """h in place of the residual or of x, y in place of x: the documented aliases, each equal to the
    call on separate buffers."""
    rng = np.random.default_rng(k)
    xb, rb, wb = rows_of(rng, 6, k), rows_of(rng, 6, k), rows_of(rng, 1, k)[0]
    w = bf16_dev(wb)
    h, y = torch.empty((6, k), dtype=torch.bfloat16, device="cuda"), torch.empty((6, k), dtype=torch.bfloat16, device="cuda")
    m.moe_rmsnorm(bf16_dev(xb), w, 1e-6, residual=bf16_dev(rb), residual_out=h, y=y)
    x, r = bf16_dev(xb), bf16_dev(rb)
    m.moe_rmsnorm(x, w, 1e-6, residual=r, y=x)
    assert torch.equal(r, h) and torch.equal(x, y)
    x, r, y2 = bf16_dev(xb), bf16_dev(rb), torch.empty_like(y)
    m.moe_rmsnorm(x, w, 1e-6, residual=r, residual_out=x, y=y2)
    assert torch.equal(x, h) and torch.equal(y2, y) and np.array_equal(bits_host(r), rb)
    x = bf16_dev(xb)
    one = m.moe_rmsnorm(bf16_dev(xb), w)
    m.moe_rmsnorm(x, w, y=x)
    assert torch.equal(x, one)


@pytest.mark.parametrize("k", [128, 2176, 16400])
def test_rmsnorm_zeros_and_non_finite_rows(m, k):
    """Rows of zeros, a row whose values are tiny, and rows holding an infinity or a NaN: the formula's
    values (a NaN or infinity spoils its own row only)."""
    rng = np.random.default_rng(3)
    v = rng.standard_normal((6, k)).astype(np.float32)
    v[0] = 0
    v[1] *= 1e-30
    v[2, 5] = np.inf
    v[3, 7] = np.nan
    v[5, : k // 2] = 0
    x = torch.from_numpy(v).bfloat16().cuda()
    w = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty((6, k), dtype=torch.uint8, device="cuda"), torch.empty((6, -(-k // 128)), device="cuda")
    y = torch.empty_like(x)
    m.moe_rmsnorm(x, w, 1e-6, y=y, q=q, scale=s)
    xd = x.double().cpu()
    want = xd / torch.sqrt((xd * xd).mean(1, keepdim=True) + 1e-6)
    got = y.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert (got[ok] - want[ok]).abs().le((2.0 ** -8 + SLACK) * want[ok].abs() + 1e-38).all()
    codes = q.cpu().numpy()
    assert not codes[0].any() and (s[0] == 1).all()
    assert ((codes[3] & 0x7F) == 0x7F).all() and (s[3] == 1).all()
    assert (codes[2, 5] & 0x7F) == 0x7F and not (np.delete(codes[2], 5) & 0x7F).any()  # 0x80 is -0
    fin = [1, 4, 5]
    check_codes(q[fin], s[fin], want[fin].numpy(), True)


def test_rmsnorm_same_bits_every_time_and_on_a_stream(m):
    rng = np.random.default_rng(9)
    x, r, w = bf16_dev(rows_of(rng, 777, 1408)), bf16_dev(rows_of(rng, 777, 1408)), bf16_dev(rows_of(rng, 1, 1408)[0])

    def call():
        h, y = torch.empty_like(x), torch.empty_like(x)
        q, s = torch.empty((777, 1408), dtype=torch.uint8, device="cuda"), torch.empty(777, device="cuda")
        m.moe_rmsnorm(x, w, 1e-6, residual=r, residual_out=h, y=y, q=q, scale=s)
        return h, y, q, s
    a = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = call()
    side.synchronize()
    assert all(torch.equal(p, v) for p, v in zip(a, b))


@pytest.mark.parametrize("k", [16, 128, 144, 512, 528, 2048, 2064, 4096, 6160, 14336])
def test_quantize_block_bit_exact(m, k):
    rows = 37
    rng = np.random.default_rng(k)
    v = rng.standard_normal((rows, k)) * np.exp(3 * rng.standard_normal((rows, k)))
    v[5] = 0
    v[6, : min(k, 128)] = 0
    v[7] *= 1e-34                      # under the floor
    xb = f32_to_bf16_bits(v.astype(np.float32))
    print(f"quantize_block k={k}", flush=True)
    wq, ws = oracle.quantize_blocks_fp8(oracle.bf16_bits_to_f64(xb))
    q, s = torch.empty((rows, k), dtype=torch.uint8, device="cuda"), torch.empty((rows, -(-k // 128)), device="cuda")
    m.moe_quantize_fp8_block(bf16_dev(xb), q, s)
    assert np.array_equal(q.cpu().numpy(), wq)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), ws.view(np.uint32))


@pytest.mark.parametrize("k", [64, 400, 1408])
def test_quantize_block_sorted_rows_only(m, k):
    """With a routing only real sorted rows are written; dropped ids leave their rows alone too."""
    rng = np.random.default_rng(k)
    T, E, top_k, bs = 29, 7, 3, 16
    ids = torch.from_numpy(rng.integers(-1, E + 1, (T, top_k)).astype(np.int32)).cuda()
    r = m.moe_align(ids, E, bs)
    xb = rows_of(rng, r.max_pad, k)
    q = torch.full((r.max_pad, k), 0x33, dtype=torch.uint8, device="cuda")
    s = torch.full((r.max_pad, -(-k // 128)), -5.0, device="cuda")
    m.moe_quantize_fp8_block(bf16_dev(xb), q, s, r)
    wq, ws = oracle.quantize_blocks_fp8(oracle.bf16_bits_to_f64(xb))
    real = (r.sorted_ids.cpu().numpy() < T * top_k)
    assert 0 < real.sum() < T * top_k
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(q[real], wq[real]) and np.array_equal(s[real], ws[real])
    assert (q[~real] == 0x33).all() and (s[~real] == -5.0).all()
