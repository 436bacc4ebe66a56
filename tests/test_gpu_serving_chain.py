"""The block-scaled layer end to end against 64 bits, through the layer's own buffers, and the norm's fp32
scales against a bound of their own.

The layer rounds by up to 2^-4 of an element where it quantises, so its output alone cannot show a wrong
scale layout or order of the projections closely.  It is checked in three steps that cover all of it: the
codes of x exactly; the codes of h against the exact h of those x codes, element by element; the output
against the exact product of those h codes.

Bars.  A sum of K products of codes on the fp8 MFMA is within 2^-12.5 + K 2^-24 of the sum of magnitudes (its
rounding of neighbouring products, and fp32): ETA for K <= 1024.  With dg and du that error of g and u,
h = silu(g) u moves by at most 1.1 |u| dg + |silu(g)| du + 1.1 dg du (|silu'| <= 1.1), and 2^-20 of itself for
the exponential and the reciprocal.  Then h rounds to bf16 (2^-8) and to its code (2^-4 of it, or 2^-10 of the
scale).  An expert's row rounds to bf16 (2^-8), the weighted sum is fp32 (2^-20 of the sum of magnitudes
covers at most 8 terms and the weights' rounding), out rounds to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import oracle
from _util import bf16_dev, bf16_host, to_dev
from moe_synth import MoeConfig, f32_to_bf16_bits
from test_gpu_serving_layer import BLOCK, TALL, block_inputs

pytestmark = pytest.mark.gpu
ETA = 2.0 ** -12.5 + 2.0 ** -14
ONE_OF_MANY = MoeConfig("block_sparse", T=40, H=656, I=144, E=24, top_k=3, block_size=32, seed=8)


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("cfg", [BLOCK, TALL, ONE_OF_MANY], ids=lambda c: c.name)
@pytest.mark.parametrize("hs_codes", [False, True])
def test_block_layer_against_64_bits(m, cfg, hs_codes):
    d = block_inputs(cfg)
    layer = m.MoeLayer.from_arrays(d, "cuda", hs_codes=hs_codes)
    b = layer.plan(cfg.T, "cuda")
    print(f"block layer {cfg.name} hs_codes={hs_codes}", flush=True)
    out = bf16_host(layer.forward(to_dev(d["logits"]), bf16_dev(d["x"]), b))

    x_codes, x_scale = oracle.quantize_blocks_fp8(oracle.bf16_bits_to_f64(d["x"]))
    assert np.array_equal(b.xq.cpu().numpy(), x_codes) and np.array_equal(b.sx.cpu().numpy(), x_scale)
    x = oracle.e4m3_to_f64(x_codes) * oracle.spread_blocks(x_scale.astype(np.float64), cfg.H)

    ids, w = oracle.route(d["logits"], cfg.top_k, True)
    rows = b.routing.inv_sorted.cpu().numpy()[: cfg.P].reshape(ids.shape)
    scale = b.sh.cpu().numpy().astype(np.float64)
    kept = oracle.e4m3_to_f64(b.hq.cpu().numpy()) * oracle.spread_blocks(scale, cfg.I)
    ref, mag, bar = np.zeros((cfg.T, cfg.H)), np.zeros((cfg.T, cfg.H)), np.zeros((cfg.T, cfg.H))
    worst_h = worst_s = 0.0
    for e in range(cfg.E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        wg, wu, wd = (oracle.fp8_block_matrix(d[k], e) for k in ("fp8_gate", "fp8_up", "fp8_down"))
        g, u = x[t] @ wg.T, x[t] @ wu.T
        dg, du = ETA * (np.abs(x[t]) @ np.abs(wg.T)), ETA * (np.abs(x[t]) @ np.abs(wu.T))
        s = oracle.silu(g)
        h = s * u
        dh = 1.1 * np.abs(u) * dg + np.abs(s) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(h)
        # the scale is the largest |h| of its block, after the rounding to bf16
        got = scale[rows[t, j]]
        amax, slack = oracle.block_amax(h), oracle.block_amax(dh + 2.0 ** -8 * (np.abs(h) + dh))
        worst_s = max(worst_s, np.max(np.abs(448 * got - amax) / (slack + 2.0 ** -22 * amax)))
        hk = kept[rows[t, j]]
        step = oracle.spread_blocks(got, cfg.I)
        h_bar = dh + (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -12) * (np.abs(h) + dh) + 2.0 ** -10 * step
        worst_h = max(worst_h, np.max(np.abs(hk - h) / h_bar))
        y, ym = hk @ wd.T, np.abs(hk) @ np.abs(wd.T)
        wt = w[t, j].astype(np.float64)[:, None]
        np.add.at(ref, t, wt * y)
        np.add.at(mag, t, wt * np.abs(y))
        np.add.at(bar, t, wt * (ETA * ym + 2.0 ** -8 * (np.abs(y) + ETA * ym)))
    bar += 2.0 ** -20 * mag
    bar += 2.0 ** -8 * (np.abs(ref) + bar)
    worst = np.max(np.abs(out - ref) / bar)
    print(f"  worst |diff|/bar: scale {worst_s:.3f}, h {worst_h:.3f}, out {worst:.3f}", flush=True)
    assert worst_s <= 1.0 and worst_h <= 1.0 and worst <= 1.0


@pytest.mark.parametrize("k", [640, 2048, 4096, 16384, 16400, 131072])
def test_row_scales_to_fp32(m, k):
    """A row's scale max |y| / 448 leaves in fp32.  A lane adds 8 squares per chunk, one after another (64
    lanes up to 2048 columns, else 256: 512 at 131072), then 8 sums join; with the division by k and eps that
    is halved by the square root; the root, the reciprocal, the product and the division by 448 follow, 2
    steps allowed for each.  (h * w is exact: 8 + 8 bits.)"""
    lanes = 64 if k <= 2048 else 256
    depth = -(-k // 8 // lanes) * 8 + 8 + 2
    rng = np.random.default_rng(k + 1)
    bits = lambda *s: f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32))
    xb, wb = bits(3, k), bits(k)
    _, y = oracle.rmsnorm(xb, wb, 1e-6)
    q, s = torch.empty((3, k), dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")
    m.moe_rmsnorm(bf16_dev(xb), bf16_dev(wb), 1e-6, q=q, scale=s)
    want = np.abs(y).max(axis=1) / 448.0
    off = np.abs(s.cpu().numpy().astype(np.float64) - want) / want
    print(f"  k={k} worst {off.max() * 2 ** 24:.2f} of {depth / 2 + 8} steps of 2^-24", flush=True)
    assert (off <= (depth / 2 + 8) * 2.0 ** -24).all()


@pytest.mark.parametrize("k", [256, 4096, 16400])
def test_norm_of_rows_at_the_ends_of_the_fp32_range(m, k):
    """As the header states them: squares that pass fp32 give zeros, squares that underflow without eps give
    infinities of h's sign (NaN where h is zero), and with eps the exact value."""
    h = torch.full((3, k), 2.0 ** 70, device="cuda")
    h[1] = 2.0 ** -80
    h[1, ::2] *= -1
    h[2] = 2.0 ** -80
    h[2, 5] = 0.0
    h, w = h.bfloat16(), torch.ones(k, dtype=torch.bfloat16, device="cuda")
    y = m.moe_rmsnorm(h, w, 0.0)
    assert (y[0] == 0).all() and torch.equal(y[1], torch.sign(h[1]) * float("inf"))
    assert y[2, 5].isnan() and y[2].isinf().sum() == k - 1
    y = m.moe_rmsnorm(h, w, 2.0 ** -20)
    assert (y[0] == 0).all() and torch.equal(y[1:], h[1:] * 2.0 ** 10)
