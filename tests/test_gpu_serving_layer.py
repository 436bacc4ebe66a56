"""MoeLayer's serving paths: block-scaled fp8 experts, the norm in front of the layer and the two-launch
form for few tokens.  Each path equals the operators it chains bit for bit (they have their own tests
against fp64), keeps the layer's results within its bar of the oracle where the definitions agree, and
replays from a graph."""
import numpy as np
import pytest
import torch

import oracle
from _util import assert_close_rows, bf16_dev, bf16_host, bits_host, to_dev
from moe_synth import MoeConfig, make_inputs
from test_gpu_few_tokens import block_weight

pytestmark = pytest.mark.gpu
TOL = 2e-2   # the layer's bar against the oracle


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


def block_inputs(cfg):
    d = make_inputs(cfg.with_(weights="fp8"))
    rng = np.random.default_rng(cfg.seed)
    for key, N, K in (("fp8_gate", cfg.I, cfg.H), ("fp8_up", cfg.I, cfg.H), ("fp8_down", cfg.H, cfg.I)):
        d[key] = block_weight(rng, cfg.E, N, K)
    return d


BLOCK = MoeConfig("block", T=70, H=400, I=272, E=6, top_k=2, block_size=16, seed=3)
TALL = MoeConfig("block_tall", T=600, H=512, I=384, E=4, top_k=2, block_size=64, seed=4)


@pytest.mark.parametrize("cfg", [BLOCK, TALL], ids=lambda c: c.name)
@pytest.mark.parametrize("hs_codes", [False, True])
def test_block_layer_is_its_chain(m, cfg, hs_codes):
    d = block_inputs(cfg)
    layer = m.MoeLayer.from_arrays(d, "cuda", hs_codes=hs_codes)
    assert layer.fp8_block and not layer.fp8
    logits, x = to_dev(d["logits"]), bf16_dev(d["x"])
    b = layer.plan(cfg.T, "cuda")
    out = layer.forward(logits, x, b).clone()
    ids, w = m.moe_route(logits, cfg.top_k, True)
    r = m.moe_align(ids, cfg.E, cfg.block_size)
    nb = lambda n: -(-n // 128)
    xq, sx = torch.empty((cfg.T, cfg.H), dtype=torch.uint8, device="cuda"), torch.empty((cfg.T, nb(cfg.H)), device="cuda")
    m.moe_quantize_fp8_block(x, xq, sx)
    hq = torch.zeros((r.max_pad, cfg.I), dtype=torch.uint8, device="cuda")
    sh = torch.zeros((r.max_pad, nb(cfg.I)), device="cuda")
    ws = m.gemm_workspace("cuda")
    if hs_codes:
        assert b.hs.numel() == 0
        m.moe_grouped_gemm_fp8_block(0, xq, sx, layer.gate, layer.up, r, q=hq, scale=sh, workspace=ws)
    else:
        hs = m.moe_grouped_gemm_fp8_block(0, xq, sx, layer.gate, layer.up, r, workspace=ws)
        m.moe_quantize_fp8_block(hs, hq, sh, r)
    ys = m.moe_grouped_gemm_fp8_block(1, hq, sh, layer.down, None, r, workspace=ws)
    assert torch.equal(out, m.moe_combine(ys, r.inv_sorted, w))
    # against the layer without any quantisation of activations (reported: both quantisations round by up
    # to 2^-4 of an element)
    mats = [lambda e, k=k: oracle.fp8_block_matrix(d[k], e) for k in ("fp8_gate", "fp8_up", "fp8_down")]
    ref = oracle.few_tokens(d["logits"][:8], d["x"][:8], *mats, cfg.top_k)[0]
    err = np.linalg.norm(bf16_host(out)[:8] - ref, axis=1) / np.linalg.norm(ref, axis=1)
    print(f"  block layer against unquantised activations: worst row {err.max():.3f}", flush=True)


@pytest.mark.parametrize("fold", ["grouped", "gather"])
def test_block_layer_with_down_lora(m, fold):
    """The down-projection fold reads the bf16 Hs of the block-scaled gate/up; the folded rows against the
    oracle's fold of the kernel's own Hs and unfolded Ys.  Bar: a bf16 rounding (2^-8) of the sum, one of xa
    and of the product's operands carried by the fold's size, as the row-scaled layer's test has it."""
    cfg = MoeConfig("block_lora", T=90, H=512, I=256, E=8, top_k=3, block_size=32, lora_rank=16, lora_max_rank=64, seed=56)
    d = block_inputs(cfg)
    d.update({k: v for k, v in make_inputs(cfg).items() if k.startswith("lora")})
    d["lora_scale"] = (d["lora_scale"] * 20).astype(np.float32)   # a fold well above a bf16 step
    layer = m.MoeLayer.from_arrays(d, "cuda", fold=fold)
    assert layer.fp8_block and layer.lora is not None
    b = layer.plan(cfg.T, "cuda")
    layer.route_align(to_dev(d["logits"]), b)
    layer.gate_up_stage(bf16_dev(d["x"]), b)
    layer.down_stage(b)
    hs, ys0 = bits_host(b.hs), bits_host(b.ys)
    layer.lora_fold(b)
    ys = bf16_host(b.ys)
    al = oracle.align(oracle.route(d["logits"], cfg.top_k, True)[0], cfg.E, cfg.block_size)
    real = np.flatnonzero(al["sorted_ids"] < cfg.P)
    hs_f = np.zeros(hs.shape)
    hs_f[real] = oracle.bf16_bits_to_f64(hs[real])
    base = np.zeros(ys0.shape)
    base[real] = oracle.bf16_bits_to_f64(ys0[real])
    want = oracle.lora_fold(base, hs_f, oracle.moe_oracle._lora_tables(d), al, cfg.top_k)
    fold_part = want - base
    moved = np.linalg.norm(fold_part[real], axis=1) > 0
    assert moved.any()
    # 2^-8 of the result, and of the fold twice: xa's rounding and its own
    bar = 2.0 ** -8 * np.linalg.norm(want[real], axis=1) + 2.0 ** -7 * np.linalg.norm(fold_part[real], axis=1)
    err = np.linalg.norm(ys[real] - want[real], axis=1)
    print(f"  fold: worst row over its bar {np.max(err / np.maximum(bar, 1e-30)):.3f}", flush=True)
    assert (err <= bar).all()
    out = layer.forward(to_dev(d["logits"]), bf16_dev(d["x"]), b)
    assert torch.equal(out, layer.combine(b))


@pytest.mark.parametrize("weights", ["bf16", "fp8", "fp8_block"])
def test_norm_stage_feeds_the_layer(m, weights):
    """norm_stage then forward(x_quantized=True) = the norm, then the layer on codes of the unrounded
    norm; the bf16 rows go to the router and, with bf16 weights, to the layer."""
    cfg = BLOCK.with_(weights="fp8" if weights == "fp8_block" else weights)
    d = block_inputs(cfg) if weights == "fp8_block" else make_inputs(cfg)
    layer = m.MoeLayer.from_arrays(d, "cuda")
    logits, x = to_dev(d["logits"]), bf16_dev(d["x"])
    res = torch.randn_like(x)
    nw = (1 + 0.1 * torch.randn(cfg.H, device="cuda")).bfloat16()
    b = layer.plan(cfg.T, "cuda")
    r0 = res.clone()
    y = layer.norm_stage(x, nw, b, 1e-5, residual=res)
    out = layer.forward(logits, y, b, x_quantized=True).clone()
    h, want = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty((cfg.T, cfg.H), dtype=torch.uint8, device="cuda")
    s = torch.empty((cfg.T,) if weights == "fp8" else (cfg.T, 4), device="cuda")
    m.moe_rmsnorm(x, nw, 1e-5, residual=r0, residual_out=h, y=want, q=q, scale=s)
    assert torch.equal(res, h) and torch.equal(y, want)
    b2 = layer.plan(cfg.T, "cuda")
    if weights == "bf16":
        assert torch.equal(out, layer.forward(logits, want, b2))
    else:
        assert torch.equal(b.xq, q) and torch.equal(b.sx, s)
        layer.route_align(logits, b2)
        b2.xq.copy_(q)
        b2.sx.copy_(s)
        layer.experts(want, b2, x_quantized=True)
        assert torch.equal(out, layer.combine(b2))
    for bufs in (None, layer.plan(cfg.T, "cuda")):
        with pytest.raises(ValueError, match="norm_stage"):
            layer.forward(logits, y, bufs, x_quantized=True)
    with pytest.raises(ValueError, match="needs"):
        layer.norm_stage(x[:-1], nw, b)          # buffers of another token count


@pytest.mark.parametrize("kw", [{}, {"hs_codes": True}, {"few_tokens": True}])
def test_no_tokens(m, kw):
    d = block_inputs(BLOCK)
    layer = m.MoeLayer.from_arrays(d, "cuda", **kw)
    b = layer.plan(0, "cuda")
    y = layer.norm_stage(torch.empty((0, BLOCK.H), dtype=torch.bfloat16, device="cuda"),
                         torch.ones(BLOCK.H, dtype=torch.bfloat16, device="cuda"), b)
    out = layer.forward(torch.empty((0, BLOCK.E), device="cuda"), y, b, x_quantized=True)
    torch.cuda.synchronize()
    assert out.shape == (0, BLOCK.H)


@pytest.mark.parametrize("weights", ["bf16", "int4_gptq"])
def test_few_tokens_layer(m, weights):
    """Batches of at most 32 tokens take the two-launch form, larger ones the stages; both within the
    layer's bar of the oracle, and buffers (ids, weights, out) filled the same way."""
    for T in (1, 32, 33):
        cfg = MoeConfig("few", T=T, H=512, I=256, E=16, top_k=4, block_size=16, weights=weights, group_size=64, seed=T)
        d = make_inputs(cfg)
        layer = m.MoeLayer.from_arrays(d, "cuda", few_tokens=True)
        b = layer.plan(T, "cuda")
        assert (b.few is not None) == (T <= 32)
        logits, x = to_dev(d["logits"]), bf16_dev(d["x"])
        out = layer.forward(logits, x, b)
        ref = oracle.moe_layer(d)
        assert np.array_equal(b.ids.cpu().numpy(), ref["ids"]) and np.array_equal(b.w.cpu().numpy(), ref["w"])
        assert_close_rows(bf16_host(out), ref["out"], TOL, f"few {weights} T={T}")
        if T <= 32:
            assert torch.equal(out, m.moe_few_tokens(m.few_tokens_plan(layer.gate, layer.up, layer.down, 4, T), logits, x)[0])


def test_norm_and_few_tokens_replay_from_a_graph(m):
    cfg = MoeConfig("few_graph", T=6, H=1024, I=512, E=16, top_k=4, block_size=16, seed=9)
    d = make_inputs(cfg)
    layer = m.MoeLayer.from_arrays(d, "cuda", few_tokens=True)
    b = layer.plan(6, "cuda")
    wr = (torch.randn((16, 1024), device="cuda") * 0.05)
    nw = torch.ones(1024, dtype=torch.bfloat16, device="cuda")
    xs = [torch.randn((6, 1024), device="cuda").bfloat16() for _ in range(3)]
    x, res, logits = xs[0].clone(), torch.zeros((6, 1024), dtype=torch.bfloat16, device="cuda"), torch.empty((6, 16), device="cuda")

    def step():
        y = layer.norm_stage(x, nw, b, residual=res)
        torch.matmul(y.float(), wr.t(), out=logits)
        return layer.forward(logits, y, b)
    want = []
    for v in xs:
        x.copy_(v)
        res.zero_()
        want.append(step().clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in (1, 2, 0, 1):
        x.copy_(xs[i])
        res.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, want[i])


def test_two_streams_at_once(m):
    """Buffers (plans) of their own on two streams, calls interleaved without waiting: as one at a time."""
    layers, ins, bufs, want = [], [], [], []
    for seed, kw in ((31, {"few_tokens": True}), (32, {"few_tokens": True}), (33, {})):
        cfg = BLOCK.with_(T=12, seed=seed)
        d = block_inputs(cfg)
        layer = m.MoeLayer.from_arrays(d, "cuda", **kw)
        b = layer.plan(cfg.T, "cuda")
        args = to_dev(d["logits"]), bf16_dev(d["x"])
        layers.append(layer), ins.append(args), bufs.append(b)
        want.append(layer.forward(*args, b).clone())
    torch.cuda.synchronize()
    for b in bufs:
        b.out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(25):
        for s, layer, args, b in zip(streams, layers, ins, bufs):
            with torch.cuda.stream(s):
                layer.forward(*args, b)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        assert torch.equal(b.out, w)
