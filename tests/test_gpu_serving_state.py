"""What the serving paths keep between calls, on the GPU: codes, weights and workspaces belong to the call
that they are used in."""
import pytest
import torch

import oracle
from _util import assert_close_rows, bf16_dev, bf16_host, to_dev
from moe_synth import MoeConfig, make_inputs
from test_gpu_serving_layer import BLOCK, block_inputs

pytestmark = pytest.mark.gpu
FEW = MoeConfig("few_state", T=6, H=512, I=256, E=16, top_k=4, block_size=16, group_size=64)


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


@pytest.mark.parametrize("weights", ["fp8", "fp8_block"])
def test_codes_of_a_norm_outlast_other_batches(m, weights):
    """norm_stage(x1), forward(x2), forward(y1, x_quantized=True): the last is the answer for x1, eagerly and
    where the forward of x2 is a graph that was captured before or after the norm."""
    d = block_inputs(BLOCK) if weights == "fp8_block" else make_inputs(BLOCK.with_(weights="fp8"))
    layer = m.MoeLayer.from_arrays(d, "cuda")
    b = layer.plan(BLOCK.T, "cuda")
    logits = to_dev(d["logits"])
    x1, x2 = bf16_dev(d["x"]), torch.randn((BLOCK.T, BLOCK.H), device="cuda").bfloat16()
    nw = torch.ones(BLOCK.H, dtype=torch.bfloat16, device="cuda")
    plain = layer.forward(logits, x2, b).clone()
    early = torch.cuda.CUDAGraph()
    with torch.cuda.graph(early):
        layer.forward(logits, x2, b)
    y = layer.norm_stage(x1, nw, b)
    want = layer.forward(logits, y, b, x_quantized=True).clone()
    assert not torch.equal(want, plain)
    late = torch.cuda.CUDAGraph()
    with torch.cuda.graph(late):
        layer.forward(logits, x2, b)
    for other in (lambda: layer.forward(logits, x2, b), early.replay, late.replay, early.replay):
        other()
        torch.cuda.synchronize()
        assert torch.equal(b.out, plain)
        assert torch.equal(layer.forward(logits, y, b, x_quantized=True), want)
    with pytest.raises(ValueError, match="norm_stage"):
        layer.forward(logits, x2, b, x_quantized=True)


@pytest.mark.parametrize("weights", ["bf16", "int4_gptq"])
def test_few_tokens_layer_follows_replaced_weights(m, weights):
    """A weight object with other tensors, and another weight object: the answer of a layer made of them."""
    first, second = (make_inputs(FEW.with_(weights=weights, seed=s)) for s in (1, 2))
    layer, other = (m.MoeLayer.from_arrays(d, "cuda", few_tokens=True) for d in (first, second))
    b = layer.plan(FEW.T, "cuda")
    args = to_dev(first["logits"]), bf16_dev(first["x"])
    before = layer.forward(*args, b).clone()
    want = other.forward(*args, other.plan(FEW.T, "cuda")).clone()
    assert not torch.equal(before, want)
    kept = [dict(vars(w)) for w in (layer.gate, layer.up, layer.down)]
    for mine, its in ((layer.gate, other.gate), (layer.up, other.up), (layer.down, other.down)):
        for name, t in vars(its).items():
            setattr(mine, name, t)
    assert torch.equal(layer.forward(*args, b), want)
    for w, tensors in zip((layer.gate, layer.up, layer.down), kept):
        for name, t in tensors.items():
            setattr(w, name, t)
    assert torch.equal(layer.forward(*args, b), before)
    layer.gate, layer.up, layer.down = other.gate, other.up, other.down
    assert torch.equal(layer.forward(*args, b), want)


@pytest.mark.parametrize("kw", [dict(weights="int4_gptq"), dict(H=256, I=128, E=40, top_k=33)],
                         ids=["int4_down_group", "top_k_33"])
def test_few_tokens_layer_outside_the_form_runs_its_stages(m, kw):
    """few_tokens=True on a layer that moe_few_tokens refuses: the stages, within the layer's bar."""
    cfg = FEW.with_(**kw)
    d = make_inputs(cfg)
    if "weights" in kw:                # gate and up in groups of 64, down in groups of 128
        d["down"] = make_inputs(cfg.with_(group_size=128))["down"]
    layer = m.MoeLayer.from_arrays(d, "cuda", few_tokens=True)
    assert not m.few_tokens_supported(layer.gate, layer.up, layer.down, cfg.top_k)
    b = layer.plan(cfg.T, "cuda")
    assert b.few is None
    nw = torch.ones(cfg.H, dtype=torch.bfloat16, device="cuda")
    out = layer.forward(to_dev(d["logits"]), bf16_dev(d["x"]), b)
    assert_close_rows(bf16_host(out), oracle.moe_layer(d)["out"], 2e-2, "stages")
    y = layer.norm_stage(bf16_dev(d["x"]), nw, b)
    out = layer.forward(to_dev(d["logits"]), y, b, x_quantized=True).clone()
    assert torch.equal(out, layer.forward(to_dev(d["logits"]), y, b))


def test_new_workspaces_serve_another_stream_at_once(m):
    """Buffers made while the current stream is busy and used on another one, which waits for nothing: their
    memory held other bytes before, so their zero counters must have been written by then."""
    layers = [(cfg, make_inputs(cfg)) for cfg in (FEW, MoeConfig("split", T=96, H=1024, I=512, E=4, top_k=2, block_size=32))]
    for cfg, d in layers:
        layer = m.MoeLayer.from_arrays(d, "cuda", few_tokens=True)
        args = to_dev(d["logits"]), bf16_dev(d["x"])
        b = layer.plan(cfg.T, "cuda")
        want = layer.forward(*args, b).clone()
        for t in (b.ws, b.few.workspace if b.few is not None else b.ws):
            t.fill_(255)               # what the allocator hands out next
        del b
        a = torch.randn((4096, 4096), device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(30):
            a = a @ a
            a /= a.abs().max()
        b = layer.plan(cfg.T, "cuda")
        with torch.cuda.stream(side):
            got = layer.forward(*args, b)
        side.synchronize()
        assert torch.equal(got, want)
        torch.cuda.synchronize()


@pytest.mark.parametrize("weights", ["bf16", "int4_gptq"])
def test_layers_share_buffers(m, weights):
    """Layers of one size in turn on the buffers of the first, as a model's layers run: each the answer of its
    own weights, renormalisation and path (the third has LoRA tables and runs its stages)."""
    lora = dict(lora_rank=16, lora_max_rank=32)
    made = []
    for seed, few, kw in ((1, True, {}), (2, True, dict(renormalize=False)), (3, False, lora), (4, False, {})):
        d = make_inputs(FEW.with_(weights=weights, seed=seed, **kw))
        layer = m.MoeLayer.from_arrays(d, "cuda", few_tokens=few)
        args = to_dev(d["logits"]), bf16_dev(d["x"])
        made.append((layer, args, layer.forward(*args, layer.plan(FEW.T, "cuda")).clone()))
    b = made[0][0].plan(FEW.T, "cuda")
    rank = made[2][0].plan(FEW.T, "cuda")
    b.xa = rank.xa                     # the LoRA scratch, which the first layer does not plan
    small = made[0][0].plan(2, "cuda")
    for _ in range(3):
        for layer, args, want in made:
            assert torch.equal(layer.forward(*args, b), want)
        layer, args, _ = made[1]
        got = layer.forward(args[0][:2].contiguous(), args[1][:2], small)
        assert torch.equal(got, m.moe_few_tokens(m.few_tokens_plan(layer.gate, layer.up, layer.down, FEW.top_k, 2, False),
                                                 args[0][:2].contiguous(), args[1][:2])[0])
