"""What the serving paths keep between calls, on the GPU: codes, weights and workspaces belong to the call
that they are used in."""
import pytest
import torch

from _util import bf16_dev, to_dev
from moe_synth import make_inputs
from test_gpu_serving_layer import BLOCK, block_inputs

pytestmark = pytest.mark.gpu


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
