"""MoeLayer's serving paths, CPU side: which buffers and which path a call takes.  The kernels' wrappers are
replaced by stand-ins that note what they are given; the layer's own code runs as it is."""
import pytest
import torch

import mixture_experts_routed_route_amd as m
from mixture_experts_routed_route_amd import layer as layer_module

T, H, I, E, K = 5, 256, 128, 4, 2


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def fp8_layer(kind, **kw):
    def w(n, k):
        scales = torch.zeros(E, n) if kind == "fp8" else torch.zeros(E, -(-n // 128), -(-k // 128))
        return (m.Fp8Weight if kind == "fp8" else m.Fp8BlockWeight)(u8(E, n, k), scales)
    return m.MoeLayer(E, H, I, K, 16, w(I, H), w(I, H), w(H, I), **kw)


@pytest.fixture
def calls(monkeypatch):
    """Stand-ins: a quantisation or norm writes its x's first value into the codes; a gate/up product notes
    the codes that it is given."""
    seen = []

    def norm(x, weight, eps=1e-6, residual=None, residual_out=None, y=None, q=None, scale=None):
        y.copy_(x)
        if q is not None:
            q.fill_(int(x[0, 0]))
            scale.fill_(float(x[0, 0]))
        return y

    def quantize(x, q, scale, routing=None):
        if routing is None:            # (Hs in the sorted layout is not computed here)
            q.fill_(int(x[0, 0]))
            scale.fill_(float(x[0, 0]))

    def gemm(op, a, a_scale, *args, **kw):
        if op == m.MOE_OP_GATE_UP_SILU:
            assert (a == a[0, 0]).all() and (a_scale == float(a[0, 0])).all()
            seen.append(int(a[0, 0]))

    for name, f in (("moe_rmsnorm", norm), ("moe_quantize_fp8", quantize), ("moe_quantize_fp8_block", quantize),
                    ("moe_grouped_gemm_fp8", gemm), ("moe_grouped_gemm_fp8_block", gemm),
                    ("moe_route_align", lambda *a: None), ("moe_combine", lambda ys, inv, w, out=None: out)):
        monkeypatch.setattr(layer_module, name, f)
    return seen


@pytest.mark.parametrize("kind", ["fp8", "fp8_block"])
def test_x_quantized_reads_the_codes_of_its_x(calls, kind):
    """The codes that forward(x_quantized=True) multiplies are those of the norm_stage output it is given,
    whatever ran on the buffers in between."""
    layer = fp8_layer(kind)
    b = layer.plan(T, "cpu")
    logits, nw = torch.zeros(T, E), bf(H)
    layer.forward(logits, bf(T, H) + 9, b)                      # before any norm_stage
    y = layer.norm_stage(bf(T, H) + 1, nw, b)
    layer.forward(logits, bf(T, H) + 2, b)                      # another batch in between
    layer.forward(logits, y, b, x_quantized=True)
    layer.forward(logits, y, b)                                 # the same rows, quantised by forward
    layer.norm_stage(bf(T, H) + 3, nw, b)
    layer.forward(logits, y, b, x_quantized=True)               # y is the buffer that norm_stage returns
    assert calls == [9, 2, 1, 1, 3]


@pytest.mark.parametrize("kind", ["fp8", "fp8_block"])
def test_x_quantized_refuses_another_x(calls, kind):
    layer = fp8_layer(kind)
    b = layer.plan(T, "cpu")
    logits = torch.zeros(T, E)
    y = layer.norm_stage(bf(T, H) + 1, bf(H), b)
    for x in (y.clone(), bf(T, H), y[:-1], b.out):
        with pytest.raises(ValueError, match="norm_stage"):
            layer.forward(logits, x, b, x_quantized=True)
        with pytest.raises(ValueError, match="norm_stage"):
            layer.experts(x, b, x_quantized=True)
    assert calls == []
    layer.forward(logits, y, b, x_quantized=True)
    assert calls == [1]


def test_a_refused_norm_leaves_the_buffers_without_codes(calls, monkeypatch):
    def refuse(*a, **kw):
        raise ValueError("moe_rmsnorm: refused")
    layer = fp8_layer("fp8_block")
    b = layer.plan(T, "cpu")
    with monkeypatch.context() as p:
        p.setattr(layer_module, "moe_rmsnorm", refuse)
        with pytest.raises(ValueError, match="refused"):
            layer.norm_stage(bf(T, H), bf(H), b)
    with pytest.raises(ValueError, match="norm_stage"):
        layer.forward(torch.zeros(T, E), bf(T, H), b, x_quantized=True)
    assert b.xn is None and b.pq is None


def test_x_quantized_refuses_a_norm_without_codes(calls, monkeypatch):
    """norm_stage of a layer that runs the two-launch form writes no codes: neither garbage nor an earlier
    norm's codes may be read for its rows."""
    form, stages = fp8_layer("fp8_block", few_tokens=True), fp8_layer("fp8_block")
    monkeypatch.setattr(m.MoeLayer, "few_plan", lambda self, b: object() if self is form else None)
    b = stages.plan(T, "cpu")
    logits, nw = torch.zeros(T, E), bf(H)
    y = form.norm_stage(bf(T, H) + 1, nw, b)
    with pytest.raises(ValueError, match="no codes"):
        stages.forward(logits, y, b, x_quantized=True)
    y = stages.norm_stage(bf(T, H) + 2, nw, b)
    stages.forward(logits, y, b, x_quantized=True)
    y = form.norm_stage(bf(T, H) + 3, nw, b)
    with pytest.raises(ValueError, match="no codes"):
        stages.forward(logits, y, b, x_quantized=True)
    stages.forward(logits, y, b)
    assert calls == [2, 3]
