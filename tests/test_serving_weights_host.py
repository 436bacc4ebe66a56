"""Expert weights of the serving operators, CPU side: the addresses and devices that reach the library.
Tensors that claim to be on a GPU stand for device memory; the launches are noted, not made."""
import ctypes

import pytest
import torch

import mixture_experts_routed_route_amd as m
from mixture_experts_routed_route_amd import serving
from mixture_experts_routed_route_amd._lib import MoeWeight


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on GPU ``index``."""
    index = 0
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


class OnOther(OnGpu):
    index = 1


def gpu(t, cls=OnGpu):
    return t.as_subclass(cls)


def bf(*shape):
    return gpu(torch.zeros(shape, dtype=torch.bfloat16))


E, H, I, K = 4, 64, 32, 2


def block(cls=OnGpu, n=I, k=H, scales_cls=None):
    return m.Fp8BlockWeight(gpu(torch.zeros((E, n, k), dtype=torch.uint8), cls),
                            gpu(torch.zeros((E, -(-n // 128), -(-k // 128))), scales_cls or cls))


@pytest.fixture
def launches(monkeypatch):
    seen = []
    monkeypatch.setattr(serving, "_launch", lambda name, index, *args: seen.append((name, index, args)))
    return seen


@pytest.fixture
def few(launches, monkeypatch):
    """A plan of bf16 weights and a call of it that gives the three data addresses."""
    monkeypatch.setattr(serving, "_zeroed", lambda n, device, wait: gpu(torch.zeros(n, dtype=torch.uint8)))
    plan = m.few_tokens_plan(m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, H, I)), K, 4)
    args = (gpu(torch.empty((3, E))), bf(3, H), gpu(torch.empty((3, K), dtype=torch.int32)),
            gpu(torch.empty((3, K))), bf(3, H))

    def call():
        m.moe_few_tokens(plan, *args)
        return [ctypes.cast(ref, ctypes.POINTER(MoeWeight)).contents.data for ref in launches.pop()[2][2:5]]
    return plan, call


def test_few_tokens_follows_replaced_weights(few):
    """A weight object that gets another tensor, or a tensor that gets other memory: the next call reads that."""
    plan, call = few
    old = plan.gate.w
    assert call() == [plan.gate.w.data_ptr(), plan.up.w.data_ptr(), plan.down.w.data_ptr()]
    plan.gate.w = bf(E, I, H)
    assert plan.gate.w.data_ptr() != old.data_ptr() and call()[0] == plan.gate.w.data_ptr()
    kept = plan.up.w.data
    plan.up.w.data = bf(E, I, H)
    assert kept.data_ptr() != plan.up.w.data_ptr() and call()[1] == plan.up.w.data_ptr()
    down = m.Bf16Weight(bf(E, H, I))
    plan.use(plan.gate, plan.up, down)
    assert call() == [plan.gate.w.data_ptr(), plan.up.w.data_ptr(), down.w.data_ptr()]


def test_few_tokens_refuses_replacements_it_cannot_read(few):
    plan, call = few
    want = call()
    before = (plan.gate, plan.up, plan.down)
    for bad, word in [(m.Bf16Weight(bf(E, I, H + 8)), "up"), (m.Bf16Weight(bf(E, I, H).transpose(1, 2)), "up"),
                      (m.Bf16Weight(gpu(torch.empty((E, I, H), dtype=torch.bfloat16), OnOther)), "not on")]:
        with pytest.raises(ValueError, match=word):
            plan.use(bad, plan.up, plan.down)
        assert (plan.gate, plan.up, plan.down) == before and call() == want
    wide = [m.Bf16Weight(bf(*s)) for s in ((E, I, H + 8), (E, I, H + 8), (E, H + 8, I))]
    with pytest.raises(ValueError, match="made for"):
        plan.use(*wide)
    plan.gate.w = bf(E, I + 8, H)
    for _ in range(2):                 # refused as long as it is there
        with pytest.raises(ValueError, match="up"):
            call()


def test_layer_hands_replaced_weights_to_its_few_token_plan(few, monkeypatch):
    plan, _ = few
    layer = m.MoeLayer(E, H, I, K, 16, plan.gate, plan.up, plan.down, few_tokens=True)
    b = m.layer.Buffers(3, None, None, None, None, None, None, None, None, few=plan, few_of=layer)
    monkeypatch.setattr(m.layer, "moe_few_tokens", lambda p, *a: (p,))
    assert layer.forward(None, None, b) is plan and plan.renormalize
    layer.down = m.Bf16Weight(bf(E, H, I))
    layer.renormalize = False
    layer.forward(None, None, b)
    assert plan.down is layer.down and plan.tensors[2][2] is layer.down.w and not plan.renormalize


def test_layers_share_buffers(few, monkeypatch):
    """Buffers that one layer planned, used by others of its size: each with its own weights and its own path."""
    plan, _ = few

    def layer(**kw):
        return m.MoeLayer(E, H, I, K, 16, m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, H, I)), **kw)
    first = m.MoeLayer(E, H, I, K, 16, plan.gate, plan.up, plan.down, few_tokens=True)
    second, third, stages = layer(few_tokens=True), layer(few_tokens=True, renormalize=False), layer()
    b = m.layer.Buffers(3, None, None, None, None, None, None, None, None, few=plan, few_of=first)
    monkeypatch.setattr(m.layer, "moe_few_tokens", lambda p, *a: ((p.gate, p.up, p.down, p.renormalize, p.workspace),))
    for _ in range(2):
        for l in (first, second, third):
            assert l.forward(None, None, b) == (l.gate, l.up, l.down, l.renormalize, plan.workspace)
    assert b.few is plan is first.few_plan(b) and plan.gate is first.gate
    kept = second.few_plan(b)
    structs = kept.structs
    other = m.layer.Buffers(2, None, None, None, None, None, None, None, None, few_of=first, few=m.serving.FewTokensPlan(
        first.gate, first.up, first.down, E, H, I, K, 2, True, gpu(torch.zeros(1 << 16, dtype=torch.uint8))))
    assert second.few_plan(other) is kept and kept.workspace is other.few.workspace and kept.max_tokens == 2
    assert second.few_plan(b) is kept and kept.workspace is plan.workspace and kept.max_tokens == plan.max_tokens
    assert kept.structs is structs                # checked once, not call by call
    assert stages.few_plan(b) is None             # a layer that did not ask for the form (it may have LoRA tables)
    short = m.layer.Buffers(3, None, None, None, None, None, None, None, None, few_of=first, few=m.serving.FewTokensPlan(
        first.gate, first.up, first.down, E, H, I, K, 3, True, gpu(torch.zeros(8200, dtype=torch.uint8))))
    assert second.few_plan(short) is None and not m.few_tokens_fit(second.gate, second.up, second.down, K, 3, short.few.workspace)
    second.down = m.Fp8Weight(torch.empty(1), torch.empty(1))
    assert second.few_plan(b) is None             # nor one that the form does not take any more


def test_gemm_fp8_block_refuses_weights_of_another_device(launches):
    """Codes or scales, gate or up: a kernel on the activations' device would read the other device's memory."""
    r = m.Routing.allocate(8, K, E, 16, "cpu")
    r = m.Routing(*[gpu(v) if isinstance(v, torch.Tensor) else v for v in vars(r).values()])
    n = 128

    def call(w0, w1):
        m.moe_grouped_gemm_fp8_block(m.MOE_OP_GATE_UP_SILU, gpu(torch.zeros((4, n), dtype=torch.uint8)),
                                     gpu(torch.zeros((4, 1))), w0, w1, r, out=bf(r.max_pad, n))
    call(block(n=n, k=n), block(n=n, k=n))
    assert len(launches) == 1 and launches[0][:2] == ("moe_grouped_gemm_fp8_block", 0)
    for kw in (dict(cls=OnOther), dict(scales_cls=OnOther)):
        for w0, w1 in ((block(n=n, k=n, **kw), block(n=n, k=n)), (block(n=n, k=n), block(n=n, k=n, **kw))):
            with pytest.raises(ValueError, match="a weight is on cuda:1"):
                call(w0, w1)
    assert len(launches) == 1


@pytest.mark.parametrize("capturing", [False, True])
@pytest.mark.parametrize("make", [lambda: m.gemm_workspace("cuda"), lambda: m.few_tokens_plan(
    m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, H, I)), K, 4).workspace], ids=["gemm", "few"])
def test_workspaces_are_filled_before_any_stream_uses_them(monkeypatch, capturing, make):
    """Their zero counters are waited for (a call on another stream would not wait); a capture records the fill."""
    import contextlib
    log, zeros = [], torch.zeros

    class Stream:
        def synchronize(self):
            log.append("wait")

    def filled(n, dtype=None, device=None):
        log.append("fill")
        return gpu(zeros(n, dtype=dtype))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch, "zeros", lambda n, **kw: filled(n, **kw) if kw.get("device") is not None else zeros(n, **kw))
    assert make().is_cuda
    assert log == (["fill"] if capturing else ["fill", "wait"])


def test_forward_without_buffers_waits_for_nothing(monkeypatch):
    """Its own buffers are used at once on the current stream, so it must not hold up the host."""
    made = []
    monkeypatch.setattr(m.layer, "gemm_workspace", lambda device, wait=True: made.append(wait))
    monkeypatch.setattr(m.layer, "few_tokens_plan", lambda *a: made.append(a[-1]))
    for name in ("route_align", "experts", "combine"):
        monkeypatch.setattr(m.MoeLayer, name, lambda *a, **kw: None)
    layer = m.MoeLayer(E, H, I, K, 16, m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, I, H)), m.Bf16Weight(bf(E, H, I)), few_tokens=True)
    layer.forward(torch.zeros(3, E), torch.zeros(3, H, dtype=torch.bfloat16))
    assert made == [False, False]
    layer.plan(3, "cpu")
    assert made == [False, False, True, True]
