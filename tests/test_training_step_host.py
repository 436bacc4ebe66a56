"""Refusals of the layer's training step, CPU side: what a later call of the step would refuse is refused before the first
one, so that no gradient holds a batch that the others do not."""
import pytest
import torch

import mixture_experts_routed_route_amd as m

T, H, I, E, K, BS = 8, 64, 32, 4, 2, 16


def bf(*shape, device="cpu"):
    return torch.zeros(shape, dtype=torch.bfloat16, device=device)


def layer(**kw):
    w = lambda *s: m.Bf16Weight(bf(*s))
    return m.MoeLayer(E, H, I, K, BS, w(E, I, H), w(E, I, H), w(E, H, I), **kw)


def unaligned(*shape):
    n = torch.Size(shape).numel()
    t = torch.zeros(n + 8, dtype=torch.float32)
    at = next(i for i in range(1, 8) if (t.data_ptr() + 4 * i) % 16)
    return t[at:at + n].view(shape)


def ready(a):
    """Buffers as they stand between a forward and its backward."""
    b = a.train_plan(T, "cpu")
    b.forward_done, b.forward_of = True, a
    return b


def sums(dtype=torch.float32):
    return [torch.full(s, 3.0, dtype=dtype) for s in ((E, I, H), (E, I, H), (E, H, I))]


def refused(a, b, what, d_out=None, x=None, logits=None, grads=None):
    grads = sums() if grads is None else grads
    before = [g.clone() if g.device.type == "cpu" else None for g in grads]
    with pytest.raises(ValueError, match=what):
        a.train_backward(bf(T, H) if d_out is None else d_out, bf(T, H) if x is None else x, b, logits, grads=grads,
                         accumulate=True)
    assert b.forward_done   # the step can still be made
    assert all(c is None or torch.equal(g, c) for g, c in zip(grads, before))


@pytest.mark.parametrize("x", [bf(T, H).float(), bf(H, T).t(), bf(T, H, device="meta"), bf(T, H + 8)[:, :H], bf(T + 1, H)])
def test_x(x):
    a = layer()
    refused(a, ready(a), "train_backward: x ", x=x)


@pytest.mark.parametrize("d_out", [bf(T, H, device="meta"), bf(H, T).t(), bf(T, H).half()])
def test_d_out(d_out):
    a = layer()
    refused(a, ready(a), "train_backward: d_out ", d_out=d_out)


@pytest.mark.parametrize("logits", [torch.zeros(T, E + 1), torch.zeros(T - 1, E), bf(T, E), torch.zeros(E, T).t(),
                                    torch.zeros(T, E, device="meta"), unaligned(T, E)])
def test_logits(logits):
    a = layer(renormalize=False)
    refused(a, ready(a), "train_backward: logits ", logits=logits)


def test_logits_that_are_not_read():
    """With renormalised weights the logits are not an operand, whatever is passed: the step goes on to its first call."""
    a = layer()
    with pytest.raises(ValueError, match="HIP device"):
        a.train_backward(bf(T, H), bf(T, H), ready(a), torch.zeros(1), grads=sums(), accumulate=True)


@pytest.mark.parametrize("which", range(3))
def test_grads_of_another_device_or_alignment(which):
    a = layer()
    for wrong in (torch.zeros(sums()[which].shape, device="meta"), unaligned(*sums()[which].shape)):
        g = sums()
        g[which] = wrong
        refused(a, ready(a), "grads", grads=g)


@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_weights(name):
    """Weights that another type or shape took the place of after the forward."""
    a = layer()
    b = ready(a)
    w = getattr(a, name)
    for other in (bf(E, I, H + 8), torch.zeros(w.shape), bf(*w.shape, device="meta")):
        setattr(a, name, m.Bf16Weight(other))
        refused(a, b, "grads|weights")
    setattr(a, name, m.Fp8Weight(torch.zeros(w.shape, dtype=torch.uint8), torch.zeros(w.shape[:2])))
    refused(a, b, "bf16 weights")


# ------------------------------------------------------------------ memory that a step writes before it has read it all
def at(t, shape, dtype=torch.bfloat16, byte=0):
    """A tensor over ``t``'s memory from ``byte`` on."""
    size = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    return t.view(-1).view(torch.uint8)[byte:byte + size].view(dtype).view(shape)


def test_grads_over_each_other():
    """gate and up have one shape: one tensor for both would hold their sum, or the later one."""
    a = layer()
    g = sums()
    refused(a, ready(a), "grads", grads=[g[0], g[0], g[2]])
    both = torch.full((E * I * H + 64,), 3.0)
    refused(a, ready(a), "grads", grads=[both[:-64].view(E, I, H), both[64:].view(E, I, H), g[2]])


@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_grads_over_operands(name):
    a = layer()
    b = ready(a)
    which = ["gate", "up", "down"].index(name)
    g = sums()
    g[which] = getattr(a, name).w
    refused(a, b, "grads", grads=g)
    room = bf(E * I * H)
    g[which] = room.view(g[which].shape)
    refused(a, b, "grads", grads=g, x=at(room, (T, H), byte=16))
    refused(a, b, "grads", grads=g, d_out=at(room, (T, H), byte=room.numel() * 2 - T * H * 2))


@pytest.mark.parametrize("name", ["g", "u", "h", "ys"])
def test_operands_over_buffers(name):
    a = layer()
    b = ready(a)
    over = at(getattr(b, name), (T, H), byte=16)
    refused(a, b, "train_backward: x ", x=over)
    if name in ("g", "u"):   # h, ys and out are replaced after the forward's last use of x: a forward alone may take it there
        with pytest.raises(ValueError, match="train_forward: x "):
            a.train_forward(torch.zeros(T, E), over, b)
        assert b.forward_done
    if name != "ys":
        refused(a, b, "train_backward: d_out ", d_out=over)


def test_x_over_the_output():
    """The buffers' output may be the x of a forward, which replaces it at its end; its backward has no x there any more."""
    a = layer()
    b = ready(a)
    refused(a, b, "train_backward: x ", x=b.out)
    with pytest.raises(ValueError, match="HIP device"):   # past the checks
        a.train_forward(torch.zeros(T, E), b.out, b)


@pytest.mark.parametrize("name", ["out", "d_x", "ys"])
def test_gradients_in_place_of_results(name):
    """d_out in the place of the output, of the gradient of x or of the experts' outputs is read before those are written."""
    a = layer()
    b = ready(a)
    with pytest.raises(ValueError, match="HIP device"):
        a.train_backward(at(getattr(b, name), (T, H)), bf(T, H), b, grads=sums())


# ------------------------------------------------------------------ whose forward the buffers hold
def test_backward_of_another_layer():
    """Layers that share buffers: a backward after another layer's forward would take that one's activations."""
    a, c = layer(), layer()
    b = ready(a)
    refused(c, b, "another layer")
    b.forward_of = None
    refused(a, b, "another layer")
    same = m.MoeLayer(E, H, I, K, BS, *(m.Bf16Weight(w.w.view_as(w.w)) for w in (a.gate, a.up, a.down)))
    b.forward_of = a
    with pytest.raises(ValueError, match="HIP device"):   # past the checks
        same.train_backward(bf(T, H), bf(T, H), b, grads=sums())
    b.forward_done = True
    other = m.MoeLayer(E, H, I, K, BS, a.gate, a.up, a.down, renormalize=False)
    refused(other, b, "another layer", logits=torch.zeros(T, E))


@pytest.mark.parametrize("name", ["lora", "lora_gate", "lora_up"])
def test_tables(name):
    """LoRA tables are refused at every step, not by the plan alone: the buffers may be another layer's, and tables may come
    after the plan.  Left out silently, the output would be the base layer's."""
    b = layer().train_plan(T, "cpu")
    a = layer(**{name: object()})
    with pytest.raises(ValueError, match="LoRA"):
        a.train_forward(torch.zeros(T, E), bf(T, H), b)
    assert not b.forward_done
    a = layer()
    b = ready(a)
    setattr(a, name, object())
    refused(a, b, "LoRA")


def test_forward_of_other_weights():
    a = layer()
    b = a.train_plan(T, "cpu")
    a.up = m.Fp8Weight(torch.zeros((E, I, H), dtype=torch.uint8), torch.zeros((E, I)))
    with pytest.raises(ValueError, match="bf16 weights"):
        a.train_forward(torch.zeros(T, E), bf(T, H), b)


# ------------------------------------------------------------------ another device than the current one
class OnGpu1(torch.Tensor):
    """A CPU tensor that says it is on GPU 1."""
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", 1)

    def get_device(self):
        return 1


OPS = ["moe_route_align", "moe_grouped_gemm", "moe_silu_mul_dropout", "moe_combine", "moe_grouped_gemm_dgrad",
       "moe_silu_mul_backward", "moe_grouped_gemm_wgrad", "moe_route_backward"]


@pytest.fixture
def launches(monkeypatch):
    """The current device of every call of an operator, with GPU 0 current outside; no call is made."""
    import mixture_experts_routed_route_amd.layer as module
    current, seen = [0], []

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *_):
            current.pop()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    for name in OPS:
        monkeypatch.setattr(module, name, lambda *args, _name=name, **kw: seen.append((_name, current[-1])))
    return seen


def on_gpu1():
    a = layer()
    b = a.train_plan(T, "cpu")
    for w in (a.gate, a.up, a.down):
        w.w = w.w.as_subclass(OnGpu1)
    for name, t in vars(b).items():
        if isinstance(t, torch.Tensor):
            setattr(b, name, t.as_subclass(OnGpu1))
    return a, b


def test_step_on_another_device(launches):
    """Every launch of a step goes to the buffers' device, whichever is current."""
    a, b = on_gpu1()
    gpu = lambda t: t.as_subclass(OnGpu1)
    a.train_forward(gpu(torch.zeros(T, E)), gpu(bf(T, H)), b)
    assert len(launches) == 6 and {d for _, d in launches} == {1}
    launches.clear()
    a.train_backward(gpu(bf(T, H)), gpu(bf(T, H)), b, grads=[gpu(g) for g in sums()])
    assert len(launches) == 8 and {d for _, d in launches} == {1}
    assert {n for n, _ in launches} == set(OPS) - {"moe_route_align", "moe_grouped_gemm", "moe_silu_mul_dropout"}


@pytest.mark.parametrize("name", ["logits", "x", "gate", "up", "down"])
def test_forward_over_two_devices(launches, name):
    """An operand of another device than the buffers' would be read through its address on the wrong one."""
    a, b = on_gpu1()
    gpu = lambda t: t.as_subclass(OnGpu1)
    args = {"logits": gpu(torch.zeros(T, E)), "x": gpu(bf(T, H))}
    if name in args:
        args[name] = args[name].as_subclass(torch.Tensor)
    else:
        setattr(a, name, m.Bf16Weight(getattr(a, name).w.as_subclass(torch.Tensor)))
    with pytest.raises(ValueError, match=f"train_forward: {name} is on"):
        a.train_forward(args["logits"], args["x"], b)
    assert not launches
