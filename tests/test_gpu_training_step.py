"""The layer's training step after calls that it refuses: the sums hold what they held, and the step can still be made."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


def make(m, T, H, I, E, k, seed=0, renormalize=True):
    g = torch.Generator().manual_seed(seed)
    bf = lambda s, *shape: (s * torch.randn(shape, generator=g)).bfloat16().cuda()
    w = [m.Bf16Weight(bf(H ** -0.5, E, I, H)), m.Bf16Weight(bf(H ** -0.5, E, I, H)), m.Bf16Weight(bf(I ** -0.5, E, H, I))]
    return (m.MoeLayer(E, H, I, k, 16, *w, renormalize=renormalize), torch.randn((T, E), generator=g).cuda(), bf(1.0, T, H),
            bf(1.0, T, H))


def sums(layer, value=0.0):
    return tuple(torch.full(w.shape, value, device="cuda") for w in (layer.gate, layer.up, layer.down))


def test_refused_calls_add_nothing(m):
    T, H, I, E, k = 40, 72, 136, 5, 2
    layer, logits, x, d_out = make(m, T, H, I, E, k, renormalize=False)
    b = layer.train_plan(T, "cuda", dropout=0.1)
    want = sums(layer, 0.5)
    layer.train_forward(logits, x, b)
    want_x, want_l, _ = (t.clone() if isinstance(t, torch.Tensor) else t
                         for t in layer.train_backward(d_out, x, b, logits, grads=want, accumulate=True))
    total = sums(layer, 0.5)
    layer.train_forward(logits, x, b)
    for wrong in (dict(x=x.float()), dict(x=x.t().contiguous().t()), dict(x=x.cpu()), dict(logits=logits[:, 1:]),
                  dict(logits=torch.zeros((T, E + 1), device="cuda")), dict(logits=logits.double()), dict(logits=logits.cpu()),
                  dict(d_out=d_out.cpu()), dict(grads=(total[0], total[1].cpu(), total[2])),
                  dict(grads=(total[0].half(), *total[1:]))):
        args = {**dict(d_out=d_out, x=x, logits=logits, grads=total), **wrong}
        with pytest.raises(ValueError):
            layer.train_backward(args["d_out"], args["x"], b, args["logits"], grads=args["grads"], accumulate=True)
        assert all((t == 0.5).all() for t in total)
    d_x, d_l, _ = layer.train_backward(d_out, x, b, logits, grads=total, accumulate=True)
    assert torch.equal(d_x, want_x) and torch.equal(d_l, want_l)
    assert all(torch.equal(p, q) for p, q in zip(total, want))


@pytest.mark.parametrize("place", ["out", "d_x"])
def test_gradient_in_place_of_a_result(m, place):
    """d_out in the memory of the output, or of the gradient of x, gives what it gives in memory of its own."""
    T, H, I, E, k = 50, 264, 72, 6, 2
    layer, logits, x, d_out = make(m, T, H, I, E, k)
    b = layer.train_plan(T, "cuda", dropout=0.2, seed=4)
    layer.train_forward(logits, x, b)
    want_x, want_l, want = layer.train_backward(d_out, x, b)
    want_x, want_l = want_x.clone(), want_l.clone()
    layer.train_forward(logits, x, b)
    there = getattr(b, place).copy_(d_out)
    d_x, d_l, grads = layer.train_backward(there, x, b)
    assert torch.equal(d_x, want_x) and torch.equal(d_l, want_l) and all(torch.equal(p, q) for p, q in zip(grads, want))


def test_one_tensor_for_two_gradients_is_refused(m):
    layer, logits, x, d_out = make(m, 20, 72, 40, 4, 2)
    b = layer.train_plan(20, "cuda")
    layer.train_forward(logits, x, b)
    g = sums(layer, 0.5)
    with pytest.raises(ValueError, match="grads"):
        layer.train_backward(d_out, x, b, grads=(g[0], g[0], g[2]), accumulate=True)
    assert all((t == 0.5).all() for t in g)
    layer.train_backward(d_out, x, b, grads=g, accumulate=True)


def test_layers_that_share_buffers(m):
    """In turn they may; a backward after the other one's forward is refused and takes nothing from it."""
    T, H, I, E, k = 30, 72, 40, 4, 2
    (a, logits, x, d_out), (c, *_) = make(m, T, H, I, E, k), make(m, T, H, I, E, k, seed=1)
    b = a.train_plan(T, "cuda", dropout=0.2, seed=4)
    want = []
    for one in (a, c):
        one.train_forward(logits, x, b)
        want.append(one.train_backward(d_out, x, b)[2])
    a.train_forward(logits, x, b)
    c.train_forward(logits, x, b)
    with pytest.raises(ValueError, match="another layer"):
        a.train_backward(d_out, x, b)
    got = c.train_backward(d_out, x, b)[2]
    assert all(torch.equal(p, q) for p, q in zip(got, want[1]))
    a.train_forward(logits, x, b)
    again = m.MoeLayer(E, H, I, k, 16, a.gate, a.up, a.down)   # the same weights
    got = again.train_backward(d_out, x, b)[2]
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))


def test_masks_follow_rng_alone(m):
    """The steps leave seed and offset as they are: the same masks until the caller changes one of them."""
    T = 30
    layer, logits, x, d_out = make(m, T, 72, 104, 4, 2)
    b = layer.train_plan(T, "cuda", dropout=0.5, seed=4)
    first = layer.train_forward(logits, x, b).clone()
    layer.train_backward(d_out, x, b)
    assert b.rng.tolist() == [4, 0]
    assert torch.equal(layer.train_forward(logits, x, b), first)
    assert torch.equal(layer.train_forward(logits, x, layer.train_plan(T, "cuda", dropout=0.5, seed=4)), first)
    b.rng[1] += 1
    assert not torch.equal(layer.train_forward(logits, x, b), first)
    assert not torch.equal(layer.train_forward(logits, x, layer.train_plan(T, "cuda", dropout=0.5, seed=5)), first)


def test_forwards_over_one_output(m):
    """Forward passes alone on shared buffers may hand the output on in place; a backward without its x is refused."""
    T, H, I, E, k = 40, 72, 40, 4, 2
    (a, logits, x, d_out), (c, *_) = make(m, T, H, I, E, k), make(m, T, H, I, E, k, seed=1)
    b, other = a.train_plan(T, "cuda"), a.train_plan(T, "cuda")
    between = a.train_forward(logits, x, b).clone()
    want = c.train_forward(logits, between, other).clone()
    assert torch.equal(c.train_forward(logits, b.out, b), want)
    with pytest.raises(ValueError, match="x lies over"):
        c.train_backward(d_out, b.out, b)
    got, ref = c.train_backward(d_out, between, b)[2], c.train_backward(d_out, between, other)[2]
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
