"""Training operators on arrays that lie side by side in one allocation: the same bits as in memory of their own, and
nothing beside the results is written."""
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


def packed(*tensors):
    """Copies of the tensors without a gap between them, and their memory."""
    room = torch.cat([t.contiguous().view(-1).view(torch.uint8) for t in tensors])
    out, at = [], 0
    for t in tensors:
        n = t.numel() * t.element_size()
        out.append(room[at:at + n].view(t.dtype).view(t.shape))
        at += n
    return out, room


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_grouped_products_side_by_side(m, dtype):
    T, k, E, N, K = 70, 2, 5, 264, 136
    g = torch.Generator(device="cuda").manual_seed(1)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].int().contiguous()
    r = m.moe_align(ids, E, 16)
    dy, x, w, w1 = bf(r.max_pad, N), bf(T, K), bf(E, N, K), bf(E, N, K)
    dx, dw, base = bf(r.max_pad, K), torch.zeros((E, N, K), dtype=dtype, device="cuda"), bf(E, N, K).to(dtype)
    want = m.moe_grouped_gemm_dgrad(dy, m.Bf16Weight(w), r, dy1=dy, w1=m.Bf16Weight(w1), out=dx.clone())
    (a, b, c, d), _ = packed(dy, dx, w, w1)
    assert torch.equal(m.moe_grouped_gemm_dgrad(a, m.Bf16Weight(c), r, dy1=a, w1=m.Bf16Weight(d), out=b), want)
    assert torch.equal(a, dy) and torch.equal(c, w) and torch.equal(d, w1)
    want = m.moe_grouped_gemm_wgrad(dy, x, r, x_by_token=True, base=base, out=dw.clone())
    (a, b, c, d), _ = packed(dy, dw, base, x)
    assert torch.equal(m.moe_grouped_gemm_wgrad(a, d, r, x_by_token=True, base=c, out=b), want)
    assert torch.equal(a, dy) and torch.equal(c, base) and torch.equal(d, x)


def test_rows_side_by_side_and_in_place(m):
    g = torch.Generator(device="cuda").manual_seed(2)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    gate, up, d, w = bf(33, 520), bf(33, 520), bf(33, 520), torch.rand(36, generator=g, device="cuda")
    h = m.moe_silu_mul_dropout(gate, up)
    want = m.moe_silu_mul_backward(gate, up, d, w)
    mark = torch.full_like(gate, 7.5)
    (a, b, c, e), room = packed(mark, gate, mark, up)
    assert torch.equal(m.moe_silu_mul_dropout(b, e, out=a), h) and torch.equal(m.moe_silu_mul_dropout(b, e, out=c), h)
    assert torch.equal(b, gate) and torch.equal(e, up)
    (a, b, c, e, f, i, j, k), room = packed(gate, mark, up, mark, d, mark, w, torch.zeros_like(w))
    got = m.moe_silu_mul_backward(a, c, f, j, d_gate=b, d_up=e, h_weighted=i, d_topk_w=k)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert torch.equal(a, gate) and torch.equal(c, up) and torch.equal(f, d) and torch.equal(j, w)


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_side_by_side_and_in_place(m, renormalize):
    g = torch.Generator(device="cuda").manual_seed(3)
    for T, E, k in ((36, 12, 2), (36, 8, 8)):
        logits, dw = torch.randn((T, E), generator=g, device="cuda"), torch.randn((T, k), generator=g, device="cuda")
        ids, w = m.moe_route(logits, k, renormalize)
        lg = None if renormalize else logits
        want = m.moe_route_backward(ids, w, dw, E, lg)
        (a, b, c, e), _ = packed(w, torch.zeros_like(logits), dw, ids)
        assert torch.equal(m.moe_route_backward(e, a, c, E, lg, out=b), want)
        assert torch.equal(a, w) and torch.equal(c, dw) and torch.equal(e, ids)
        if not renormalize:
            over = logits.clone()
            assert torch.equal(m.moe_route_backward(ids, w, dw, E, over, out=over), want)
        if k == E:
            over = dw.clone()
            assert torch.equal(m.moe_route_backward(ids, w, over, E, lg, out=over), want)
