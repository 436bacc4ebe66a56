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
