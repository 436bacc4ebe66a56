"""SiLU * up and its backward on the widest row that their entry points take, 2^31 - 8 columns: elementwise outputs are
those of the same columns in a short row, bit for bit, and the row's sum is exact on values whose sum is."""
import pytest
import torch

pytestmark = pytest.mark.gpu
N = 2**31 - 8


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


def test_widest_row(m):
    g = torch.Generator(device="cuda").manual_seed(7)
    parts = [slice(0, 4096), slice(2**30 - 2048, 2**30 + 2048), slice(N - 8192, N)]
    guard = 8192
    rows = []
    for size in (2.0, 1.0, 0.1):   # gate, up, d: 4.3 GB each, with room on both sides that stays as it is
        t = torch.zeros(N + 2 * guard, dtype=torch.bfloat16, device="cuda")
        t[:guard], t[-guard:] = 7.5, 7.5
        for s in parts:
            n = s.stop - s.start
            t[guard + s.start:guard + s.stop] = (size * torch.randn(n, generator=g, device="cuda")).bfloat16()
        rows.append(t)
    gate, up, d = (t[guard:-guard].view(1, N) for t in rows)
    w, dw = torch.full((1,), 0.75, device="cuda"), torch.full((1,), -3.0, device="cuda")
    want = [[v.clone() for v in m.moe_silu_mul_backward(*(t[:, s].contiguous() for t in (gate, up, d)), w)] for s in parts]
    h = [m.moe_silu_mul_dropout(*(t[:, s].contiguous() for t in (gate, up))) for s in parts]
    print("widest row: forward", flush=True)
    out = torch.empty_like(gate)
    m.moe_silu_mul_dropout(gate, up, out=out)
    for s, one in zip(parts, h):
        assert torch.equal(out[:, s], one)
    del out
    print("widest row: backward, in place", flush=True)
    got = m.moe_silu_mul_backward(gate, up, d, w, d_gate=gate, d_up=up, h_weighted=d, d_topk_w=dw)
    for s, one in zip(parts, want):
        for a, b in zip(got[:3], one):
            assert torch.equal(a[:, s], b)
    # zeros everywhere else: the row's sum is that of the parts, added in another order (16384 terms of up to 2^-24 of the
    # sum of magnitudes each, which the parts' values bound)
    total = sum(one[3].item() for one in want)
    size = sum((t[2].double() / 0.75).abs().sum().item() for t in want)   # |h|; |d| stays below 1
    assert abs(dw.item() - total) <= 2 * 16384 * 2.0 ** -24 * size
    for t in rows:
        assert (t[:guard] == 7.5).all() and (t[-guard:] == 7.5).all()
