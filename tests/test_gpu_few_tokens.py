"""The layer for a few tokens against the fp64 oracle: weight types, token counts, odd sizes, expert
counts, repeated and skewed routing, workspaces, graphs and streams.

Bars.  ids and weights: bit-exact.  out: h is a sum of two bf16 values (the second rounds what the first
left, 2^-8 of h, by 2^-8 of that: 2^-16 of h) and out rounds to bf16 (half a step, 2^-8 of itself), so
|got - ref| <= 2^-8 |ref| + 2^-16 spread, plus fp32 arithmetic: a sum of n
products in any order is off by at most n 2^-24 of the sum of their magnitudes (n = max(H, I) + the
waves' and experts' sums), and the exponential and reciprocal of SiLU by 2^-20 of h.  ``spread`` and
``noise`` (oracle) carry those to the output.  The rounding of out moves a row by at most 2^-8 of its norm,
h and the arithmetic by far less than another 2^-8 of it: 2^-7."""
import numpy as np
import pytest
import torch

import oracle
from _util import bf16_dev, bf16_host, bits_host, to_dev
from moe_synth import MoeConfig, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")
    import mixture_experts_routed_route_amd as m
    m.lib()
    return m


def block_weight(rng, E, N, K):
    codes = (rng.integers(4 * 8, 11 * 8, (E, N, K)) | (rng.integers(0, 2, (E, N, K)) << 7)).astype(np.uint8)
    return {"codes": codes, "scales": rng.uniform(0.002, 0.006, (E, -(-N // 128), -(-K // 128))).astype(np.float32)}


def inputs(cfg):
    """(inputs, device weights, oracle matrices) of a case; weights "fp8_block" are drawn here."""
    import mixture_experts_routed_route_amd as m
    if cfg.weights == "fp8_block":
        d = make_inputs(cfg.with_(weights="bf16"))
        rng = np.random.default_rng(cfg.seed + 100)
        for key, N, K in (("wg", cfg.I, cfg.H), ("wu", cfg.I, cfg.H), ("wd", cfg.H, cfg.I)):
            d[key] = block_weight(rng, cfg.E, N, K)
        keys = ("wg", "wu", "wd")
        dev = [m.Fp8BlockWeight(to_dev(d[k]["codes"]), to_dev(d[k]["scales"])) for k in keys]
        mat = [lambda e, k=k: oracle.fp8_block_matrix(d[k], e) for k in keys]
        return d, dev, mat
    d = make_inputs(cfg)
    if cfg.weights == "bf16":
        keys = ("wg", "wu", "wd")
        return d, [m.Bf16Weight(bf16_dev(d[k])) for k in keys], [lambda e, k=k: oracle.expert_matrix(d[k], e) for k in keys]
    if cfg.weights == "fp8":
        keys = ("fp8_gate", "fp8_up", "fp8_down")
        dev = [m.Fp8Weight(to_dev(d[k]["codes"]), to_dev(d[k]["scales"])) for k in keys]
        return d, dev, [lambda e, k=k: oracle.fp8_expert_matrix(d[k], e) for k in keys]
    keys = ("gate", "up", "down")
    dev = [m.GptqWeight(to_dev(d[k]["qweight"]), to_dev(d[k]["scales"], dtype=torch.float16), to_dev(d[k]["qzeros"]),
                        cfg.group_size) for k in keys]
    return d, dev, [lambda e, k=k: oracle.expert_matrix(d[k], e) for k in keys]


def reference(cfg, d, mat):
    return oracle.few_tokens(d["logits"], d["x"], *mat, cfg.top_k, cfg.renormalize)


def check(cfg, got, ref):
    out, ids, w = got
    r, rids, rw, spread, noise = ref
    assert np.array_equal(ids.cpu().numpy(), rids)
    assert np.array_equal(w.cpu().numpy().view(np.uint32), rw.view(np.uint32))
    o = bf16_host(out)
    n = max(cfg.H, cfg.I) + 64 + cfg.T * cfg.top_k
    bar = 2.0 ** -8 * np.abs(r) + (2.0 ** -16 + 2.0 ** -20 + n * 2.0 ** -24) * spread + n * 2.0 ** -24 * noise
    bad = np.abs(o - r) - bar
    err = np.linalg.norm(o - r, axis=1) / np.linalg.norm(r, axis=1)
    print(f"  worst |diff|/bar {np.max(np.abs(o - r) / np.maximum(bar, 1e-300)):.3f}, worst row {err.max():.2e}", flush=True)
    assert bad.max() <= 0, f"element {np.unravel_index(bad.argmax(), bad.shape)} off by {bad.max():.3e} over its bar"
    assert err.max() <= 2.0 ** -7


def C(name, T, H, I, E, k, weights="bf16", **kw):
    return MoeConfig(name, T=T, H=H, I=I, E=E, top_k=k, block_size=16, weights=weights, **kw)


CASES = [
    # token counts on both sides of the fragment (16), wave (8) and limit (32) borders
    *[C(f"bf16_T{T}", T, 256, 128, 8, 2, seed=T) for T in (1, 2, 7, 8, 9, 15, 16, 17, 31, 32)],
    # odd sizes: widths that are no multiple of a panel, a load or a wave's share
    C("bf16_odd", 5, 264, 200, 6, 3, seed=1), C("bf16_tiny", 3, 8, 8, 2, 1, seed=2), C("bf16_k8", 4, 1048, 8, 4, 2, seed=3),
    C("bf16_n8", 4, 8, 1048, 4, 2, seed=4), C("bf16_wide", 2, 2056, 1000, 4, 2, seed=5),
    # one panel's split count at its limits: few panels with many experts, more panels than the grid
    C("bf16_split", 32, 24, 72, 64, 8, seed=6), C("bf16_panels", 1, 8448, 32, 2, 1, seed=7),
    # experts: one, one wave's worth and beyond, the limit; every expert chosen; no renormalisation
    C("e1", 6, 128, 64, 1, 1, seed=8), C("e63", 9, 128, 64, 63, 5, seed=9), C("e65", 9, 128, 64, 65, 5, seed=10),
    C("e200", 20, 64, 64, 200, 8, seed=11), C("e256", 32, 64, 32, 256, 32, seed=12), C("all", 4, 128, 64, 12, 12, seed=13),
    C("no_renorm", 5, 128, 64, 8, 2, renormalize=False, seed=14), C("skewed", 32, 128, 64, 128, 8, logits="zipf", seed=15),
    # experts with more than 16 tokens (two groups): one more, all of them
    *[C(f"{w}_two_groups_T{T}", T, 256, 128, E, E, w, group_size=64, seed=T + E)
      for w in ("bf16", "int4_gptq", "fp8", "fp8_block") for T, E in ((17, 3), (32, 8))],
    C("two_groups_e256", 32, 64, 32, 256, 32, logits="zipf", seed=33),
    # int4: every group size, one and two token fragments, few groups per wave
    *[C(f"int4_g{G}_T{T}", T, 512, 256, 8, 2, "int4_gptq", group_size=G, seed=G + T) for G in (32, 64, 128, 256) for T in (1, 19)],
    C("int4_one_unit", 3, 64, 64, 4, 2, "int4_gptq", group_size=64, seed=20), C("int4_mid", 16, 1024, 704, 16, 4, "int4_gptq", group_size=64, seed=21),
    # rows of x that do not fit LDS beside the panel sums (and the widest that do)
    *[C(f"{w}_x{H}_T{T}", T, H, 64, 4, 2, w, group_size=64, seed=H + T)
      for w in ("bf16", "int4_gptq", "fp8_block") for T, H in ((16, 2688), (16, 4096), (8, 8192), (20, 1792), (32, 2048), (24, 4096))],
    # fp8: channel and block scales, widths that end inside a block
    *[C(f"{w}_T{T}", T, 384, 256, 8, 2, w, seed=T) for w in ("fp8", "fp8_block") for T in (1, 16, 23)],
    *[C(f"{w}_odd", 5, 400, 208, 6, 3, w, seed=30) for w in ("fp8", "fp8_block")],
    *[C(f"{w}_tiny", 2, 16, 16, 3, 2, w, seed=31) for w in ("fp8", "fp8_block")],
]


@pytest.mark.parametrize("cfg", CASES, ids=[c.name for c in CASES])
def test_few_tokens(m, cfg):
    print(f"few_tokens {cfg}", flush=True)
    d, dev, mat = inputs(cfg)
    plan = m.few_tokens_plan(*dev, cfg.top_k, cfg.T, cfg.renormalize)
    logits, x = to_dev(d["logits"]), bf16_dev(d["x"])
    got = m.moe_few_tokens(plan, logits, x)
    check(cfg, got, reference(cfg, d, mat))
    again = m.moe_few_tokens(plan, logits, x)      # the counters are back at zero; same bits
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    ids, w = m.moe_route(logits, cfg.top_k, cfg.renormalize)
    assert torch.equal(ids, got[1]) and torch.equal(w, got[2])


def test_few_tokens_ties_and_equal_tokens(m):
    """Equal logits pick the lower experts, and equal tokens (the same row 32 times) get equal rows."""
    cfg = C("ties", 32, 256, 128, 40, 4, seed=3)
    d, dev, mat = inputs(cfg)
    d["logits"][:] = 0.0
    d["logits"][0, 5] = -0.0
    d["x"][:] = d["x"][0]
    got = m.moe_few_tokens(m.few_tokens_plan(*dev, 4), to_dev(d["logits"]), bf16_dev(d["x"]))
    assert np.array_equal(got[1].cpu().numpy(), np.tile(np.arange(4, dtype=np.int32), (32, 1)))
    o = bits_host(got[0])
    assert (o == o[0]).all()
    check(cfg, got, reference(cfg, d, mat))


def test_few_tokens_no_tokens(m):
    cfg = C("none", 1, 64, 64, 4, 2)
    d, dev, _ = inputs(cfg)
    plan = m.few_tokens_plan(*dev, 2, 4)
    out, ids, w = m.moe_few_tokens(plan, torch.empty((0, 4), device="cuda"), torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert out.shape == (0, 64) and ids.shape == (0, 2) and w.shape == (0, 2)


@pytest.mark.parametrize("weights", ["bf16", "int4_gptq", "fp8_block"])
def test_few_tokens_one_plan_many_counts(m, weights):
    """One workspace for calls of changing token counts, each equal to a call on a fresh plan; nothing
    outside the caller's rows is written."""
    cfg = C("counts", 32, 512, 256, 16, 4, weights, group_size=128, seed=5)
    d, dev, _ = inputs(cfg)
    logits, x = to_dev(d["logits"]), bf16_dev(d["x"])
    plan = m.few_tokens_plan(*dev, 4)
    for T in (32, 1, 17, 3, 16, 32, 2):
        fresh = m.moe_few_tokens(m.few_tokens_plan(*dev, 4, T), logits[:T], x[:T])
        out = torch.full((T + 1, 512), 9.0, dtype=torch.bfloat16, device="cuda")
        ids = torch.full((T * 4 + 4,), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T * 4 + 4,), -7.0, device="cuda")
        m.moe_few_tokens(plan, logits[:T], x[:T], topk_ids=ids, topk_w=w, out=out[:T])
        assert torch.equal(out[:T], fresh[0]) and (out[T] == 9).all()
        assert torch.equal(ids[: T * 4].view(T, 4), fresh[1]) and (ids[T * 4:] == -7).all()
        assert torch.equal(w[: T * 4].view(T, 4), fresh[2]) and (w[T * 4:] == -7).all()


def test_few_tokens_layers_share_a_workspace(m):
    """Layers of different sizes and weight types, one after the other on the larger one's workspace:
    no call leaves anything where the next one's counters have to be zero."""
    import dataclasses
    cfgs = [C("a", 20, 1024, 256, 32, 8, seed=1), C("b", 20, 64, 512, 64, 8, "int4_gptq", group_size=64, seed=2),
            C("c", 20, 4160, 64, 8, 2, "fp8_block", seed=3)]
    made = [(c, *inputs(c)) for c in cfgs]
    plans = [m.few_tokens_plan(*dev, c.top_k, c.T) for c, _, dev, _ in made]
    big = max((p.workspace for p in plans), key=lambda t: t.numel())
    shared = [dataclasses.replace(p, workspace=big) for p in plans]
    want = [m.moe_few_tokens(p, to_dev(d["logits"]), bf16_dev(d["x"])) for p, (c, d, _, _) in zip(plans, made)]
    for order in ((0, 1, 2), (2, 1, 0), (1, 1, 0, 2, 0)):
        for i in order:
            got = m.moe_few_tokens(shared[i], to_dev(made[i][1]["logits"]), bf16_dev(made[i][1]["x"]))
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


@pytest.mark.parametrize("weights", ["bf16", "int4_gptq"])
def test_few_tokens_graph_and_stream(m, weights):
    """Captured and replayed with new inputs between the replays, with eager calls of another plan in
    between, and run on a side stream: the eager call's bits every time."""
    cfg = C("graph", 9, 1024, 512, 32, 4, weights, group_size=128, seed=8)
    d, dev, _ = inputs(cfg)
    rng = np.random.default_rng(0)
    sets = [(to_dev(rng.standard_normal((9, 32)).astype(np.float32)),
             torch.from_numpy(rng.standard_normal((9, 1024))).to("cuda", torch.bfloat16)) for _ in range(4)]
    eager = m.few_tokens_plan(*dev, 4, 9)
    want = [m.moe_few_tokens(eager, *s) for s in sets]
    plan = m.few_tokens_plan(*dev, 4, 9)
    logits, x = sets[0][0].clone(), sets[0][1].clone()
    ids, w, out = torch.empty_like(want[0][1]), torch.empty_like(want[0][2]), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = m.moe_few_tokens(plan, logits, x)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, want[0]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_few_tokens(plan, logits, x, topk_ids=ids, topk_w=w, out=out)
    for i in (0, 1, 2, 3, 1):
        logits.copy_(sets[i][0])
        x.copy_(sets[i][1])
        g.replay()
        other = m.moe_few_tokens(eager, *sets[(i + 1) % 4])
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][0]) and torch.equal(ids, want[i][1]) and torch.equal(w, want[i][2])
        assert torch.equal(other[0], want[(i + 1) % 4][0])


@pytest.mark.parametrize("weights", ["bf16", "int4_gptq", "fp8", "fp8_block"])
@pytest.mark.parametrize("T", [3, 20])
def test_few_tokens_non_finite_rows_stay_their_own(m, weights, T):
    """A token of NaN or infinities spoils its own row only, and an expert nobody chose is not read."""
    cfg = C("nan", T, 256, 128, 8, 2, weights, group_size=64, seed=21)
    d, dev, _ = inputs(cfg)
    d["logits"][:, 5] = -100.0       # expert 5 is chosen by nobody
    for w in dev:
        if weights == "int4_gptq":
            w.scales[5] = float("nan")
        elif weights == "bf16":
            w.w[5] = float("nan")
        else:
            w.codes[5] = 0x7F
    plan = m.few_tokens_plan(*dev, 2, T)
    logits, x = to_dev(d["logits"]), bf16_dev(d["x"])
    clean = m.moe_few_tokens(plan, logits, x)[0]
    assert torch.isfinite(clean.float()).all()
    bad = x.clone()
    bad[1] = float("nan")
    bad[2, 7] = float("inf")
    got = m.moe_few_tokens(plan, logits, bad)[0]
    keep = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[1].float()).all() and not torch.isfinite(got[2].float()).any()
