"""Measured cases of the serving operators of the routed expert path: the residual addition with
root-mean-square norm and its 8-bit output, 8-bit quantisation and grouped products with one scale
per block of 128, and the whole layer for a few tokens.

``run`` computes an operator in plain torch (``own`` false) or through the package (``own`` true);
``exact`` gives the same outputs from the definitions in fp64.
"""
import math

import torch

own = False

BLOCK = 128      # values under one scale of the block-scaled 8-bit format
E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of a 64-expert int4 model: latency of routing, experts and combine
        _few("few_token1_int4", 1, 2048, 1408, 64, 6, "int4"),
        # a decode batch of the same model: most experts active, their weights streamed once
        _few("few_batch16_int4", 16, 2048, 1408, 64, 6, "int4"),
        # four tokens of a model of 8 large experts in bf16: the longest weight stream
        _few("few_batch4_bf16", 4, 4096, 14336, 8, 2, "bf16"),
        # an odd batch over 128 fine-grained experts with block-scaled 8-bit weights
        _few("few_batch23_fp8_block", 23, 2048, 768, 128, 8, "fp8_block"),
        # the norm in front of the layer for one decoded token
        _norm("norm_token1", 1, 2048, True, "bf16"),
        # the same for a prefill batch, with the per-row 8-bit codes the fp8 experts read and the
        # bf16 rows the router reads
        _norm("norm_prefill_fp8_row", 4096, 4096, True, "both_row"),
        # a ragged prefill batch and width, straight to block-scaled codes
        _norm("norm_ragged_fp8_block", 5003, 5136, True, "fp8_block"),
        # activations quantised by blocks: tokens in front of gate/up, sorted rows in front of down
        _quant("quant_tokens", 8191, 4096, 0, 0, 0),
        _quant("quant_sorted_rows", 2048, 1408, 64, 6, 64),
        # block-scaled experts, prefill: gate/up with 8 large experts
        _gemm("gate_up_prefill", "gate_up", 4096, 14336, 4096, 8, 2, 64),
        # gate/up that hands the down product its codes
        _gemm("gate_up_codes", "gate_up_codes", 2048, 1408, 4096, 64, 6, 64),
        # down over many fine-grained experts: few rows each, a short contraction
        _gemm("down_fine", "down", 8192, 2048, 768, 128, 8, 64),
    ]


def _few(name, T, H, I, E, k, weights, group=128):
    return {"name": name, "op": "few", "T": T, "H": H, "I": I, "E": E, "k": k, "weights": weights, "group": group}


def _norm(name, rows, width, residual, out):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "residual": residual, "out": out}


def _quant(name, T, width, E, k, block):
    return {"name": name, "op": "quant", "T": T, "width": width, "E": E, "k": k, "block": block}


def _gemm(name, kind, T, N, K, E, k, block):
    return {"name": name, "op": "gemm", "kind": kind, "T": T, "N": N, "K": K, "E": E, "k": k, "block": block}


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["few", "few", "norm", "quant", "gemm", "gemm"])
    if op == "few":
        weights = rng.choice(["bf16", "int4", "fp8", "fp8_block"])
        group = rng.choice([32, 64, 128]) if weights == "int4" else 128
        step = {"bf16": 8, "int4": max(64, group), "fp8": 16, "fp8_block": 16}[weights]
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 32)
        H, I = _log(rng, 256, 6144, step), _log(rng, 128, 6144, step)
        while max(E, T * k) * H * I > 8 * 4096 * 14336:  # no larger than the largest listed case
            H, I = max(step, H // 2 // step * step), max(step, I // 2 // step * step)
        c = _few("", T, H, I, E, k, weights, group)
    elif op == "norm":
        out = rng.choice(["bf16", "both_row", "both_block", "fp8_row", "fp8_block"])
        c = _norm("", _log(rng, 1, 4500), _log(rng, 64, 6000, 16), rng.random() < 0.7, out)
    elif op == "quant":
        if rng.random() < 0.5:
            c = _quant("", _log(rng, 1, 8000), _log(rng, 64, 5000, 16), 0, 0, 0)
        else:
            E = _log(rng, 4, 256)
            c = _quant("", _log(rng, 1, 1500), _log(rng, 64, 4000, 16), E, rng.randint(1, min(6, E)), rng.choice([16, 32, 64]))
    else:
        kind = rng.choice(["gate_up", "gate_up_codes", "down"])
        E = _log(rng, 4, 160)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 16, 4096)
        N, K = _log(rng, 128, 6144, 16), _log(rng, 128, 6144, 16)
        while max(8 * T * k, E * 512) * N * K > 65536 * 4096 * 14336:
            N, K = max(128, N // 2 // 16 * 16), max(128, K // 2 // 16 * 16)
        c = _gemm("", kind, T, N, K, E, k, rng.choice([16, 32, 64, 128]))
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(g, shape):
    """E4M3 codes of random sign, exponent field 4..10 and mantissa: finite, magnitudes 1/8 to 15."""
    c = torch.randint(0, 7 * 8, shape, generator=g, device="cuda", dtype=torch.uint8) + 4 * 8
    return c | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)


def _uniform(g, shape, lo, hi):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


def _expert_weight(g, kind, E, N, K, group):
    """Expert matrices of one projection: a dict of tensors in the package's layouts."""
    if kind == "bf16":
        return {"w": torch.randn((E, N, K), generator=g, device="cuda", dtype=torch.bfloat16).mul_(0.02)}
    if kind == "int4":
        word = dict(generator=g, device="cuda", dtype=torch.int32)
        return {"q": torch.randint(-2**31, 2**31 - 1, (E, K // 8, N), **word),
                "s": _uniform(g, (E, K // group, N), 0.005, 0.02).half(),
                "z": torch.randint(-2**31, 2**31 - 1, (E, K // group, N // 8), **word), "group": group}
    if kind == "fp8":
        return {"c": _codes(g, (E, N, K)), "s": _uniform(g, (E, N), 0.002, 0.006)}
    return {"c": _codes(g, (E, N, K)), "s": _uniform(g, (E, -(-N // BLOCK), -(-K // BLOCK)), 0.002, 0.006)}


def _package_weight(m, w):
    if "w" in w:
        return m.Bf16Weight(w["w"])
    if "q" in w:
        return m.GptqWeight(w["q"], w["s"], w["z"], w["group"])
    return m.Fp8Weight(w["c"], w["s"]) if w["s"].dim() == 2 else m.Fp8BlockWeight(w["c"], w["s"])


def _alignment(g, T, E, k, bs):
    """The sorted, block-padded layout of random routing: expert by expert, pairs ascending, the
    number of pairs in every row without one."""
    P = T * k
    ids = torch.sort(torch.randn((T, E), generator=g, device="cuda"), dim=1, descending=True).indices[:, :k]
    flat = ids.reshape(-1)
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").index_add_(0, flat, torch.ones_like(flat))
    padded = (counts + bs - 1) // bs * bs
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[1:] = torch.cumsum(padded, 0)
    first = torch.cumsum(counts, 0) - counts
    order = torch.sort(flat, stable=True).indices
    rank = torch.empty_like(order)
    rank[order] = torch.arange(P, device="cuda") - first[flat[order]]
    pos = off[flat] + rank
    mp = -(-(P + E * (bs - 1)) // bs) * bs
    sorted_ids = torch.full((mp,), P, dtype=torch.int32, device="cuda")
    sorted_ids[pos] = torch.arange(P, device="cuda", dtype=torch.int32)
    block = torch.arange(mp // bs, device="cuda") * bs
    owner = torch.searchsorted(off[1:].contiguous(), block, right=True)
    owner = torch.where(block < off[-1], owner, -1).int()
    return {"P": P, "k": k, "E": E, "bs": bs, "mp": mp, "expert": flat, "rank": rank, "pos": pos,
            "most": int(counts.max()), "counts": counts.int(), "off": off.int(), "sorted": sorted_ids,
            "block": owner, "total": off[-1:].int(), "inv": pos.int()}


def _package_routing(m, a):
    return m.Routing(a["counts"], a["off"], a["sorted"], a["block"], a["total"], a["inv"],
                     torch.empty(1, dtype=torch.int32, device="cuda"), a["P"], a["k"], a["E"], a["bs"], a["mp"])


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if own:
        import mixture_experts_routed_route_amd as m
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if c["op"] == "few":
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        s = {"case": c, "logits": torch.randn((T, E), generator=g, device="cuda"),
             "x": torch.randn((T, H), generator=g, **bf)}
        for name, N, K in (("gate", I, H), ("up", I, H), ("down", H, I)):
            s[name] = _expert_weight(g, c["weights"], E, N, K, c["group"])
        if own:  # the layer's weights checked and its workspace made once, as a server does
            s["plan"] = m.few_tokens_plan(*[_package_weight(m, s[n]) for n in ("gate", "up", "down")], c["k"], T)
        return s
    if c["op"] == "norm":
        R, W = c["rows"], c["width"]
        s = {"case": c, "x": torch.randn((R, W), generator=g, **bf),
             "weight": (1 + 0.1 * torch.randn(W, generator=g, device="cuda")).bfloat16()}
        if c["residual"]:
            s["r"], s["h"] = 2 * torch.randn((R, W), generator=g, **bf), torch.empty((R, W), **bf)
        if c["out"] != "fp8_row" and c["out"] != "fp8_block":
            s["y"] = torch.empty((R, W), **bf)
        if c["out"] != "bf16":
            s["q"] = torch.empty((R, W), dtype=torch.uint8, device="cuda")
            s["scale"] = torch.empty((R,) if c["out"].endswith("row") else (R, -(-W // BLOCK)), device="cuda")
        return s
    if c["op"] == "quant":
        rows = c["T"]
        s = {"case": c}
        if c["E"]:
            s["a"] = _alignment(g, c["T"], c["E"], c["k"], c["block"])
            rows = s["a"]["mp"]
            if own:
                s["routing"] = _package_routing(m, s["a"])
        # SiLU * up rows: heavy-tailed, so that blocks of one row differ in scale
        u = torch.randn((rows, c["width"]), generator=g, device="cuda")
        s["x"] = (u * torch.randn((rows, c["width"]), generator=g, device="cuda").abs()).bfloat16()
        s["q"] = torch.zeros((rows, c["width"]), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros((rows, -(-c["width"] // BLOCK)), device="cuda")
        return s
    N, K, E = c["N"], c["K"], c["E"]
    a = _alignment(g, c["T"], E, c["k"], c["block"])
    rows = a["mp"] if c["kind"] == "down" else c["T"]
    s = {"case": c, "a": a, "x": _codes(g, (rows, K)), "sx": _uniform(g, (rows, -(-K // BLOCK)), 0.01, 0.05),
         "w0": _expert_weight(g, "fp8_block", E, N, K, 0)}
    if c["kind"] != "down":
        s["w1"] = _expert_weight(g, "fp8_block", E, N, K, 0)
    # outputs start at zero: rows without a token are never written
    if c["kind"] == "gate_up_codes":
        s["q"] = torch.zeros((a["mp"], N), dtype=torch.uint8, device="cuda")
        s["scale"] = torch.zeros((a["mp"], -(-N // BLOCK)), device="cuda")
    else:
        s["out"] = torch.zeros((a["mp"], N), **bf)
    if own:
        s["routing"] = _package_routing(m, a)
        s["workspace"] = m.gemm_workspace("cuda")
        s["pw"] = [_package_weight(m, s[n]) for n in ("w0", "w1") if n in s]
    return s


# --------------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _e4m3(q):
    return q.view(torch.float8_e4m3fn)


def _run_own(s):
    import mixture_experts_routed_route_amd as m
    c = s["case"]
    if c["op"] == "few":
        out, ids, w = m.moe_few_tokens(s["plan"], s["logits"], s["x"])
        return {"out": out, "ids": ids, "w": w}
    if c["op"] == "norm":
        m.moe_rmsnorm(s["x"], s["weight"], EPS, residual=s.get("r"), residual_out=s.get("h"), y=s.get("y"),
                      q=s.get("q"), scale=s.get("scale"))
        got = {n: s[n] for n in ("h", "y", "scale") if n in s}
        return {**got, "q": _e4m3(s["q"])} if "q" in s else got
    if c["op"] == "quant":
        m.moe_quantize_fp8_block(s["x"], s["q"], s["scale"], s.get("routing"))
        return {"q": _e4m3(s["q"]), "scale": s["scale"]}
    op = m.MOE_OP_DOWN if c["kind"] == "down" else m.MOE_OP_GATE_UP_SILU
    w0, w1 = s["pw"][0], s["pw"][1] if len(s["pw"]) > 1 else None
    if "q" in s:
        m.moe_grouped_gemm_fp8_block(op, s["x"], s["sx"], w0, w1, s["routing"], q=s["q"], scale=s["scale"],
                                     workspace=s["workspace"])
        return {"q": _e4m3(s["q"]), "scale": s["scale"]}
    return {"out": m.moe_grouped_gemm_fp8_block(op, s["x"], s["sx"], w0, w1, s["routing"], out=s["out"],
                                                workspace=s["workspace"])}


def _spread(scale, width):
    """One value per block of 128 -> one per element."""
    return scale.repeat_interleave(BLOCK, dim=-1)[..., :width]


def _dequant(w, pick=None):
    """fp32 matrices [.., N, K] of the experts ``pick`` (all without it)."""
    take = (lambda t: t) if pick is None else (lambda t: t[pick])
    if "w" in w:
        return take(w["w"]).float()
    if "q" in w:
        q, z, sc = take(w["q"]), take(w["z"]), take(w["s"]).float()
        nib = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)
        q = ((q.unsqueeze(2) >> nib.view(1, 1, 8, 1)) & 15).flatten(1, 2).float()
        z = ((z.unsqueeze(3) >> nib) & 15).flatten(2, 3).float()
        G = w["group"]
        return ((q - z.repeat_interleave(G, 1)) * sc.repeat_interleave(G, 1)).transpose(1, 2)
    v, sc = _e4m3(take(w["c"])).float(), take(w["s"])
    if sc.dim() == 2:
        return v * sc.unsqueeze(2)
    return v * _spread(sc.repeat_interleave(BLOCK, 1)[:, : v.shape[1]], v.shape[2])


def _silu(g):
    return g / (1 + torch.exp(-g))


def _quantise(v, groups):
    """Codes and scales of fp32 values [rows, width] over blocks of 128 columns or whole rows."""
    rows, width = v.shape
    if groups == "row":
        amax = v.abs().amax(1, keepdim=True)
    else:
        nb = -(-width // BLOCK)
        pad = torch.zeros((rows, nb * BLOCK), device=v.device, dtype=v.dtype)
        pad[:, :width] = v
        amax = pad.view(rows, nb, BLOCK).abs().amax(2)
    one = torch.ones_like(amax)
    scale = torch.where(amax > 0, amax / E4M3_MAX, one)
    f = torch.where(amax > 0, E4M3_MAX / amax, one)
    f = f if groups == "row" else _spread(f, width)
    return (v * f).to(torch.float8_e4m3fn), scale.squeeze(1) if groups == "row" else scale


def _run_plain(s):
    c = s["case"]
    if c["op"] == "few":
        T, k, I = c["T"], c["k"], c["I"]
        lg = s["logits"]
        ids = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]
        p = torch.exp(lg.double() - lg.double().amax(1, keepdim=True))
        w = torch.gather(p, 1, ids)
        w = w / w.sum(1, keepdim=True)
        flat = ids.reshape(-1)
        x = s["x"].float().repeat_interleave(k, 0).unsqueeze(2)
        h = _silu(torch.bmm(_dequant(s["gate"], flat), x)) * torch.bmm(_dequant(s["up"], flat), x)
        y = torch.bmm(_dequant(s["down"], flat), h).view(T, k, c["H"])
        out = (w.float().unsqueeze(2) * y).sum(1)
        return {"out": out.bfloat16(), "ids": ids.int(), "w": w.float()}
    if c["op"] == "norm":
        h = s["x"].float()
        got = {}
        if "r" in s:
            got["h"] = (h + s["r"].float()).bfloat16()
            h = got["h"].float()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
        if "y" in s:
            got["y"] = y.bfloat16()
        if "q" in s:
            got["q"], got["scale"] = _quantise(y, "row" if c["out"].endswith("row") else "block")
        return got
    if c["op"] == "quant":
        q, scale = _quantise(s["x"].float(), "block")
        if c["E"]:
            real = (s["a"]["sorted"] < s["a"]["P"]).unsqueeze(1)
            q, scale = _e4m3(torch.where(real, q.view(torch.uint8), 0)), torch.where(real, scale, 0.0)
        return {"q": q, "scale": scale}
    a, N, K = s["a"], c["N"], c["K"]
    x = _e4m3(s["x"]).float() * _spread(s["sx"], K)
    rows = a["pos"] if c["kind"] == "down" else torch.arange(a["P"], device="cuda") // a["k"]
    at = a["expert"] * a["most"] + a["rank"]     # expert by expert, each with room for the busiest's rows
    xs = torch.zeros((a["E"] * a["most"], K), device="cuda")
    xs[at] = x[rows]
    xs = xs.view(a["E"], a["most"], K)
    y = torch.bmm(xs, _dequant(s["w0"]).transpose(1, 2)).view(-1, N)[at]
    if c["kind"] != "down":
        y = _silu(y) * torch.bmm(xs, _dequant(s["w1"]).transpose(1, 2)).view(-1, N)[at]
    if "q" in s:
        q, scale = _quantise(y, "block")
        qs = torch.zeros((a["mp"], N), dtype=torch.uint8, device="cuda")
        qs[a["pos"]] = q.view(torch.uint8)
        ss = torch.zeros((a["mp"], scale.shape[1]), device="cuda")
        ss[a["pos"]] = scale
        return {"q": _e4m3(qs), "scale": ss}
    out = torch.zeros((a["mp"], N), dtype=torch.bfloat16, device="cuda")
    out[a["pos"]] = y.bfloat16()
    return {"out": out}


# ---------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "few":
        return _exact_few(s)
    if c["op"] == "norm":
        v = s["x"].double()
        got = {}
        if "r" in s:
            v = (v + s["r"].double()).to(torch.bfloat16).double()
            got["h"] = v
        v = s["weight"].double() * v * torch.rsqrt(v.pow(2).mean(1, keepdim=True) + EPS)
        if "y" in s:
            got["y"] = v
        if "q" in s:
            got["q"], got["scale"] = _exact_quantise(v, v.shape[1] if c["out"].endswith("row") else BLOCK)
            if c["out"].endswith("row"):
                got["scale"] = got["scale"].reshape(-1)
        return got
    if c["op"] == "quant":
        q, scale = _exact_quantise(s["x"].double(), BLOCK)
        if c["E"]:
            drop = torch.ones(q.shape[0], dtype=torch.bool, device="cuda")
            drop[s["a"]["pos"]] = False
            q[drop], scale[drop] = 0, 0
        return {"q": q, "scale": scale}
    return _exact_gemm(s)


def _exact_quantise(v, width):
    """Unrounded codes v / scale and scales amax / 448, block by block."""
    q = torch.empty_like(v)
    scales = []
    for lo in range(0, v.shape[1], width):
        part = v[:, lo:lo + width]
        top = part.abs().max(1).values
        sc = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
        q[:, lo:lo + width] = part / sc[:, None]
        scales.append(sc)
    return q, torch.stack(scales, 1)


def _exact_matrix(w, e):
    """Expert e's [N, K] matrix in fp64."""
    if "w" in w:
        return w["w"][e].double()
    if "q" in w:
        words, G = w["q"][e].long(), w["group"]
        q = torch.stack([(words >> (4 * i)) & 0xF for i in range(8)], 1).reshape(-1, words.shape[1]).double()
        zw = w["z"][e].long()
        z = torch.stack([(zw >> (4 * i)) & 0xF for i in range(8)], 2).reshape(zw.shape[0], -1).double()
        group = torch.arange(q.shape[0], device=q.device) // G
        return ((q - z[group]) * w["s"][e].double()[group]).t()
    v = w["c"][e].view(torch.float8_e4m3fn).double()
    sc = w["s"][e].double()
    if sc.dim() == 1:
        return v * sc[:, None]
    n, k = (torch.arange(m, device=v.device) // BLOCK for m in v.shape)
    return v * sc[n][:, k]


def _exact_few(s):
    c = s["case"]
    p = torch.softmax(s["logits"].double(), 1)
    out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = p.gather(1, order)
    w = w / w.sum(1, keepdim=True)
    pairs = order.tolist()
    for e in sorted({v for row in pairs for v in row}):
        ts = [t for t in range(c["T"]) if e in pairs[t]]
        x = s["x"][ts].double()
        g = x @ _exact_matrix(s["gate"], e).t()
        h = g * torch.sigmoid(g) * (x @ _exact_matrix(s["up"], e).t())
        y = h @ _exact_matrix(s["down"], e).t()
        for i, t in enumerate(ts):
            out[t] += w[t, pairs[t].index(e)] * y[i]
    return {"out": out, "ids": None, "w": w}


def _exact_gemm(s):
    c, a = s["case"], s["a"]
    y = torch.zeros((a["mp"], c["N"]), dtype=torch.float64, device="cuda")
    kb = torch.arange(c["K"], device="cuda") // BLOCK
    for e in range(a["E"]):
        mine = (a["expert"] == e).nonzero().reshape(-1)
        if not len(mine):
            continue
        at = a["pos"][mine]
        src = at if c["kind"] == "down" else mine // a["k"]
        x = s["x"][src].view(torch.float8_e4m3fn).double() * s["sx"][src].double()[:, kb]
        v = x @ _exact_matrix(s["w0"], e).t()
        if c["kind"] != "down":
            v = v * torch.sigmoid(v) * (x @ _exact_matrix(s["w1"], e).t())
        y[at] = v
    if c["kind"] != "gate_up_codes":
        return {"out": y}
    q, scale = _exact_quantise(y, BLOCK)
    real = a["sorted"] < a["P"]
    scale[~real] = 0
    return {"q": q, "scale": scale}


# ------------------------------------------------------------------------------------------- work
def _matrix_bytes(kind, N, K, group):
    if kind == "bf16":
        return 2 * N * K
    if kind == "int4":
        return N * K / 2 + N * K / group * 2.5
    return N * K + (4 * N if kind == "fp8" else 4 * -(-N // BLOCK) * -(-K // BLOCK))


def work(case):
    c = case
    if c["op"] == "few":
        T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
        active = E * (1 - (1 - k / E) ** T)  # experts that T random choices of k are expected to reach
        mats = 2 * _matrix_bytes(c["weights"], I, H, c["group"]) + _matrix_bytes(c["weights"], H, I, c["group"])
        return {"bytes": active * mats + 4 * T * E + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}
    if c["op"] == "norm":
        n, scales = c["rows"] * c["width"], 4 * c["rows"] * (1 if c["out"].endswith("row") else -(-c["width"] // BLOCK))
        y = 0 if c["out"].startswith("fp8") else 2
        q = 0 if c["out"] == "bf16" else 1
        return {"bytes": n * (2 + (4 if c["residual"] else 0) + y + q) + q * scales + 2 * c["width"], "flops": 6 * n}
    if c["op"] == "quant":
        rows = c["T"] * c["k"] if c["E"] else c["T"]
        return {"bytes": rows * (3 * c["width"] + 4 * -(-c["width"] // BLOCK)), "flops": 3 * rows * c["width"]}
    T, N, K, E, k = c["T"], c["N"], c["K"], c["E"], c["k"]
    mats = 1 if c["kind"] == "down" else 2
    active = E * (1 - (1 - k / E) ** T)
    rows_in = T * k if c["kind"] == "down" else T
    out = T * k * ((N + 4 * -(-N // BLOCK)) if c["kind"] == "gate_up_codes" else 2 * N)
    return {"bytes": active * mats * _matrix_bytes("fp8_block", N, K, 0) + rows_in * (K + 4 * -(-K // BLOCK)) + out,
            "flops": 2 * mats * T * k * N * K}
