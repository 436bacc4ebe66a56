"""Measured cases of the gradients of the routed expert path: SiLU * up with dropout and its backward,
the grouped products for the gradients of their inputs and of their weights, and the gradient of the
router's logits.

``run`` computes an operator in plain torch (``own`` false) or through the package (``own`` true);
``exact`` gives the same outputs from the definitions in fp64.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # hidden activations of 128 fine-grained experts, a training batch, with dropout
        _act("dropout_fine", "dropout", 8192, 768, 128, 8, 64, 0.1),
        # the same of the smallest layer: latency
        _act("dropout_tiny", "dropout", 64, 128, 8, 2, 16, 0.4),
        # backward of SiLU * up for 8 large experts, no dropout
        _act("act_backward_prefill", "act_backward", 4096, 14336, 8, 2, 64, 0.0),
        # a ragged batch over 64 experts, with dropout
        _act("act_backward_ragged", "act_backward", 1999, 1408, 64, 6, 64, 0.1),
        # gradient of the hidden activations from that of the layer's output: 8 large experts
        _grad("dgrad_down_prefill", "dgrad", 4096, 4096, 14336, 8, 2, 64, by_token=True),
        # gradient of the layer's input through gate and up: many small experts, skewed routing
        _grad("dgrad_gate_up_skewed", "dgrad", 8192, 768, 2048, 128, 8, 64, pair=True, skew=1.26),
        # the same for a few tokens: the weights are streamed once
        _grad("dgrad_gate_up_few", "dgrad", 16, 1408, 2048, 64, 6, 16, pair=True),
        # weight gradient of the gate projection of 8 large experts
        _grad("wgrad_gate_prefill", "wgrad", 4096, 14336, 4096, 8, 2, 64, x_by_token=True),
        # weight gradient of the down projection added to fp32 sums of earlier batches, skewed routing
        _grad("wgrad_down_skewed_sum", "wgrad", 8192, 2048, 768, 128, 8, 64, by_token=True, skew=1.26, out="fp32", base=True),
        # a ragged batch over 64 experts: short contractions, the gradients' bytes count
        _grad("wgrad_ragged", "wgrad", 2047, 1408, 4096, 64, 6, 32, x_by_token=True),
        # gradient of the router's logits: a training batch, weights renormalised over the chosen
        _route("route_backward_batch", 8192, 128, 8, True),
        # and over all experts, a few tokens: latency
        _route("route_backward_few", 64, 256, 8, False),
    ]


def _act(name, op, T, I, E, k, block, p):
    return {"name": name, "op": op, "T": T, "I": I, "E": E, "k": k, "block": block, "p": p}


def _grad(name, op, T, N, K, E, k, block, pair=False, by_token=False, x_by_token=False, skew=0.0, out="bf16", base=False):
    return {"name": name, "op": op, "T": T, "N": N, "K": K, "E": E, "k": k, "block": block, "pair": pair,
            "by_token": by_token, "x_by_token": x_by_token, "skew": skew, "out": out, "base": base}


def _route(name, T, E, k, renormalize):
    return {"name": name, "op": "route_backward", "T": T, "E": E, "k": k, "renormalize": renormalize}


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["dropout", "act_backward", "dgrad", "dgrad", "wgrad", "wgrad", "route_backward"])
    E = _log(rng, 4, 160)
    k = rng.randint(1, min(8, E))
    block = rng.choice([16, 32, 64, 128])
    if op == "route_backward":
        c = _route("", _log(rng, 1, 8192), _log(rng, k, 256), k, rng.random() < 0.6)
    elif op in ("dropout", "act_backward"):
        c = _act("", op, _log(rng, 1, 8192), _log(rng, 64, 8192, 8), E, k, block, rng.choice([0.0, 0.05, 0.1, 0.3, 0.5]))
        while c["T"] * k * c["I"] > 8192 * 8192:
            c["T"] = max(1, c["T"] // 2)
    else:
        N, K, T = _log(rng, 128, 6144, 8), _log(rng, 128, 6144, 8), _log(rng, 1, 4096)
        while max(8 * T * k, E * 512) * N * K > 65536 * 4096 * 14336 or E * N * K > 2**28:
            N, K = max(128, N // 2 // 8 * 8), max(128, K // 2 // 8 * 8)
        c = _grad("", op, T, N, K, E, k, block, by_token=rng.random() < 0.5, skew=rng.choice([0.0, 0.0, 1.26]))
        if op == "dgrad":
            c["pair"] = rng.random() < 0.5
        else:
            c["x_by_token"] = rng.random() < 0.5
            c["out"] = rng.choice(["bf16", "bf16", "fp32"])
            c["base"] = rng.random() < 0.4
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, size=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(size)


def _alignment(g, T, E, k, bs, skew):
    """The sorted, block-padded layout of a random router (with ``skew``, of a few busy experts): expert by
    expert, pairs ascending, the number of pairs in every row without one."""
    P = T * k
    logits = torch.randn((T, E), generator=g, device="cuda")
    if skew:
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        logits = logits - skew * torch.log(rank.float())
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = torch.exp(logits.gather(1, ids))
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
            "block": owner, "total": off[-1:].int(), "inv": pos.int(), "w": chosen / chosen.sum(1, keepdim=True)}


def _package_routing(m, a):
    return m.Routing(a["counts"], a["off"], a["sorted"], a["block"], a["total"], a["inv"],
                     torch.empty(1, dtype=torch.int32, device="cuda"), a["P"], a["k"], a["E"], a["bs"], a["mp"])


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if own:
        import mixture_experts_routed_route_amd as m
    if c["op"] == "route_backward":
        T, E, k = c["T"], c["E"], c["k"]
        logits = torch.randn((T, E), generator=g, device="cuda")
        p = torch.exp(logits.double() - logits.double().amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        w = p.gather(1, ids)
        if c["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return {"case": c, "logits": logits, "ids": ids.int(), "w": w.float().contiguous(),
                "dw": torch.randn((T, k), generator=g, device="cuda"), "out": torch.zeros((T, E), device="cuda")}
    a = _alignment(g, c["T"], c["E"], c["k"], c["block"], c.get("skew", 0.0))
    s = {"case": c, "a": a}
    if own:
        s["routing"] = _package_routing(m, a)
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")  # rows without a token: not written
    if c["op"] in ("dropout", "act_backward"):
        I, mp = c["I"], a["mp"]
        s["g"], s["u"] = _normal(g, (mp, I), 1.5), _normal(g, (mp, I))
        s["rng"] = torch.randint(0, 2**62, (2,), generator=g, device="cuda")  # seed and offset of the generator
        s["h"] = zeros(mp, I)
        if c["op"] == "act_backward":
            s["d"], s["dg"], s["du"] = _normal(g, (mp, I), 0.05), zeros(mp, I), zeros(mp, I)
            s["dw"] = torch.zeros((c["T"], c["k"]), device="cuda")
        return s
    N, K, E, T = c["N"], c["K"], c["E"], c["T"]
    s["dy"] = _normal(g, (T if c["by_token"] else a["mp"], N), 0.1)
    if own:
        s["workspace"] = m.gemm_workspace("cuda")
    if c["op"] == "dgrad":
        s["w"] = _normal(g, (E, N, K), 0.02)
        if c["pair"]:
            s["dy1"], s["w1"] = _normal(g, s["dy"].shape, 0.1), _normal(g, (E, N, K), 0.02)
        s["out"] = zeros(a["mp"], K)
        if own:
            s["pw"] = [m.Bf16Weight(s[n]) for n in ("w", "w1") if n in s]
        return s
    s["x"] = _normal(g, (T if c["x_by_token"] else a["mp"], K))
    dtype = torch.float32 if c["out"] == "fp32" else torch.bfloat16
    s["out"] = torch.empty((E, N, K), dtype=dtype, device="cuda")
    if c["base"]:
        s["base"] = torch.randn((E, N, K), generator=g, device="cuda", dtype=dtype)
    return s


# --------------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import mixture_experts_routed_route_amd as m
    c = s["case"]
    if c["op"] == "route_backward":
        return {"dlogits": m.moe_route_backward(s["ids"], s["w"], s["dw"], c["E"],
                                                logits=None if c["renormalize"] else s["logits"], out=s["out"])}
    if c["op"] == "dropout":
        return {"h": m.moe_silu_mul_dropout(s["g"], s["u"], s["routing"], c["p"], s["rng"], out=s["h"])}
    if c["op"] == "act_backward":
        dg, du, h, dw = m.moe_silu_mul_backward(s["g"], s["u"], s["d"], s["a"]["w"], s["routing"], c["p"], s["rng"],
                                                d_gate=s["dg"], d_up=s["du"], h_weighted=s["h"], d_topk_w=s["dw"])
        return {"dg": dg, "du": du, "h": h, "dw": dw}
    if c["op"] == "dgrad":
        w1 = s["pw"][1] if c["pair"] else None
        return {"dx": m.moe_grouped_gemm_dgrad(s["dy"], s["pw"][0], s["routing"], dy1=s.get("dy1"), w1=w1,
                                               by_token=c["by_token"], out=s["out"], workspace=s["workspace"])}
    return {"dw": m.moe_grouped_gemm_wgrad(s["dy"], s["x"], s["routing"], dy_by_token=c["by_token"],
                                           x_by_token=c["x_by_token"], base=s.get("base"), out=s["out"],
                                           workspace=s["workspace"])}


_LOW = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, seed):
    """Philox 4x32, ten rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011), of int64
    tensors that hold 32-bit words; products wrap at 64 bits and the words are masked out of them."""
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return c0, c1, c2, c3


def _dropped_below(p):
    """16-bit random numbers below this drop their value."""
    return min(65535, int(math.floor(p * 65536 + 0.5)))


def _keep(rng, pairs, I, p):
    """Factors 0 or 1 / (1 - p) of the hidden values of ``pairs``: eight columns from each counter
    (column / 8, pair, offset), two from each word, the low half first."""
    below = _dropped_below(p)
    if not below:
        return 1.0
    n = -(-I // 8)
    c0 = torch.arange(n, device=pairs.device).expand(len(pairs), n)
    c1 = pairs.long().unsqueeze(1).expand(len(pairs), n)
    lo, hi = (rng[1] & _LOW).expand(len(pairs), n), ((rng[1] >> 32) & _LOW).expand(len(pairs), n)
    words = torch.stack(_philox(c0, c1, lo, hi, rng[0]), 2)
    r = torch.stack((words & 0xFFFF, words >> 16), 3).reshape(len(pairs), 8 * n)[:, :I]
    return (r >= below).float() * (65536.0 / (65536 - below))


def _run_plain(s):
    c = s["case"]
    if c["op"] == "route_backward":
        ids, w, dw = s["ids"].long(), s["w"], s["dw"]
        dot = (w * dw).sum(1, keepdim=True)
        if c["renormalize"]:
            return {"dlogits": torch.zeros_like(s["out"]).scatter_(1, ids, w * (dw - dot))}
        p = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        d = torch.zeros_like(p).scatter_(1, ids, dw)
        return {"dlogits": p * (d - dot)}
    a = s["a"]
    if c["op"] in ("dropout", "act_backward"):
        pos = a["pos"]
        g, u = s["g"][pos].float(), s["u"][pos].float()
        keep = _keep(s["rng"], torch.arange(a["P"], device="cuda"), c["I"], c["p"])
        sig = 1 / (1 + torch.exp(-g))
        h = g * sig * u * keep
        full = lambda v: torch.zeros_like(s["h"]).index_copy_(0, pos, v.bfloat16())
        if c["op"] == "dropout":
            return {"h": full(h)}
        d, w = s["d"][pos].float(), a["w"].reshape(-1, 1)
        dh = w * d * keep
        return {"dg": full(dh * u * sig * (1 + g * (1 - sig))), "du": full(dh * g * sig), "h": full(w * h),
                "dw": (d * h).sum(1).view(c["T"], c["k"])}
    N, K, E, most = c["N"], c["K"], c["E"], a["most"]
    at = a["expert"] * most + a["rank"]          # expert by expert, each with room for the busiest's rows
    tokens = torch.arange(a["P"], device="cuda") // a["k"]

    def rows(t, by_token):
        r = torch.zeros((E * most, t.shape[1]), device="cuda")
        r[at] = t[tokens if by_token else a["pos"]].float()
        return r.view(E, most, -1)
    if c["op"] == "dgrad":
        y = torch.bmm(rows(s["dy"], c["by_token"]), s["w"].float())
        if c["pair"]:
            y = y + torch.bmm(rows(s["dy1"], c["by_token"]), s["w1"].float())
        return {"dx": torch.zeros_like(s["out"]).index_copy_(0, a["pos"], y.view(-1, K)[at].bfloat16())}
    dw = torch.bmm(rows(s["dy"], c["by_token"]).transpose(1, 2), rows(s["x"], c["x_by_token"]))
    if c["base"]:
        dw = dw + s["base"].float()
    return {"dw": dw.to(s["out"].dtype)}


# ---------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route_backward":
        # through the matrix of derivatives dw_j / dl_m = w_j ([j is m] - w_m), of the chosen or of all
        T, E = c["T"], c["E"]
        l = s["logits"].double()
        chosen = torch.zeros((T, E), dtype=torch.bool, device="cuda")
        chosen[torch.arange(T, device="cuda")[:, None], s["ids"].long()] = True
        q = torch.softmax(torch.where(chosen, l, -math.inf) if c["renormalize"] else l, 1)
        d = torch.zeros((T, E), dtype=torch.float64, device="cuda")
        d[torch.arange(T, device="cuda")[:, None], s["ids"].long()] = s["dw"].double()
        return {"dlogits": q * d - q * (q * d).sum(1)[:, None]}
    a = s["a"]
    real = torch.nonzero(a["sorted"] < a["P"]).reshape(-1)
    pair = a["sorted"][real].long()
    if c["op"] in ("dropout", "act_backward"):
        keep = _exact_keep(s["rng"], pair, c["I"], c["p"])
        g, u = s["g"][real].double(), s["u"][real].double()
        silu = g * torch.sigmoid(g)
        h = silu * u * keep

        def full(v):
            out = torch.zeros((a["mp"], c["I"]), dtype=torch.float64, device="cuda")
            out[real] = v
            return out
        if c["op"] == "dropout":
            return {"h": full(h)}
        d = s["d"][real].double()
        w = a["w"].reshape(-1)[pair].double()[:, None]
        slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
        dw = torch.zeros(a["P"], dtype=torch.float64, device="cuda")
        dw[pair] = (h * d).sum(1)
        return {"dg": full(w * d * keep * u * slope), "du": full(w * d * keep * silu), "h": full(w * h),
                "dw": dw.view(c["T"], c["k"])}
    off, counts = a["off"].tolist(), a["counts"].tolist()
    tok = torch.div(a["sorted"].long(), a["k"], rounding_mode="floor")
    if c["op"] == "dgrad":
        y = torch.zeros((a["mp"], c["K"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            r = slice(off[e], off[e] + counts[e])
            take = tok[r] if c["by_token"] else r
            for dy, w in (("dy", "w"), ("dy1", "w1")):
                if dy in s:
                    y[r] += s[dy][take].double() @ s[w][e].double()
        return {"dx": y}
    dw = torch.zeros((c["E"], c["N"], c["K"]), dtype=torch.float64, device="cuda")
    for e in range(c["E"]):
        r = slice(off[e], off[e] + counts[e])
        dy = s["dy"][tok[r] if c["by_token"] else r].double()
        dw[e] = dy.t() @ s["x"][tok[r] if c["x_by_token"] else r].double()
        if c["base"]:
            dw[e] += s["base"][e].double()
    return {"dw": dw}


def _exact_keep(rng, pairs, I, p):
    """The generator again on the host, in unsigned 64-bit words, pair by pair of the sorted order."""
    below = _dropped_below(p)
    if not below:
        return 1.0
    seed, offset = (int(v) for v in rng.tolist())
    n = -(-I // 8)
    out = np.empty((len(pairs), n, 8), dtype=np.uint16)
    pairs = pairs.cpu().numpy().astype(np.uint64)
    u, low = np.uint64, np.uint64(_LOW)
    for lo in range(0, len(pairs), 4096):
        some = pairs[lo:lo + 4096, None]
        x = [np.broadcast_to(np.arange(n, dtype=u), (len(some), n)), np.broadcast_to(some, (len(some), n)),
             u(offset & _LOW), u(offset >> 32)]
        for i in range(10):
            key = u((seed + i * 0x9E3779B9) & _LOW), u(((seed >> 32) + i * 0xBB67AE85) & _LOW)
            p0, p1 = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
            x = [(p1 >> u(32)) ^ x[1] ^ key[0], p1 & low, (p0 >> u(32)) ^ x[3] ^ key[1], p0 & low]
        for i in range(4):
            out[lo:lo + 4096, :, 2 * i] = x[i] & u(0xFFFF)
            out[lo:lo + 4096, :, 2 * i + 1] = x[i] >> u(16)
    kept = torch.from_numpy((out >= below).reshape(len(pairs), 8 * n)[:, :I].copy()).to("cuda")
    return kept.double() / (1 - below / 65536)


# ------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "route_backward":
        n = c["T"] * c["E"]
        return {"bytes": 4 * n * (1 if c["renormalize"] else 2) + 12 * c["T"] * c["k"], "flops": 4 * n}
    P = c["T"] * c["k"]
    if c["op"] in ("dropout", "act_backward"):
        n = P * c["I"]
        return ({"bytes": 6 * n + 4 * P, "flops": 6 * n} if c["op"] == "dropout" else
                {"bytes": 12 * n + 12 * P, "flops": 16 * n})
    N, K, E, k, T = c["N"], c["K"], c["E"], c["k"], c["T"]
    active = E * (1 - (1 - k / E) ** T) if not c["skew"] else min(E, P)  # experts that random choices reach
    dy = 2 * N * (T if c["by_token"] else P)
    if c["op"] == "dgrad":
        pairs = 2 if c["pair"] else 1
        return {"bytes": pairs * (dy + 2 * active * N * K) + 2 * P * K, "flops": 2 * pairs * P * N * K}
    size = (4 if c["out"] == "fp32" else 2) * E * N * K
    return {"bytes": dy + 2 * K * (T if c["x_by_token"] else P) + size * (2 if c["base"] else 1),
            "flops": 2 * P * N * K}
