"""CPU model of the addressing of the layer for a few tokens (few_tokens.hip): the work list, the
granules each wave walks, the token rows in LDS and memory, h's two planes and the partial panels.  The
model restates the kernels' integer arithmetic; the tests show every index in bounds and every
(group, column panel, granule) multiplied exactly once.  CPU only."""
import ctypes
import itertools

import numpy as np
import pytest

import mixture_experts_routed_route_amd as m

MAX_E, GROUPS, TOKENS, TOPK, NO_TOKEN = 256, 256 + 64, 32, 32, 0x8000
TYPES = {"bf16": 0, "int4": 1, "fp8": 2, "fp8_block": 3}
LDS = 160 * 1024


def shape(kind, group, src):
    """(columns of a panel, k of a granule, waves of a workgroup) of a stream."""
    if kind == "int4":
        steps = {32: 1, 64: 2}.get(group, 2 if src == "row" else 4)
        cols, unit = 64, 32 * steps
    else:
        steps = 1
        us = 2 if kind != "bf16" else 4 if src == "tile" else 3
        cols, unit = 32, (32 if kind == "bf16" else 64) * us
    return cols, unit, 16 if src != "pair" else 8 if steps == 4 else 12


def work_list(ids, E):
    """act [(expert, rows)] and pair [group][16] from ids [T, k], as list_active builds them."""
    T, k = ids.shape
    tok = [0] * E
    for t, j in itertools.product(range(T), range(k)):
        tok[ids[t, j]] |= 1 << t
    act, base = [], {}
    for e in range(E):
        n = bin(tok[e]).count("1")
        f = (n + 15) // 16
        if f:
            base[e] = len(act)
            act += [(e, min(n, 16))] + ([(e, n - 16)] if f > 1 else [])
    assert len(act) <= GROUPS and all(e + MAX_E * rows < 1 << 16 for e, rows in act)
    cleared = min(T * k, GROUPS)
    assert len(act) <= cleared                      # every group's rows were set to "none" before
    pair = [[NO_TOKEN] * 16 for _ in range(cleared)]
    for t, j in itertools.product(range(T), range(k)):
        e = ids[t, j]
        rank = bin(tok[e] & ((1 << t) - 1)).count("1")
        g = base[e] + rank // 16
        assert act[g][0] == e and rank % 16 < act[g][1] and pair[g][rank % 16] == NO_TOKEN
        pair[g][rank % 16] = t + TOKENS * j
    assert sum(p != NO_TOKEN for row in pair for p in row) == T * k
    return act, pair


def routing(rng, T, E, k, how):
    if how == "same":          # every token the same experts: groups of up to 32 tokens
        return np.tile(np.arange(E - k, E), (T, 1))
    if how == "skewed":
        p = 1.0 / np.arange(1, E + 1) ** 2
        return np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)])
    return np.stack([rng.permutation(E)[:k] for _ in range(T)])


CASES = [(1, 64, 6, 2048, 1408), (16, 64, 6, 2048, 1408), (32, 64, 8, 4096, 1408), (23, 128, 8, 2048, 768),
         (32, 256, 32, 64, 64), (17, 3, 3, 256, 128), (32, 8, 8, 512, 256), (5, 6, 3, 8448, 64), (32, 40, 32, 256, 256)]


@pytest.mark.parametrize("kind,group", [("bf16", 0), ("int4", 32), ("int4", 64), ("int4", 128), ("int4", 256),
                                        ("fp8", 0), ("fp8_block", 0)])
@pytest.mark.parametrize("T,E,k,H,I", CASES)
def test_few_tokens_addressing(kind, group, T, E, k, H, I):
    step = max(64, group) if kind == "int4" else 8 if kind == "bf16" else 16
    H, I = -(-H // step) * step, -(-I // step) * step
    need = m.lib().moe_few_tokens_workspace_bytes(T, E, k, H, I, TYPES[kind])
    es = 2 if kind == "bf16" else 1
    rng = np.random.default_rng(T + E)
    for how in ("random", "skewed", "same"):
        act, pair = work_list(routing(rng, T, E, k, how), E)

        # ---- gate/up: panels of one group per workgroup, the wave pairs' shares of K
        cols, unit, _ = shape(kind, group, "tile")
        kpad = -(-H // unit) * unit
        routed = 4 * MAX_E + 2 * TOKENS * TOPK + 2 * MAX_E + 2 * GROUPS + 32 * GROUPS + 17 * 4
        x_bytes = LDS - 256 - routed - 16 * (cols // 16) * 1024
        src = "tile" if T * kpad * 2 <= x_bytes else "row"
        cols, unit, waves = shape(kind, group, src)
        grans, parts, panels = -(-H // unit), waves // 2, -(-I // cols)
        shares = [(w * grans // parts, (w + 1) * grans // parts) for w in range(parts)]
        assert [g for lo, hi in shares for g in range(lo, hi)] == list(range(grans))
        if src == "tile":
            # fragment by fragment, quarter wave by quarter wave, token by token; 16 bytes each
            top = ((kpad // 32 - 1) * 4 + 3) * T + T - 1
            assert (top + 1) * 16 <= x_bytes
            for row in pair[: len(act)]:
                assert all(p % TOKENS < T for p in row)    # rows past the group read token 0
        for e, rows in act:
            assert 0 <= e < E and 1 <= rows <= 16
        if kind == "int4":
            words = H // 8 * I
            assert ((grans - 1) * (unit // 8) + (unit // 32 - 1) * 4 + 3) * I + (panels - 1) * cols + 64 <= words + cols
            assert grans * unit == H and (unit <= group or unit % group == 0)
        else:
            # 16 bytes at k < K of rows n < N: the last one ends with the matrix
            assert H * es % 16 == 0 and (I - 1) * H * es + (H * es - 16) + 16 == I * H * es < 1 << 31
        if kind == "fp8_block":
            assert (panels - 1) * cols // 128 < -(-I // 128) and 128 % cols == 0
            assert (grans - 1) * unit // 128 < -(-H // 128) and 128 % unit == 0
        # h: two planes of [T * k, I], CPL columns at a time
        plane = T * k * I
        for row in pair[: len(act)]:
            for p in row:
                if p != NO_TOKEN:
                    assert (p % TOKENS * k + p // TOKENS) * I + I <= plane

        # ---- down: equal shares of the granules of all groups, split over the workgroups of a panel
        cols, unit, waves = shape(kind, group, "pair")
        assert waves * 64 >= TOKENS * 16 and waves * TOKENS * cols * 4 + routed + 4 * TOKENS * TOPK + 64 <= LDS
        grans, panels = -(-I // unit), -(-H // cols)
        most = min(T * k, E)
        splits = max(1, min(-(-256 // panels), most, 16))
        total = len(act) * grans
        cut = [total * w // (splits * waves) for w in range(splits * waves + 1)]
        assert cut[0] == 0 and cut[-1] == total and all(a <= b for a, b in zip(cut, cut[1:]))
        assert panels * 4 <= 65536 // 32 * 4
        hs_at = 65536 // 32 * 4 + (-(-panels * splits * T * cols * 4 // 256) * 256 if splits > 1 else 0)
        assert need == hs_at + -(-T * k * I * 4 // 256) * 256
        # the last cell of the last workgroup's partial panel ends with the area
        assert ((panels * splits - 1) * T * 16 + T * 16) * (cols // 16) * 4 <= max(hs_at - 8192, panels * T * cols * 4)


def test_groups_never_exceed_the_list():
    """T * k = 1024 pairs over 256 experts: as many experts as can be with 17 tokens, the others with one."""
    ids = -np.ones((32, 32), dtype=int)
    full = 59                                          # experts of 17 tokens
    left = [32] * 32
    for e in range(full):
        for t in sorted(range(32), key=lambda t: -left[t])[:17]:
            ids[t, 32 - left[t]] = e
            left[t] -= 1
    nxt = full
    for t in range(32):
        while left[t]:
            ids[t, 32 - left[t]] = nxt
            nxt += 1
            left[t] -= 1
    assert nxt <= 256
    act, _ = work_list(ids, 256)
    assert len(act) == nxt + full <= GROUPS
