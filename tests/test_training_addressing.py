"""The grouped gradient products' lists, slots and offsets on a CPU model: every tile is computed once, by a workgroup
whose table holds it; every half of a contraction is loaded once, zeros past its end; the loads fill a slot and the
matrix operands that leave it are the elements that the products need; every result leaves for its own place.  The
constants are read from the source."""
import os
import re

import numpy as np
import pytest

from _util import ROOT

SRC = open(os.path.join(ROOT, "mixture_experts_routed_route_amd", "csrc", "grad_gemm.hip")).read()


def const(name):
    return int(re.search(rf"constexpr int {name} = (\d+);", SRC).group(1))


TILE, BK, SLOTS, BAND, TAB = (const(n) for n in ("kTile", "kBK", "kSlots", "kBand", "kTab"))
MAX_PIECES, MAX_SPLIT, MIN_PIECE, SEGS = (const(n) for n in ("kMaxPieces", "kMaxSplit", "kMinPiece", "kSegs"))
WAVES = const("kNT") // 64
PART = TILE * BK * 2
up = lambda a, b: -(-a // b)


def test_constants():
    assert (TILE, BK, WAVES, PART) == (256, 32, 8, 16384)   # what the model below is written for
    assert re.search(r"kPartB = kTile \* kBK \* 2;", SRC) and re.search(r"kSlotB = 2 \* kPartB;", SRC)


# ------------------------------------------------------------------ lists of tiles
def units_of(tiles_e, tiles):
    units_e = up(tiles_e, 32)
    if tiles < 2048:
        per = 1 if tiles < 128 else tiles // 64
        units_e = min(max(units_e, tiles_e // per), tiles_e)
    return up(tiles_e, units_e), units_e


def grid_for(tiles, entries, ws, cus=256):
    most, want = cus // 8, up(tiles, 8)
    n = most if ws or want > most else want
    if entries > n * TAB:
        n = up(entries, TAB)
    return n * 8


def order(idx, rows_all, n_tiles):
    band = idx // (BAND * n_tiles)
    at = idx - band * BAND * n_tiles
    rows = min(BAND, rows_all - band * BAND)
    return band * BAND + at % rows, at // rows


def run_dgrad(spans, N, K, pair, P, ws):
    """(row tile start, row tile end, column tile, first half, halves) of every tile or piece, per workgroup."""
    E, n_tiles = len(spans), up(K, TILE)
    max_pad = max((hi for _, hi in spans), default=0)
    host = (max_pad // TILE + min(P, E)) * n_tiles
    grid = grid_for(host, up(host, 8), ws)
    row_tiles = [(lo + i * TILE, min(lo + (i + 1) * TILE, hi), e) for e, (lo, hi) in enumerate(spans) for i in range(up(hi - lo, TILE))]
    T, all_nh = len(row_tiles) * n_tiles, up(N, BK) * (2 if pair else 1)
    assert T <= host
    out = []
    pieces = 1
    if ws and T > 0 and 2 * T <= grid:
        pieces = max(min(min(grid, MAX_PIECES) // T, MAX_SPLIT, all_nh // MIN_PIECE), 1)
    for b in range(grid):
        mine = []
        if pieces > 1:
            if b // T < pieces:
                j = b // T
                m, n = order(b % T, len(row_tiles), n_tiles)
                h0, h1 = all_nh * j // pieces, all_nh * (j + 1) // pieces
                mine.append((*row_tiles[m], n, h0, h1 - h0))
        else:
            xcd, slot = b & 7, b >> 3
            lo, hi = T * xcd // 8, T * (xcd + 1) // 8
            for i in range(lo + slot, hi, grid >> 3):
                m, n = order(i, len(row_tiles), n_tiles)
                mine.append((*row_tiles[m], n, 0, all_nh))
        assert len(mine) <= TAB
        out.append(mine)
    return out, row_tiles, n_tiles, all_nh, pieces, T


def run_wgrad(spans, N, K, ws):
    E, n_tiles, r_tiles = len(spans), up(K, TILE), up(N, TILE)
    tiles_e = n_tiles * r_tiles
    T = E * tiles_e
    unit, units_e = units_of(tiles_e, T)
    grid = grid_for(T, up(E * units_e, 8) * unit, ws)
    halves = [up(hi - lo, BK) for lo, hi in spans]
    by_length = sorted(range(E), key=lambda e: (-(spans[e][1] - spans[e][0]), e))
    pieces = 1
    if ws and 2 * T <= grid:
        pieces = max(min(min(grid, MAX_PIECES) // T, MAX_SPLIT, halves[by_length[0]] // MIN_PIECE), 1)
    out = []
    for b in range(grid):
        mine = []
        if pieces > 1:
            if b // T < pieces:
                j, e = b // T, b % T // tiles_e
                m, n = order(b % T % tiles_e, r_tiles, n_tiles)
                h0, h1 = halves[e] * j // pieces, halves[e] * (j + 1) // pieces
                r0 = spans[e][0] + h0 * BK
                mine.append((e, m, n, r0, min(spans[e][1], r0 + (h1 - h0) * BK)))
        else:
            xcd, slot, per_xcd = b & 7, b >> 3, grid >> 3
            entries = range(slot, up(E * units_e, 8) * unit, per_xcd)
            assert len(entries) <= TAB
            for i in entries:
                v, j = divmod(i, unit)
                u = v * 8 + (7 - xcd if v & 1 else xcd)
                idx = u % units_e * unit + j
                if u < E * units_e and idx < tiles_e:
                    e = by_length[u // units_e]
                    m, n = order(idx, r_tiles, n_tiles)
                    mine.append((e, m, n, *spans[e]))
            lengths = [hi - lo for *_, lo, hi in mine]
            assert all(a >= c for a, c in zip(lengths, lengths[1:]))   # tiles without halves come last
        out.append(mine)
    return out, T, pieces, r_tiles, n_tiles


def some_spans(rng, E, most, bs=16):
    n = rng.integers(0, most, E) * (rng.random(E) < 0.7)
    off = np.concatenate([[0], np.cumsum(-(-n // bs) * bs)])
    return [(int(off[e]), int(off[e + 1])) for e in range(E)]


LISTS = [(1, 40, 16, 8), (3, 900, 264, 2056), (8, 1100, 4096, 14336), (64, 300, 1408, 4096), (128, 3000, 768, 2048),
         (256, 20, 8, 33032), (256, 40, 1408, 2048), (5, 700, 14336, 8), (2, 9000, 1024, 1024), (7, 60, 4104, 40), (17, 9000, 2048, 1032)]


@pytest.mark.parametrize("E,most,N,K", LISTS)
@pytest.mark.parametrize("ws", [False, True])
def test_every_tile_once(E, most, N, K, ws):
    rng = np.random.default_rng(E + N)
    for _ in range(2):
        spans = some_spans(rng, E, most)
        for pair in (False, True):
            lists, row_tiles, n_tiles, all_nh, pieces, T = run_dgrad(spans, N, K, pair, 1 << 20, ws)
            seen = {}
            for mine in lists:
                for lo, hi, e, n, h0, nh in mine:
                    assert nh > 0 and spans[e][0] <= lo < hi <= spans[e][1]
                    seen.setdefault((lo, n), []).append((h0, nh))
            assert len(seen) == T
            for parts in seen.values():
                parts.sort()
                assert parts[0][0] == 0 and sum(nh for _, nh in parts) == all_nh and len(parts) == pieces
                assert all(a + n == b for (a, n), (b, _) in zip(parts, parts[1:]))
        lists, T, pieces, r_tiles, n_tiles = run_wgrad(spans, N, K, ws)
        seen = {}
        for mine in lists:
            for e, m, n, lo, hi in mine:
                assert m < r_tiles and n < n_tiles
                seen.setdefault((e, m, n), []).append((lo, hi))
        assert len(seen) == T
        for (e, _, _), parts in seen.items():
            parts.sort()
            covered = [r for lo, hi in parts for r in range(lo, hi)]
            assert covered == list(range(*spans[e])) and len(parts) == pieces


# ------------------------------------------------------------------ the issuing cursor of dgrad
@pytest.mark.parametrize("N", [8, 24, 32, 40, 64, 72, 520, 1000])
@pytest.mark.parametrize("pair", [False, True])
def test_halves_of_a_contraction(N, pair):
    """From every first half on: the n that a half's rows of W hold, zeros past N, both pairs in turn."""
    nkh = up(N, BK)
    all_nh = nkh * (2 if pair else 1)
    for first in range(0, all_nh, max(1, all_nh // 5)):
        nh, i_h, got, w = all_nh - first, 0, [], None
        while i_h < nh:
            at = first + i_h
            second, h = at >= nkh, at - nkh if at >= nkh else at
            if i_h == 0 or h == 0:
                w = [second, h * BK]                     # the pointers are set anew, else they have moved on by themselves
            left = min(N // BK - h, nh - i_h)
            whole = left > 0
            left = left if whole else 1
            for _ in range(left):
                assert w[0] == second
                got += [(w[0], n) for n in range(w[1], w[1] + BK) if whole or n < N]
                assert not whole or w[1] + BK <= N
                w[1] += BK
            i_h += left
        want = [(p, n) for p in range(1 + pair) for n in range(N)]
        assert got == [x for x in want if x[0] * nkh + x[1] // BK >= first]


# ------------------------------------------------------------------ a slot
def slot_by_columns():
    """What the loads of a half put into an operand that is read by columns: (contraction row, first column) of the 16
    bytes at each 16-byte place."""
    place = {}
    for wave in range(WAVES):
        for q in range(2):
            for lane in range(64):
                row = wave * 4 + q * 2 + (lane >> 5)
                bit = ((wave >> 1) ^ (wave >> 2)) & 1
                chunk = (lane & 31) ^ (((q * 2 + (lane >> 5)) << 2) | (bit << 1))
                at = wave * 2048 + q * 1024 + lane * 16
                assert at not in place
                place[at] = (row, chunk * 8)
    assert sorted(place) == list(range(0, PART, 16))
    assert sorted(place.values()) == [(r, c) for r in range(BK) for c in range(0, TILE, 8)]
    return place


def tr_off(block, lane):
    i16, gr = lane & 15, lane >> 4
    row, bit = gr * 8 + (i16 >> 2), (gr ^ (gr >> 1)) & 1
    return row * 512 + (((((block >> 1) ^ (i16 >> 2)) << 2) | (((block & 1) ^ bit) << 1) | ((i16 & 3) >> 1)) << 4) + (i16 & 1) * 8


def banks(addresses, width):
    """Lanes of a half wave touch each of the 64 4-byte banks at most once."""
    for half in (addresses[:32], addresses[32:]):
        used = [(a // 4 + i) % 64 for a in half for i in range(width // 4)]
        assert len(set(used)) == len(used)


def test_column_operand_leaves_the_slot():
    place = slot_by_columns()
    for wave in range(WAVES):
        for j in range(8):                                  # blocks of 16 columns of the wave
            block = ((j >> 1) & 1) * 4 + (wave & 1) * 2 + (j & 1)
            extra = (j >> 2) * 256
            for hi in (0, 4):                               # contraction rows +0..3 and +4..7 of each lane group
                loaded = []
                for lane in range(64):
                    at = tr_off(block, lane) + extra + hi * 512
                    row, col = place[at & ~15]
                    loaded.append([(row, col + (at & 15) // 2 + c) for c in range(4)])
                banks([tr_off(block, lane) + extra + hi * 512 for lane in range(64)], 8)
                for lane in range(64):
                    i, g = lane & 15, lane >> 4
                    got = [loaded[g * 16 + 4 * r + i // 4][i % 4] for r in range(4)]   # what the transposing read returns
                    column = (j // 2) * 64 + (wave & 1) * 32 + (j % 2) * 16 + i
                    assert got == [(g * 8 + hi + r, column) for r in range(4)]


def test_row_operands_leave_the_slot():
    by_columns = slot_by_columns()
    place = {}
    for wave in range(WAVES):
        for q in range(2):
            for lane in range(64):
                row = wave * 32 + q * 16 + (lane >> 2)
                place[wave * 2048 + q * 1024 + lane * 16] = (row, ((lane & 3) ^ ((lane >> 4) & 3)) * 8)
    assert sorted(place.values()) == [(r, k) for r in range(TILE) for k in range(0, BK, 8)]
    for wave in range(WAVES):
        wm = wave >> 1
        for i in range(4):
            at = [(wm * 16 + (lane & 15)) * 64 + (((lane >> 4) ^ ((lane & 15) >> 2)) << 4) + i * 4096 for lane in range(64)]
            for lane in range(64):                          # dgrad: 8 contraction indices of a row, 16 bytes
                assert place[at[lane]] == (i * 64 + wm * 16 + (lane & 15), (lane >> 4) * 8)
            for quarter in range(4):                        # (16-byte reads go 16 lanes at a time)
                used = [(a // 4 + w) % 64 for a in at[quarter * 16:quarter * 16 + 16] for w in range(4)]
                assert len(set(used)) == 64
            for lane in range(64):                          # wgrad: as the column operand
                a = tr_off((i & 1) * 4 + wm, lane) + (i >> 1) * 256
                row, col = by_columns[a & ~15]
                assert (row, col + (a & 15) // 2) == ((lane >> 4) * 8 + ((lane & 15) >> 2), i * 64 + wm * 16 + (lane & 3) * 4)


# ------------------------------------------------------------------ results
@pytest.mark.parametrize("size", [2, 4])
def test_results_leave_for_their_places(size):
    """A wave's accumulators through its 1 KB of LDS: each value at its row and column, once, whole 64-byte pieces."""
    seen = np.zeros((TILE, TILE), int)
    for wave in range(WAVES):
        em, en = wave >> 1, wave & 1
        for i in range(4):
            for q in range(8 if size == 4 else 4):          # pieces of 16 rows x 64 bytes
                stage = {}
                for lane in range(64):
                    br, bg = lane & 15, lane >> 4
                    for b in range(1 if size == 4 else 2):
                        block = q if size == 4 else 2 * q + b
                        chunk, off = (bg, 0) if size == 4 else (2 * b + (bg >> 1), (bg & 1) * 8)
                        at = br * 64 + ((chunk ^ (br >> 2)) * 16) + off
                        col = (block // 2) * 64 + en * 32 + (block % 2) * 16 + bg * 4
                        for v in range(4):
                            assert at + v * size not in stage
                            stage[at + v * size] = (i * 64 + em * 16 + br, col + v)
                assert len(stage) == 1024 // size
                for lane in range(64):
                    sr = lane >> 2
                    at = sr * 64 + ((lane & 3) ^ (sr >> 2 & 3)) * 16
                    got = [stage[at + v] for v in range(0, 16, size)]
                    col0 = en * 32 + (lane & 3) * (16 // size)
                    col = col0 + ((q >> 1) * 64 + (q & 1) * 16 if size == 4 else q * 64)
                    assert got == [(i * 64 + em * 16 + sr, col + v) for v in range(16 // size)]
                    for r, c in got:
                        seen[r, c] += 1
    assert (seen == 1).all()


# ------------------------------------------------------------------ slots in time
@pytest.mark.parametrize("group", [0, 1])
def test_slots_are_read_before_they_are_filled_again(group):
    """The two groups alternate between reading a half and computing it, a barrier after each; group 0 issues 3 halves
    ahead while it computes, group 1 4 halves ahead.  A slot's last read by either group lies in an earlier phase than
    the first load into it, and loads are awaited at a barrier before either group reads them."""
    read_phase = lambda g, h: 2 * h + g                     # phases are numbered by barriers
    compute_phase = lambda g, h: 2 * h + 1 + g
    ahead = 3 + group
    for h in range(ahead, 200):
        issued = compute_phase(group, h - ahead)
        if h >= SLOTS:
            assert max(read_phase(g, h - SLOTS) for g in (0, 1)) < issued
        # The barrier that ends a phase: group 0 waits in the compute phase of h - 1, group 1 in the read phase of h - 1
        waited = compute_phase(0, h - 1) if group == 0 else read_phase(1, h - 1)
        assert issued < waited
        # with the loads of two later halves in flight, 4 each, vmcnt(8): no more than those may have been issued by then
        newest = h - 1 + ahead - (0 if group == 0 else 1)
        assert newest - h == 2
        assert waited < min(read_phase(g, h) for g in (0, 1))
