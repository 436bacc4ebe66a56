"""The grouped gradient products' lists and LDS addresses as the kernel has them: the functions are taken out of its source,
compiled for the CPU and held against the model of ``test_training_addressing`` and against what they are for."""
import ctypes
import itertools
import re
import subprocess

import numpy as np
import pytest

import test_training_addressing as model
from test_training_addressing import SRC, TILE, BAND, TAB, MAX_PIECES, MAX_SPLIT, MIN_PIECE, WAVES, up

BEGIN, END = "// ---- Lists of tiles and addresses in LDS", "// ---- (end)"
I = ctypes.c_int
LANES, BLOCKS = range(64), range(8)


@pytest.fixture(scope="module")
def f(tmp_path_factory):
    """The functions by name, each on ints; those with results behind references return a tuple."""
    where = tmp_path_factory.mktemp("schedule")
    constants = "\n".join(re.findall(r"^constexpr int .*;", SRC, flags=re.M))
    part = SRC[SRC.index(BEGIN):SRC.index(END)]
    code = f"""
#include <cstdint>
#define __host__
#define __device__
#define __forceinline__ inline
{constants}
{part}
extern "C" {{
void units(int tiles_e, int tiles, int* out) {{ units_of(tiles_e, tiles, out[0], out[1]); }}
void tile(int idx, int row_tiles, int n_tiles, int* out) {{ tile_of(idx, row_tiles, n_tiles, out[0], out[1]); }}
int round_(int v, int xcd) {{ return unit_of_round(v, xcd); }}
int pieces(int T, int grid, int most) {{ return pieces_of(T, grid, most); }}
int64_t per_xcd(int64_t tiles, int64_t entries, int ws, int cus) {{ return per_xcd_for(tiles, entries, ws != 0, cus); }}
int column_load(int wave, int lane, int q) {{ return column_loaded(wave, lane, q); }}
int column_fragment(int lane, int block) {{ return column_read(lane, block); }}
int row_load(int lane) {{ return row_loaded(lane); }}
int row_fragment(int lane, int wm) {{ return row_read(lane, wm); }}
int stage(int row, int chunk) {{ return staged(row, chunk); }}
}}
"""
    (where / "schedule.cpp").write_text(code)
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-o", where / "schedule.so", where / "schedule.cpp"], check=True, timeout=60)
    L = ctypes.CDLL(str(where / "schedule.so"))
    L.per_xcd.argtypes, L.per_xcd.restype = [ctypes.c_int64, ctypes.c_int64, I, I], ctypes.c_int64

    def two(name):
        out = (I * 2)()

        def call(*a):
            getattr(L, name)(*a, out)
            return out[0], out[1]
        return call
    L.units_, L.tile_ = two("units"), two("tile")
    return L


def test_the_kernel_uses_them():
    part = SRC[SRC.index(BEGIN):SRC.index(END)]
    rest = SRC.replace(part, "")
    names = re.findall(r"__forceinline__ \w+ (\w+)\(", part)
    assert len(names) == 10
    for n in names:
        assert re.search(rf"\b{n}\(", rest), n


def test_units(f):
    rng = np.random.default_rng(0)
    for tiles_e, E in itertools.chain([(1, 1), (32, 1), (33, 8), (3584, 8), (16, 128)], zip(rng.integers(1, 4000, 400), rng.integers(1, 257, 400))):
        unit, units_e = f.units_(int(tiles_e), int(tiles_e * E))
        assert (unit, units_e) == model.units_of(int(tiles_e), int(tiles_e * E))
        assert unit <= 32 and units_e * unit >= tiles_e   # no tile without a unit
    for rounds in (1, 2, 7):
        seen = sorted(f.round_(v, x) for v in range(rounds) for x in range(8))
        assert seen == list(range(8 * rounds))


@pytest.mark.parametrize("row_tiles,n_tiles", [(1, 1), (3, 1), (4, 7), (5, 3), (9, 130), (56, 16), (257, 2)])
def test_tiles(f, row_tiles, n_tiles):
    got = [f.tile_(i, row_tiles, n_tiles) for i in range(row_tiles * n_tiles)]
    assert got == [model.order(i, row_tiles, n_tiles) for i in range(row_tiles * n_tiles)]
    assert sorted(got) == sorted(itertools.product(range(row_tiles), range(n_tiles)))
    assert all(m // BAND == got[0][0] // BAND for m, _ in got[:min(BAND, row_tiles) * n_tiles])


def test_pieces(f):
    for T in [0, 1, 2, 3, 7, 16, 31, 64, 85, 127, 128, 129, 200, 256, 300, 5000]:
        for grid in (8, 64, 256, 304, 4096):
            for most in (0, 1, 15, 16, 31, 32, 100, 128, 900):
                n = f.pieces(T, grid, most)
                want = 1
                if T > 0 and 2 * T <= grid:
                    want = max(min(min(grid, MAX_PIECES) // T, MAX_SPLIT, most // MIN_PIECE), 1)
                assert n == want
                assert n == 1 or (n * T <= min(grid, MAX_PIECES) and most >= n * MIN_PIECE)   # a workgroup and a slot each


def test_workgroups(f):
    rng = np.random.default_rng(1)
    for _ in range(400):
        tiles, cus = int(2 ** rng.uniform(0, 28)), int(rng.choice([8, 64, 256, 304]))
        entries = up(tiles, 8) * int(rng.integers(1, 3))
        for ws in (0, 1):
            n = f.per_xcd(tiles, entries, ws, cus)
            assert n * 8 == model.grid_for(tiles, entries, ws, cus)
            assert n >= 1 and n * TAB >= entries   # every list fits its tables


def test_columns(f):
    place = {w * 2048 + q * 1024 + lane * 16: (w * 4 + q * 2 + (lane >> 5), f.column_load(w, lane, q))
             for w in range(WAVES) for q in range(2) for lane in LANES}
    assert place == model.slot_by_columns()
    for block in BLOCKS:
        for lane in LANES:
            at = f.column_fragment(lane, block)
            assert at == model.tr_off(block, lane)
            row, col = place[at & ~15]      # 8 bytes of contraction row lane / 16 * 8 + lane % 16 / 4, for the transposing read
            assert (row, col + (at & 15) // 2) == ((lane >> 4) * 8 + (lane & 15) // 4, block * 16 + (lane & 3) * 4)


def test_rows(f):
    place = {w * 2048 + q * 1024 + lane * 16: (w * 32 + q * 16 + (lane >> 2), f.row_load(lane))
             for w in range(WAVES) for q in range(2) for lane in LANES}
    assert len(set(place.values())) == TILE * 4
    for wm in range(4):
        for i in range(4):
            for lane in LANES:
                assert place[f.row_fragment(lane, wm) + i * 4096] == (i * 64 + wm * 16 + (lane & 15), (lane >> 4) * 8)


def test_results_on_their_way_out(f):
    at = {(r, c): f.stage(r, c) for r in range(16) for c in range(4)}
    assert sorted(at.values()) == list(range(0, 1024, 16))
    assert all(v // 64 == r for (r, _), v in at.items())
    # 16-byte accesses go 16 lanes at a time, through all 64 banks once: a chunk of 16 rows in, 4 whole rows out
    for some in [[(r, c) for r in range(16)] for c in range(4)] + [[(r, c) for r in range(r0, r0 + 4) for c in range(4)] for r0 in range(0, 16, 4)]:
        assert sorted((at[i] // 4 + w) % 64 for i in some for w in range(4)) == list(range(64))
