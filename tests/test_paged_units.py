"""How the chunk kernel cuts a batch into units, pieces and shares (csrc/paged_math.h, compiled for
the host; no GPU), against counting row by row."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_opt_decode_b200", "csrc")
ROWS, TILE = 256, 128


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_units")
    (d / "u.cpp").write_text(
        '#include "paged_math.h"\nusing namespace flexq;\nextern "C" {\n'
        "int units(int n, int g) { return row_units(n * g); }\n"
        "int rows(int n, int g, int c0) { return unit_rows(n * g, c0); }\n"
        "int tiles(int f, int g, int c0, int r) { return unit_tiles(f, g, c0, r); }\n"
        "int longs(int f, int n, int g, int t) { return long_units(f, n, g, row_units(n * g), t); }\n"
        "int none() { return long_units(0, 0, 1, 0, 1) + long_units(500, 0, 1, 0, 1) + long_units(-3, 3, 1, 0, 2); }\n"
        "int share(int t, int r, int s) { return share_tiles(t, r, s); }\n"
        "long long total(int r, int b, int g) { return unit_total(r, b, g, kUnitRowShift, 1); }\n"
        "int limits() { return kUnitRows * 1000 + kKeyTile; }\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=all", "-I" + CSRC, str(d / "u.cpp"), "-o", str(d / "u.so")], check=True)
    so = C.CDLL(str(d / "u.so"))
    so.total.restype = C.c_longlong
    return so


def test_sizes(lib):
    assert lib.limits() == ROWS * 1000 + TILE


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 16, 20, 56, 255, 256, 300])
def test_units_hold_every_row_and_tile_and_the_long_ones_are_the_last(lib, group):
    rng = np.random.default_rng(group)
    for n in list(range(1, 40)) + [127, 128, 129, 255, 256, 257, 511, 513] + rng.integers(1, 3000, 20).tolist():
        for first in [0, 1, 126, 127, 128, 129, 255, 256, 1000] + rng.integers(0, 5000, 6).tolist():
            units = lib.units(n, group)
            c0 = np.arange(units) * ROWS
            rows = [lib.rows(n, group, int(c)) for c in c0]
            assert sum(rows) == n * group and min(rows) > 0 and max(rows) <= ROWS
            last_pos = first + (c0 + rows - 1) // group  # position of each unit's last row
            tiles = np.array([lib.tiles(first, group, int(c), r) for c, r in zip(c0, rows)])
            assert (tiles == last_pos // TILE + 1).all()
            assert (np.diff(tiles) >= 0).all()
            for t in sorted({1, 2, 3, 16, 48, int(tiles[0]), int(tiles[-1]), int(tiles[-1]) + 1, int(np.median(tiles))}):
                longs = lib.longs(first, n, group, t)
                assert longs == (tiles >= t).sum(), (n, first, t)
    assert lib.none() == 0


def test_batches_have_no_more_units_than_the_launch_counts(lib):
    rng = np.random.default_rng(0)
    for _ in range(500):
        b, group = int(rng.integers(1, 50)), int(rng.integers(1, 60))
        new = rng.integers(0, 700, b) * (rng.random(b) < 0.7)
        rows = int(new.sum() + rng.integers(0, 5))
        assert sum(lib.units(int(n), group) for n in new if n) <= lib.total(rows, b, group)
    assert lib.units(1 << 24, 64) == 1 << 22 and lib.rows(1 << 24, 64, ((1 << 22) - 1) << 8) == 256
    assert lib.longs(0, 1 << 24, 64, 48) == (1 << 22) - 47 * 128 * 64 // 256


@pytest.mark.parametrize("splits", [1, 2, 4, 8])
def test_shares_of_a_cluster_cover_its_tiles(lib, splits):
    for tiles in range(0, 300):
        share = [lib.share(tiles, r, splits) for r in range(splits)]
        mine = [len(range(r, tiles, splits)) for r in range(splits)]
        assert share == mine and sum(share) == tiles
        # a piece of 128 tiles a CTA gives none more
        assert max(share) <= 128 or tiles > 128 * splits
