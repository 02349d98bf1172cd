"""CPU tests of csrc/group_tiles.h, the arithmetic by which the kernels over groups of rows find their tiles,
compiled here from the header that they include."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "layout_general_tensor_gb300", "csrc")
SHIM = """
#include "group_tiles.h"
static uint32_t recip[lgt::kGgBand + 1];
extern "C" {
uint32_t band() { lgt::band_reciprocals(recip); return lgt::kGgBand; }
uint32_t divide(uint32_t n, uint32_t d) { return lgt::divide_few(recip, n, d); }
uint32_t width(uint32_t rows, uint32_t tiles, uint32_t step) { return lgt::even_width(recip, rows, tiles, step); }
uint64_t place(uint32_t r, uint32_t p_tiles, uint32_t q_tiles) {
  uint32_t p, q;
  lgt::tile_in_bands(recip, r, p_tiles, q_tiles, p, q);
  return static_cast<uint64_t>(p) << 32 | q;
}
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    at = tmp_path_factory.mktemp("tiles")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(at / "shim.cpp"), "-o", str(at / "shim.so")], check=True)
    lib = ctypes.CDLL(str(at / "shim.so"))
    for f in (lib.band, lib.divide, lib.width):
        f.restype = ctypes.c_uint32
    lib.place.restype = ctypes.c_uint64
    lib.band()
    return lib


def test_divisions_by_reciprocals(tiles):
    r = random.Random(0)
    for d in range(1, tiles.band() + 1):
        near = list(range(300)) + [(1 << 29) - 1, (1 << 29) // d * d - 1] + [r.randrange(1 << 29) // d * d + e for e in (-1, 0, 1) for _ in range(2000)]
        for n in near:
            if 0 <= n < 1 << 29:
                assert tiles.divide(n, d) == n // d, (n, d)


@pytest.mark.parametrize("step,most", [(16, 64), (16, 128), (16, 256), (32, 256), (16, 112), (16, 96)])
def test_tiles_cover_a_group_once(tiles, step, most):
    """None empty, none wider than the most, the first start behind the last end."""
    r = random.Random(step + most)
    for rows in [*range(1, 700), *(r.randrange(1, 1 << 22) for _ in range(3000)), (1 << 30) - 1, 1 << 30]:
        n = -(-rows // most)
        width = tiles.width(rows, n, step)
        assert width % step == 0 and width <= most and (n - 1) * width < rows <= n * width, (rows, n, width)


def test_tiles_in_bands_come_once_each(tiles):
    for p_tiles in (1, 2, 3, 7, 12, 33):
        for q_tiles in (*range(1, 20), 40, 41):
            seen = [tiles.place(r, p_tiles, q_tiles) for r in range(p_tiles * q_tiles)]
            assert sorted(seen) == [p << 32 | q for p in range(p_tiles) for q in range(q_tiles)]
            # tiles of one stretch of n within a band follow each other
            for r, (a, b) in enumerate(zip(seen, seen[1:])):
                assert b - a == 1 or (a & 0xffffffff) % 8 == 7 or (a & 0xffffffff) == q_tiles - 1, r
    # the largest: 2^31 tiles
    p_tiles, q_tiles = 1 << 11, (1 << 20) - 1
    for r in (0, 7, 8, p_tiles * 8 - 1, p_tiles * 8, p_tiles * q_tiles - 1, p_tiles * (q_tiles - 7) - 1, p_tiles * (q_tiles - 7)):
        band, left = divmod(r, p_tiles * 8)
        high = min(8, q_tiles - band * 8)
        assert tiles.place(r, p_tiles, q_tiles) == (left // high << 32 | band * 8 + left % high)
