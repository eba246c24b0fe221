"""The spread of an expert's blocks of rows over its row tiles
(moe_layer_zero_amd/csrc/row_split.h) against exact integers, up to the largest
layers that the kernels take: fewer than 2^22 rows of one expert.  Compiled for the
host, where a product past 31 bits wraps as on the GPU."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = """
#include "row_split.h"
extern "C" int first(int blocks, int mt, int tiles) { return zc::first_block(blocks, mt, tiles); }
extern "C" int first32(int blocks, int mt, int tiles) { return zc::first_block32(blocks, mt, tiles); }
// the first tile whose start is not the quotient in 64 bits, -1 if there is none
extern "C" int differs(int blocks, int tiles) {
  for (int mt = 0; mt <= tiles; ++mt)
    if (zc::first_block(blocks, mt, tiles) != (long long)blocks * mt / tiles) return mt;
  return -1;
}
"""


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    tmp = tmp_path_factory.mktemp("split")
    (tmp / "split.cpp").write_text(SRC)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fwrapv", "-I",
                    os.path.join(ROOT, "moe_layer_zero_amd", "csrc"), str(tmp / "split.cpp"),
                    "-o", str(tmp / "split.so")], check=True)
    return C.CDLL(str(tmp / "split.so"))


MANY = [(1 << 21) - 1, 1 << 21, (1 << 21) + 1, 2_350_000, 3_000_001, (1 << 22) - 32, (1 << 22) - 1]


@pytest.mark.parametrize("block,tile", [(16, 128), (16, 160), (32, 128), (32, 256)])
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 129, 1000, 4097, 70000, *MANY])
def test_spread(split, rows, block, tile):
    blocks, tiles = -(-rows // block), -(-rows // tile)
    assert split.differs(blocks, tiles) == -1
    firsts = [split.first(blocks, mt, tiles) for mt in (0, 1, tiles // 2, tiles - 1, tiles)]
    assert firsts == [blocks * mt // tiles for mt in (0, 1, tiles // 2, tiles - 1, tiles)]
    # every tile has a block, and none more than it has room for
    starts = [split.first(blocks, mt, tiles) for mt in range(min(tiles, 3000) + 1)]
    assert all(0 < b - a <= tile // block for a, b in zip(starts, starts[1:]))


def test_small_layers(split):
    for tiles in range(1, 40):
        for blocks in range(tiles, 10 * tiles + 1, 3):
            assert split.differs(blocks, tiles) == -1


@pytest.mark.parametrize("rows", [1, 257, 70000, (1 << 22) - 257, (1 << 22) - 32, (1 << 22) - 31, (1 << 22) - 1])
def test_spread_of_32_row_blocks(split, rows):
    # blocks of 32 rows, tiles of 256: the product reaches 2^31 itself
    blocks, tiles = -(-rows // 32), -(-rows // 256)
    got = [split.first32(blocks, mt, tiles) for mt in range(tiles + 1)]
    assert got == [blocks * mt // tiles for mt in range(tiles + 1)]
