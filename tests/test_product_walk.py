"""How the 8-bit grouped product's workgroups share its tiles (csrc/walk.h, compiled here for the host): whatever the
offsets, every tile is taken once, and a workgroup that goes on to a next tile has found it during the tile before,
past a barrier after the stores of the one before that.

Groups may overlap where offsets fall, and then have more tiles than the launch counts on."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_load_layer_amd", "csrc")
SOURCE = """
#include "walk.h"
extern "C" {
void walk(int64_t tiles, uint32_t block, uint32_t blocks, int64_t *out) {
    const ep::TileWalk w = ep::tile_walk(tiles, block, blocks);
    out[0] = w.at, out[1] = w.to, out[2] = w.stride;
}
int find_step(int steps, int stages) { return ep::find_step(steps, stages); }
int chained(int steps, int stages) { return ep::tiles_chained(steps, stages); }
int64_t blocks(int64_t m, int64_t groups, int64_t n, int rows, int columns) {
    return ep::tile_blocks(m, groups, n, rows, columns);
}
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    at = tmp_path_factory.mktemp("walk")
    (at / "walk.cpp").write_text(SOURCE)
    lib = str(at / "libwalk.so")
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-O1", "-shared", "-fPIC", "-I", CSRC,
                    str(at / "walk.cpp"), "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    i64, u32, i32 = ctypes.c_int64, ctypes.c_uint32, ctypes.c_int
    L.walk.argtypes = [i64, u32, u32, ctypes.POINTER(i64)]
    L.walk.restype = None
    L.find_step.argtypes = L.chained.argtypes = [i32, i32]
    L.blocks.argtypes = [i64, i64, i64, i32, i32]
    L.blocks.restype = i64
    return L


def _row_tiles(offsets, m, rows):
    o = np.clip(np.asarray(offsets), 0, m)
    return int((-(-np.maximum(o[1:] - o[:-1], 0) // rows)).sum())


@pytest.mark.parametrize("stages,tile", [(4, 256), (4, 128), (6, 64)])
@pytest.mark.parametrize("m,n,offsets", [
    (6400, 64, [0, 6400, 0, 6400]), (6400, 200, [0, 6400] * 8), (1000, 700, [0, 300, 300, 1000]), (1, 1, [0, 1]),
    (500, 300, [7, 2, 400, -5, 900, 0, 500, 100, 500]), (12288, 1024, [0, 12288, 0, 12288]),
    (777, 1000, [777, 0, 777, 0, 777]), (64, 64, [0, 0, 0])])
@pytest.mark.parametrize("blocks_of_k", [1, 2, 3, 4, 5, 6, 7, 33])
def test_every_tile_is_found_before_it_is_taken(walk, stages, tile, m, n, offsets, blocks_of_k):
    steps = 2 * blocks_of_k
    tiles = _row_tiles(offsets, m, tile) * -(-n // tile)
    launched = walk.blocks(m, len(offsets) - 1, n, tile, tile)
    chained = bool(walk.chained(steps, stages))
    assert launched % 8 == 0
    if (np.diff(np.clip(offsets, 0, m)) >= 0).all():
        assert launched >= tiles                       # each its own, where groups do not overlap
    for blocks in ({launched, min(launched, 64)} if chained else {launched}):
        taken = np.zeros(tiles, dtype=int)
        out = (ctypes.c_int64 * 3)()
        for b in range(blocks):
            walk.walk(tiles, b, blocks, out)
            own = range(out[0], out[1], out[2])
            for at in own:
                taken[at] += 1
            if chained and len(own) > 1:
                s = walk.find_step(steps, stages)
                assert 0 < s < steps - stages and s % 2 == 0
        assert (taken == 1).all()
