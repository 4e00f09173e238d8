"""The way that a product of block-scaled E4M3 matrices goes, by its sizes, on the
host (``csrc/ss1_dense8_choice.h``, compiled here for the CPU): the sizes that the
GPU tests multiply reach every tile, type and number of splits that there is, and
the workspace that a call asks for fits whatever its type chooses."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from sketched_parameter_sharing_amd import _lib

torch = pytest.importorskip("torch")
from test_gpu_dense_tiles import F, H, TILES  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sketched_parameter_sharing_amd", "csrc")
RING = {(64, 64): 4, (64, 128): 3, (128, 128): 2, (192, 256): 2, (256, 256): 2}  # LDS buffers

MODEL = r"""
#include "ss1_dense8_choice.h"
using namespace ss1;
extern "C" int tiles() { return kTiles; }
extern "C" void tile(int i, int* out) { out[0] = kRates[i].bm; out[1] = kRates[i].bn; }
// -1: by the weight's rows
extern "C" int way(int64_t M, int64_t N, int64_t K, int f32, int* splits) {
    if (few_rows(M, N, K)) return -1;
    const Choice c = choose(M, N, K, f32);
    *splits = c.splits;
    return c.tile;
}
extern "C" int pair(int64_t M, int64_t N, int64_t K, int f32) { return pairable(M, N, K, f32); }
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("choice")
    (d / "model.cpp").write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", f"-I{CSRC}", str(d / "model.cpp"),
                    "-o", str(d / "model.so")], check=True)
    lib = ctypes.CDLL(str(d / "model.so"))
    i64, i32, p = ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ctypes.c_int)
    lib.way.argtypes, lib.pair.argtypes, lib.tile.argtypes = [i64, i64, i64, i32, p], [i64, i64, i64, i32], [i32, p]
    return lib


def tiles_of(model):
    out = (ctypes.c_int * 2)()
    for i in range(model.tiles()):
        model.tile(i, out)
        yield out[0], out[1]


def way(model, M, N, K, f32):
    splits = ctypes.c_int(0)
    i = model.way(M, N, K, f32, ctypes.byref(splits))
    return None if i < 0 else (list(tiles_of(model))[i], splits.value)


def test_the_listed_products_go_the_way_they_are_listed_for(model):
    for expected, types in TILES.items():
        for dtype, sizes in types.items():
            for M, N, stages in sizes:
                assert way(model, M, N, stages * 128, dtype == F) == expected, (M, N, stages, dtype)


def test_every_tile_type_and_ring_is_listed(model):
    assert set(tiles_of(model)) == set(RING) == {tile for tile, _ in TILES}
    assert {splits for _, splits in TILES} == {1, 2, 4, 8}
    for ((bm, bn), splits), types in TILES.items():
        # a float32 y has no 256 x 256 tile
        assert set(types) == ({H} if (bm, bn) == (256, 256) else {H, F})
        for sizes in types.values():
            assert all(M % bm and N % bn for M, N, _ in sizes)
            if splits == 1:
                ring = RING[bm, bn]
                assert {s % ring for _, _, s in sizes} == set(range(ring)) and max(s for _, _, s in sizes) > ring


def test_the_workspace_fits_whatever_is_chosen(model):
    lib, n, rng = _lib.load(), ctypes.c_size_t(0), random.Random(5)
    for _ in range(20000):
        M, N, K = (int(round(2 ** rng.uniform(0, top))) for top in (14, 14, 15))
        K = -(-K // 128) * 128
        a, b = _lib.Fp8BlocksView(None, None, M, K, 1, 0), _lib.Fp8BlocksView(None, None, N, K, 1, 0)
        assert lib.ss1_matmul_fp8_blocks_query(ctypes.byref(a), ctypes.byref(b), ctypes.byref(n)) == _lib.OK
        for f32 in (0, 1):
            w = way(model, M, N, K, f32)
            if w is None:
                assert n.value == 0 and M <= 16
            elif w[1] > 1:
                assert n.value >= w[1] * M * N * 4 and w[0] == (64, 64) and w[1] * 4 * 128 <= K
            # two products in one launch have no workspace
            if model.pair(M, N, K, f32):
                assert w is None or w == ((64, 64), 1)


def test_few_rows_stay_within_a_grid(model):
    for M in (1, 4, 5, 16):
        for N in (1 << 28) - 16, (1 << 28) - 15, 1 << 28, (1 << 29) - 128:
            if way(model, M, N, 128, 0) is None:
                assert -(-N // 16) * 256 < 1 << 32
    assert way(model, 1, (1 << 28) - 16, 128, 0) is None and way(model, 17, 1000, 128, 0) is not None
