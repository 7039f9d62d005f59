"""The tiles that the block-scaled product and the orthogonalised update take for a size: csrc/blocks_plan.h and
csrc/ortho_plan.h through a small host library."""
from __future__ import annotations

import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "vocabulary_cross_entropy_row_amd", "csrc")
SHAPES = ("256x256", "256x128", "128x64", "64x32", "16 tokens", "32 tokens")
ORTHO_SHAPES = ("256", "128", "64", "128 deep", "32")
SOURCE = """#include "blocks_plan.h"
#include "ortho_plan.h"
extern "C" int blocks(long n, long K, long M, int pow2) {
    const auto p = lce::blocks_plan::plan_of(n, K, M, pow2 != 0);
    return p.shape * 100 + p.splits;
}
extern "C" int ortho(long batch, long rows_x, long rows_w, long steps, int sym, int ranges) {
    const auto p = lce::ortho_plan::plan_of(batch, rows_x, rows_w, steps, sym != 0, ranges != 0);
    return p.shape * 2 + (p.groups != p.total);
}
"""


def load(directory: str):
    """(n, K, M, e8m0) -> (shape, splits) and (batch, rows, cols) -> three times (shape, equal ranges of the
    steps?), for X X^T, the polynomial and the product that forms X; compiled into ``directory``."""
    src, so = os.path.join(directory, "plans.cpp"), os.path.join(directory, "plans.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{CSRC}", src, "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.blocks.argtypes = [ctypes.c_long] * 3 + [ctypes.c_int]
    lib.ortho.argtypes = [ctypes.c_long] * 4 + [ctypes.c_int] * 2

    def blocks(n, K, M, e8m0):
        v = lib.blocks(n, K, M, int(e8m0))
        return SHAPES[v // 100], v % 100

    def ortho(batch, rows, cols):
        rp, cp = (-(-s // 64) * 64 for s in (min(rows, cols), max(rows, cols)))
        out = [lib.ortho(batch, rp, w, k // 64, *f) for w, k, *f in ((rp, cp, 1, 1), (rp, rp, 1, 0), (cp, rp, 0, 0))]
        return [(ORTHO_SHAPES[v // 2], bool(v % 2)) for v in out]

    return blocks, ortho


# Sizes that take every shape of tile, with K in whole blocks of 128 and with a last one that is cut, in one
# launch and split along K; n and M end inside a tile.  By whether both scales are e8m0.
COVER = {
    True: [(1, 128, 49243), (1, 103, 49630), (898, 2176, 137), (819, 2318, 133), (1, 128, 65), (1, 104, 70),
           (136, 128, 21890), (196, 104, 17438), (2739, 6656, 131), (1901, 7955, 263), (264, 128, 26598),
           (385, 108, 18780), (5616, 8448, 263), (5754, 8172, 285), (17, 128, 66), (18, 101, 68), (33, 128, 65),
           (35, 108, 67), (34, 1408, 68), (34, 1286, 72)],
    False: [(1, 128, 49336), (1, 104, 49685), (1224, 2304, 207), (681, 2579, 351), (1, 384, 65), (1, 266, 67),
            (133, 128, 22057), (326, 101, 10984), (137, 5120, 5639), (2975, 5098, 276), (258, 128, 26156),
            (5997, 103, 1328), (5735, 7552, 265), (5480, 6671, 270), (17, 384, 67), (17, 262, 65), (1, 128, 65),
            (1, 108, 65), (33, 1152, 69), (34, 1076, 68)],
}
# (batch, rows, columns) that take every shape of tile for each of the update's products, and equal ranges of
# the steps where those are taken
ORTHO_COVER = [(1, 71, 65), (13, 145, 131), (1, 1932, 66), (19, 591, 598), (3, 587, 3556), (19, 422, 394),
               (15, 195, 8283), (19, 786, 877), (2, 2007, 5396), (20, 803, 65), (18, 334, 260), (13, 1801, 392),
               (17, 65, 68)]
