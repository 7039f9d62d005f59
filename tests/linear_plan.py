"""The tiles that the matrix product takes for a size: csrc/linear_plan.h through a small host library."""
from __future__ import annotations

import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "vocabulary_cross_entropy_row_amd", "csrc")
SHAPES = ("256x256", "256x128", "128x64", "64x32", "16 tokens", "32 tokens")
SOURCE = """#include "linear_plan.h"
extern "C" int plan(long n, long K, long M, int fp8) {
    const auto p = lce::linear_plan::plan_of(n, K, M, fp8 != 0);
    return p.shape * 100 + p.splits;
}
"""


def load(directory: str):
    """(n, K, M, e4m3) -> (shape, splits), compiled into ``directory``."""
    src, so = os.path.join(directory, "plan.cpp"), os.path.join(directory, "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", f"-I{CSRC}", src, "-o", so], check=True)
    fn = ctypes.CDLL(so).plan
    fn.argtypes = [ctypes.c_long, ctypes.c_long, ctypes.c_long, ctypes.c_int]

    def plan(n, K, M, e4m3=False):
        v = fn(n, K, M, int(e4m3))
        return SHAPES[v // 100], v % 100

    return plan


# Sizes, by the operands' type, that take every shape of tile, with K in whole steps of 128 bytes and with a
# last one that is cut, in one launch and split along K; n and M end inside a tile.
COVER = {
    "bf16": [(5719, 200, 132), (67, 2056, 999), (65, 256, 11285), (65, 2688, 855), (1, 264, 102), (5, 320, 101),
             (145, 208, 22353), (5465, 1264, 271), (137, 256, 22107), (131, 1280, 11831), (277, 200, 27071),
             (6029, 3472, 279), (260, 256, 26401), (5545, 3840, 275), (17, 352, 103), (18, 384, 102), (34, 200, 67),
             (34, 904, 81), (33, 256, 66), (33, 1024, 68), (77, 1000, 50257)],
    "e4m3": [(66, 400, 5510), (65, 3776, 2033), (2762, 512, 133), (908, 3840, 135), (1, 656, 100), (5, 768, 101),
             (140, 416, 22733), (5792, 3104, 258), (130, 512, 22103), (140, 3200, 11335), (258, 400, 29283),
             (5491, 8256, 274), (387, 512, 20013), (5612, 9472, 294), (17, 208, 114), (17, 256, 104), (33, 416, 70),
             (33, 2608, 65), (35, 512, 66), (33, 2304, 71)],
}
