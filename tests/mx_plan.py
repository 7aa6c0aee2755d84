"""The rule that picks an MXFP4 product's kernel, compiled for the host from the library's own source: which tiles, K parts
and column split a size runs with on a device of 256 compute units."""
import ctypes
import functools
import os
import shutil
import subprocess
import tempfile
from collections import namedtuple

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_fp4_w4a16_amd", "csrc")
CUS = 256

SOURCE = """
#include "mx_plan.h"
extern "C" void plan(int64_t M, int64_t N, int64_t K, int cus, int64_t* out) {
  const mx::Plan p = mx::plan_of(M, N, K, cus);
  const mx::Plan rest = p.first_n ? mx::plan_of(M, N - p.first_n, K, cus, false) : mx::Plan{};
  out[0] = p.tile, out[1] = p.parts, out[2] = p.per, out[3] = p.first_n, out[4] = rest.tile, out[5] = mx::fused(M, N, K);
}
"""

# tile: 0 for the kernel of few rows, else 64, 128 or 256; first_n: columns of a first product (0: one product), whose
# others run with tiles of `rest`; streamed: workgroups take several tiles of 256
Plan = namedtuple("Plan", "tile parts per first_n rest fused streamed")


@functools.cache
def _lib():
    folder = tempfile.mkdtemp(prefix="mx_plan")
    try:
        source, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
        with open(source, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, source, "-o", lib], check=True, capture_output=True)
        return ctypes.CDLL(lib)
    finally:
        shutil.rmtree(folder)


def plan(m, n, k):
    out = (ctypes.c_int64 * 6)()
    _lib().plan(ctypes.c_int64(m), ctypes.c_int64(n), ctypes.c_int64(k), CUS, out)
    tile, parts, per, first_n, rest, fused = out
    tiles = -(-m // tile) * -(-(first_n or n) // tile) * parts if tile else 0
    return Plan(tile, parts, per, first_n, rest, bool(fused), tile == 256 and tiles > CUS)


# Products that reach the large tiles, with what each is meant to run: (m, n, k) -> (tile, K parts, columns of a first
# product, tiles of the others, several tiles per workgroup)
TILE_CASES = {
    (8192, 8192, 800): (256, 1, 0, 0, True),       # 1024 tiles on 256 workgroups, four stages
    (8190, 8100, 1100): (256, 1, 0, 0, True),      # five stages, the last one part full, both edges ragged
    (16001, 8191, 289): (256, 1, 0, 0, True),      # two stages, odd rows of y
    (12033, 16129, 200): (256, 1, 0, 0, True),     # one stage, the last tile row and column one row and column wide
    (8190, 8200, 1100): (256, 1, 8192, 64, True),  # columns behind the whole rounds in tiles of 64
    (8192, 2560, 9728): (256, 1, 2048, 128, False),  # and of 128
    (4090, 4090, 1300): (256, 1, 0, 0, False),     # one tile per workgroup
    (2000, 2100, 1300): (128, 1, 0, 0, False),
    (1999, 2111, 1100): (128, 1, 0, 0, False),
    (300, 2000, 32768): (128, 4, 0, 0, False),     # K in parts
    (299, 2001, 33000): (128, 4, 0, 0, False),
    (300, 260, 5000): (64, 4, 0, 0, False),
}
# layers whose product, gradients of x and of w (m n k, m k n, n k m) all run in tiles of 128 or 256
LAYER_CASES = [(4100, 4300, 2050), (8192, 2050, 2570)]
