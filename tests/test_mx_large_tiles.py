"""What the sizes of the GPU tests of large tiles run with, by the rules compiled from the library's own source: a change of the cost
figures that moves one to other tiles shows here."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import pytest

from tests import mx_large_tile_cases as cases
from tests.mx_plan import CSRC, CUS

SOURCE = """
#include "mx_plan.h"
extern "C" int grouped(int64_t T, int64_t N, int64_t K, int64_t E) { return mx::grouped_tile(T, N, K, E, 256); }
extern "C" int gradient(int64_t T, int64_t M, int64_t N, int64_t E) { return mx::gradient_tile(T, M, N, E, 256); }
extern "C" int dense(int64_t M, int64_t N, int64_t K, int act, int residual, int z) {
  const mx::EpilogueCosts c = mx::epilogue_costs(act == 3, act == 2 || act == 4, residual, z);
  const mx::Plan p = mx::plan_of(M, N, K, 256, true, c.of);
  return p.parts == 1 && p.first_n == 0 ? p.tile : -1;
}
"""


@pytest.fixture(scope="module")
def rules():
    folder = tempfile.mkdtemp(prefix="mx_large")
    try:
        source, lib = os.path.join(folder, "large.cpp"), os.path.join(folder, "large.so")
        with open(source, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, source, "-o", lib], check=True, capture_output=True)
        yield ctypes.CDLL(lib)
    finally:
        shutil.rmtree(folder)


def test_every_case_runs_tiles_of_256(rules):
    wide = lambda *v: [ctypes.c_int64(i) for i in v]  # noqa: E731
    for (m, n, k), (streamed, large) in cases.DENSE.items():
        assert (-(-m // 256) * -(-n // 256) > CUS, 2 * m * n > 32 << 20) == (streamed, large)
        for name, _, residual, z, _ in cases.EPILOGUES:
            act = [None, "relu", "silu", "gelu", "gelu_tanh"].index(name)
            assert rules.dense(*wide(m, n, k), act, int(residual is not None), int(z)) == 256, (m, n, k, name, residual, z)
    for sizes, n, k, (front, behind) in cases.GROUPED:
        assert rules.grouped(*wide(sum(sizes) + front + behind, n, k, len(sizes))) == 256
    for sizes, (front, behind), m, n in cases.GRADIENTS:
        assert rules.gradient(*wide(sum(sizes) + front + behind, m, n, len(sizes))) == 256
        stages = [-(-s // 256) for s in sizes]
        assert {0, 1, 2, 3, 5} <= set(stages)  # of 256 positions
    # every way out: each activation without a residual, rounded in the tile, and with the sums kept
    for kept in (False, True):
        assert {e[0] for e in cases.EPILOGUES if e[3] == kept and e[2] is None} == {None, "relu", "silu", "gelu", "gelu_tanh"}


def test_cases_of_many_groups_run_tiles_of_128(rules):
    for sizes in cases.MANY_GROUPS:
        assert rules.grouped(*(ctypes.c_int64(v) for v in sizes)) == 128, sizes
    for sizes in cases.MANY_GRADIENTS:
        assert rules.gradient(*(ctypes.c_int64(v) for v in sizes)) == 128, sizes
