"""Workspaces of MXFP4 products with an epilogue, without a GPU: what the queries name holds the planes of the plan that runs, and
with less of it the plan has planes that fit. The rule is compiled for the host from the library's own source."""
import ctypes
import math
import os
import random
import shutil
import subprocess
import tempfile

import pytest

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")

ARG, SHAPE, ALIGN, UNSUP = -1, -2, -3, -4
FAKE = 1 << 20
ACTS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
EPILOGUES = [(act, residual, z) for act in ACTS for residual in (False, True) for z in (False, True)]

SOURCE = """
#include "mx_plan.h"
extern "C" void plan(int64_t M, int64_t N, int64_t K, int act, int residual, int z, int64_t room, double* out) {
  const mx::EpilogueCosts c = mx::epilogue_costs(act == 3, act == 2 || act == 4, residual, z);
  const mx::Plan p = act < 0 ? mx::plan_of(M, N, K, 256) : mx::plan_of(M, N, K, 256, true, c.of, room);
  out[0] = p.tile, out[1] = p.parts, out[2] = p.us, out[3] = (double)mx::plane_bytes(p, M), out[4] = mx::fused(M, N, K);
}
"""


@pytest.fixture(scope="module")
def plan():
    folder = tempfile.mkdtemp(prefix="mx_room")
    try:
        source, lib = os.path.join(folder, "room.cpp"), os.path.join(folder, "room.so")
        with open(source, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(os.path.dirname(fp4.__file__), "csrc"), source,
                        "-o", lib], check=True, capture_output=True)
        rule = ctypes.CDLL(lib).plan
    finally:
        shutil.rmtree(folder)

    def call(m, n, k, epilogue=None, room=1 << 62):
        act, residual, z = (-1, 0, 0) if epilogue is None else (ACTS[epilogue[0]], *epilogue[1:])
        out = (ctypes.c_double * 5)()
        rule(*(ctypes.c_int64(v) for v in (m, n, k)), act, int(residual), int(z), ctypes.c_int64(room), out)
        return dict(tile=int(out[0]), parts=int(out[1]), us=out[2], planes=int(out[3]), fused=bool(out[4]))
    return call


def native(epilogue, n):
    act, residual, z = epilogue
    return fp4.Epilogue(FAKE, FAKE if residual else None, FAKE if z else None, n, n, 2, 2, ACTS[act])


def sizes(count, seed):
    rng = random.Random(seed)
    spread = lambda low, high: round(math.exp(rng.uniform(math.log(low), math.log(high))))  # noqa: E731
    return [(spread(1, 4096), spread(16, 14336), spread(32, 32768)) for _ in range(count)]


SIZES = [(20, 635, 8192), (19, 589, 8192), (23, 1687, 8192), (80, 2176, 26080), (17, 1024, 23360), (41, 688, 15840), (1, 4096, 4096),
         (333, 2560, 9728), (8192, 9728, 2560)] + sizes(400, 1)


def test_the_workspace_holds_the_planes(plan):
    """Asked of the shape alone, it serves every epilogue; asked of one call, it is that call's."""
    lib, some, none = fp4.lib(), 0, 0
    for m, n, k in SIZES:
        operand = lib.w4a4_linear_epilogue_workspace_bytes(m, n, k, None) - lib.w4a4_matmul_epilogue_workspace_bytes(m, n, k, None)
        assert lib.w4a4_matmul_epilogue_workspace_bytes(m, n, k, None) == plan(m, n, k)["planes"]
        for epilogue in EPILOGUES:
            p, e = plan(m, n, k, epilogue), native(epilogue, n)
            assert lib.w4a4_matmul_epilogue_workspace_bytes(m, n, k, e) == p["planes"], (m, n, k, epilogue)
            assert lib.w4a4_matmul_workspace_bytes(m, n, k) >= p["planes"], (m, n, k, epilogue)
            linear = lib.w4a4_linear_epilogue_workspace_bytes(m, n, k, e)
            assert linear == (0 if p["fused"] else operand + p["planes"]), (m, n, k, epilogue)
            assert lib.w4a4_linear_workspace_bytes(m, n, k) >= linear
            some += p["parts"] > 1
            none += p["parts"] == 1
    assert some > 500 and none > 500


def test_less_room_has_fewer_parts(plan):
    for m, n, k in SIZES[:60] + [(17, 1024, 23360), (80, 2176, 26080)]:
        for epilogue in EPILOGUES[::3]:
            full = plan(m, n, k, epilogue)
            before = plan(m, n, k, epilogue, 0)
            assert before["parts"] == 1
            for part in (0.1, 0.3, 0.5, 0.9, 1.0):
                p = plan(m, n, k, epilogue, int(part * full["planes"]))
                assert p["planes"] <= part * full["planes"] and full["us"] <= p["us"] <= before["us"]
                before = p
            assert before == full


def test_the_epilogue_leaves_the_number_of_parts_alone(plan):
    """Tiles that write planes have no epilogue: where K is in parts with and without one, in the same ones."""
    both = 0
    for m, n, k in SIZES:
        bare = plan(m, n, k)
        for epilogue in EPILOGUES:
            p = plan(m, n, k, epilogue)
            if bare["parts"] > 1 and p["parts"] > 1:
                both += 1
                assert (p["tile"], p["parts"]) == (bare["tile"], bare["parts"]), (m, n, k, epilogue)
    assert both > 500


def test_refusals_of_the_queries():
    for query in (fp4.lib().w4a4_matmul_epilogue_workspace_bytes, fp4.lib().w4a4_linear_epilogue_workspace_bytes):
        for e in (None, native(("silu", True, True), 16)):
            assert query(-1, 16, 32, e) == SHAPE and query(1, 0, 32, e) == SHAPE and query(1, 16, 0, e) == SHAPE
            assert query(1, 16, 1 << 23, e) == UNSUP and query(0, 16, 32, e) == 0
        assert query(40, 17, 32, native(("silu", True, False), 16)) == SHAPE                 # the residual's rows are shorter
        bad = native((None, False, False), 16)
        bad.activation = 9
        assert query(40, 16, 32, bad) == ARG
        bad = native((None, False, False), 16)
        bad.bias = FAKE + 1
        assert query(40, 16, 32, bad) == ALIGN
