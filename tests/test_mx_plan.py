"""What the sizes of the GPU tests run with: a change of the cost figures that moves one to another kernel shows here."""
import pytest

from tests.mx_plan import LAYER_CASES, TILE_CASES, plan


@pytest.mark.parametrize("size", TILE_CASES)
def test_tile_cases_run_what_they_are_meant_to(size):
    p = plan(*size)
    assert (p.tile, p.parts, p.first_n, p.rest, p.streamed) == TILE_CASES[size]


@pytest.mark.parametrize("m,n,k", LAYER_CASES)
def test_layer_cases_reach_the_large_tiles(m, n, k):
    plans = [plan(m, n, k), plan(m, k, n), plan(n, k, m)]
    assert all(p.tile in (128, 256) for p in plans)


def test_few_rows_and_parts():
    assert plan(1, 4096, 4096).tile == 0 and plan(16, 2560, 9728).tile == 0 and plan(17, 2560, 9728).tile == 64
    assert plan(1, 4096, 4096).fused and not plan(1, 14336, 4096).fused
    for m, n, k in ((40, 100, 32768), (64, 2560, 9728), (300, 2000, 32768)):
        p = plan(m, n, k)
        stages = -(-k // 256)
        assert p.parts > 1 and p.per % 2 == 0 and p.per * (p.parts - 1) < stages <= p.per * p.parts   # no part is empty
