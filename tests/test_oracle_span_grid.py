"""Grid positions of the oracle at both ends of a grid, against the index they stand for (CPU)."""

import math

import pytest

from oracle import span as ref


@pytest.mark.parametrize("grid", [(3, 2, 4), (5,), (1, 7), (2, 3, 1, 4)])
def test_first_and_last_cells(grid):
    cells = math.prod(grid)
    at = ref.grid_positions(grid, 0, cells)
    assert at.shape == (len(grid), cells)
    assert at[:, 0].tolist() == [0.0] * len(grid) and at[:, -1].tolist() == [g - 1.0 for g in grid]
    # every cell once, in row-major order
    for n in range(cells):
        index = 0
        for size, x in zip(grid, at[:, n]):
            assert 0 <= x < size
            index = index * size + int(x)
        assert index == n
    assert ref.grid_positions(grid, cells - 1, 1)[:, 0].tolist() == at[:, -1].tolist()
