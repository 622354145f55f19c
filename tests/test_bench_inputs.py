"""The inputs that bench.py's graph replays go through: three times L2 between two uses of one set, every
set in the graph."""

import pytest

import bench

L2 = 126 * 2 ** 20


@pytest.mark.parametrize("nbytes", [1, 800_000, 2_100_000, 9_830_400, 10_200_000, 40 << 20, 126 << 20, 1 << 30])
def test_input_sets(nbytes):
    n, per, resident = bench.input_sets(nbytes)
    assert per % n == 0 and per >= 30 and (n == 1 or per < 30 + n)
    assert resident == (n * nbytes < 3 * L2)
    assert n <= 512 and (n - 1) * nbytes < 3 * L2
