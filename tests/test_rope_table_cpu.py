"""Sizes of the rotation's table."""
import pytest

from tiled_stage_software_amd import ops


@pytest.mark.parametrize("rows,rot", [(10, 5), (10, 1), (10, -2), (-1, 4)])
def test_rope_table_refuses_odd_sizes(rows, rot):
    with pytest.raises(ValueError):
        ops.rope_table(rows, rot)


def test_rope_table_of_nothing():
    assert ops.rope_table(10, 0)[0].shape == (10, 0) and ops.rope_table(0, 6)[1].shape == (0, 3)
