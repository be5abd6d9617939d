"""Arguments of a rotation that are refused before anything is looked up."""
import pytest

import sparse_linear_hybrid_top_b200 as salad


@pytest.mark.parametrize("grid", [(), (4,), (3, 4, 5), [2, 3, 4, 5]])
def test_a_grid_has_two_sides(grid):
    """(F, Hh, Wh) would be read as a frame of F x Hh."""
    with pytest.raises(ValueError, match="Hh, Wh"):
        salad._rotation(64, None, "adjacent", None, grid, 1, 60, 0)
    assert salad._rotation(64, None, "adjacent", None, (4, 5), 1, 60, 0)[-2:] == (4, 5)
