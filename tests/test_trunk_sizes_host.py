"""Sizes at and beyond what the trunk operators' C entry points hold in an int, on the host."""
import pytest

from recurrent_cfc_cell_gb300 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("n", [1, 8, 60, 256, 1024, 5000, 8192])
def test_workspace_of_the_most_rows(n):
    """From some number of rows on the grid is full and the workspace stays the same, up to the
    largest int."""
    full = _lib.layernorm_workspace_bytes(10**8, n)
    assert full > 0
    for rows in (2**31 - 64, 2**31 - 2, 2**31 - 1):
        assert _lib.layernorm_workspace_bytes(rows, n) == full
