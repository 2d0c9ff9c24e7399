"""Calls of the grouped and 4-bit products that would read or write out of range, or compute
something else than was asked, are refused before any HIP call."""
import pytest

from adapter_gemv_amd import _lib

# fake device addresses: never dereferenced, every call below is refused
IDS, PERM, STARTS = 1 << 40, 2 << 40, 3 << 40


@pytest.mark.parametrize("n", [1, 64, 8192, 1 << 30])
def test_group_rows_outputs_stand_alone(n):
    """Workgroups read ids while others write the tables."""
    rows = _lib.lib().sgmv_group_rows
    for perm, starts in ((IDS, STARTS), (IDS + 4 * n - 4, STARTS), (IDS - 4 * n + 4, STARTS),
                         (PERM, IDS), (PERM, IDS + 4 * n - 4), (PERM, IDS - 4 * 7), (PERM, PERM),
                         (PERM, PERM + 4 * n - 4), (PERM, PERM - 4 * 7)):
        assert rows(None, IDS, n, 7, perm, starts) == _lib.ERR_ALIAS
