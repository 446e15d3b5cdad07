"""sdcp_pool_workspace_bytes: 0 for the sizes that the calls refuse (no GPU work)."""
import pytest

from test_pool_refusals import TOO_LARGE, compact, pool, reserve, sdcp  # noqa: F401  (a fixture)


@pytest.mark.parametrize("n_pages,n_slots", [(2**30 + 1, 3), (2**31 - 1, 3), (9, 2**30 + 1), (9, 2**31 - 1)])
def test_sizes_that_are_refused_have_no_workspace(sdcp, n_pages, n_slots):  # noqa: F811
    assert sdcp.lib.sdcp_pool_workspace_bytes(n_pages, n_slots) == 0
    p = pool(sdcp, n_pages=n_pages, n_slots=n_slots)
    assert reserve(sdcp, p, wb=1 << 40, most=2**30) == compact(sdcp, p, wb=1 << 40) == TOO_LARGE


def test_the_largest_sizes_have_one(sdcp):  # noqa: F811
    assert sdcp.lib.sdcp_pool_workspace_bytes(2**30, 2**30) >= 20 * 2**30
