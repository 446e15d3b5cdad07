"""Sizes of sdcp_attend_shared_kv that its arithmetic does not hold are refused (no GPU work)."""
import pytest

from test_attend_shared_refusals import TOO_LARGE, attend, sdcp  # noqa: F401  (a fixture)


@pytest.mark.parametrize("B,groups", [(1, 2**31 - 1), (2**20, 2**31 - 2**20), (1, 2**30), (2**20, 2**30 - 1)])
def test_groups_and_sessions_are_counted_together(sdcp, B, groups):  # noqa: F811
    """Entries of both kinds are one list, walked in 32 bits."""
    assert sdcp.lib.sdcp_attend_shared_workspace_bytes(B, 0, groups, 1, 1, 64) == 0
    assert attend(sdcp, B=B, total=0, ng=groups, nq=2) == TOO_LARGE


def test_many_empty_groups_are_taken(sdcp):  # noqa: F811
    assert sdcp.lib.sdcp_attend_shared_workspace_bytes(2, 0, 2**29, 1, 1, 64) > 2**29 * 8
