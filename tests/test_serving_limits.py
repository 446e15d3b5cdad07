"""Sizes that do not fit are refused, not wrapped (no GPU work)."""
from test_serving_refusals import TOO_LARGE, adjust, append, attend, read, sdcp  # noqa: F401


def test_totals_near_the_end_of_64_bits(sdcp):  # noqa: F811
    for total in (2**31, 2**62, 2**63 - 1):
        assert adjust(sdcp, total=total) == TOO_LARGE
        assert append(sdcp, total=total) == TOO_LARGE
        assert read(sdcp, n=total) == TOO_LARGE
        assert attend(sdcp, total=total) == TOO_LARGE
