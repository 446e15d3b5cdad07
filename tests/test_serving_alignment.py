"""Arrays of 32-bit words off a 4-byte boundary (a slice of a packed byte buffer) are refused on the host:
a kernel that read them would fault.  No GPU work."""
import pytest

from test_serving_refusals import ALIGN, P, adjust, append, attend, cache, read, sdcp  # noqa: F401


@pytest.mark.parametrize("name", ["off", "tok", "ctl", "hist", "bt", "bv", "masks", "mr", "st"])
@pytest.mark.parametrize("by", [1, 2])
def test_adjust(sdcp, name, by):  # noqa: F811
    assert adjust(sdcp, **{name: P + by}) == ALIGN


@pytest.mark.parametrize("call,names", [(append, ("off", "lens", "st")), (read, ("off", "start", "st")), (attend, ("off", "lens", "st"))])
@pytest.mark.parametrize("by", [1, 2])
def test_the_cache_calls(sdcp, call, names, by):  # noqa: F811
    for name in names:
        assert call(sdcp, **{name: P + by}) == ALIGN
    assert call(sdcp, c=cache(sdcp, page_table=P + by)) == ALIGN
