"""Sizes that do not fit are refused, not wrapped (no GPU work)."""
import pytest

from test_serving_refusals import TOO_LARGE, adjust, append, attend, read, sdcp  # noqa: F401


def test_totals_near_the_end_of_64_bits(sdcp):  # noqa: F811
    for total in (2**31, 2**62, 2**63 - 1):
        assert adjust(sdcp, total=total) == TOO_LARGE
        assert append(sdcp, total=total) == TOO_LARGE
        assert read(sdcp, n=total) == TOO_LARGE
        assert attend(sdcp, total=total) == TOO_LARGE


def test_a_window_beyond_32_bits(sdcp, monkeypatch):  # noqa: F811
    """Positions are 32-bit: such a window would reach the library as another number."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(sdcp, "_call", lambda *a: None)
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros((3, 1, 64), dtype=torch.bfloat16)
    call = lambda w: sdcp.sdcp_attend_kv(sdcp.KvCache(2, 16, 1, 64, "cpu"), z(2, 1), z(3), 1, z(2), q, q.clone(), z(2), z(4), window=w)  # noqa: E731
    call(2**31 - 1)
    for w in (2**31, 2**32, 2**32 + 5):
        with pytest.raises(ValueError):
            call(w)
