"""More refusals of the paged KV cache operators that the host makes before it
touches the device."""

import pytest

from tests.test_cache_abi_cpu import B, BASE, _evict  # noqa: F401  (B: the fixture)


@pytest.mark.parametrize("change", [dict(dstride=1), dict(dstride=3), dict(B=1, dstride=1)])
def test_evict_into_its_own_table_of_another_width(B, change):  # noqa: F811
    """The same pages as source and destination, without the order that makes
    that safe in place (a one-row table and its slice start alike)."""
    assert _evict(B, change=dict(change, dst=BASE)) == 1
