"""More refusals of the paged KV cache operators that the host makes before it
touches the device."""

import pytest

from tests.test_cache_abi_cpu import B, BASE, _evict  # noqa: F401  (B: the fixture)


@pytest.mark.parametrize("change", [dict(dstride=1), dict(dstride=3), dict(B=1, dstride=1)])
def test_evict_into_its_own_table_of_another_width(B, change):  # noqa: F811
    """The same pages as source and destination, without the order that makes
    that safe in place (a one-row table and its slice start alike)."""
    assert _evict(B, change=dict(change, dst=BASE)) == 1


@pytest.mark.parametrize("current,capturing,shares", [
    (0, {}, False), (1, {}, True), (0, {1: True}, False), (1, {1: True}, False),
    (1, {0: True}, True)])
def test_a_captured_call_never_takes_a_shared_workspace(B, current, capturing, shares):  # noqa: F811
    """Whether a stream is being captured is asked of the current device: a
    call for another device's pool has a workspace of its own."""
    import types
    fake = types.SimpleNamespace(_C=types.SimpleNamespace(
        _cuda_getDevice=lambda: current,
        _cuda_isCurrentStreamCapturing=lambda: capturing.get(current, False)))
    pool = types.SimpleNamespace(index=1, torch=fake)
    assert B._cache_shares(pool, 1024, None) is shares
    assert not B._cache_shares(pool, 1 << 40, None)
    assert not B._cache_shares(pool, 1024, object())
