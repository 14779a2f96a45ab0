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


@pytest.mark.parametrize("dt,dim,group,keeps", [
    ("bf16", 64, 16, True), ("bf16", 128, 17, False), ("e4m3", 64, 9, True), ("e4m3", 64, 40, False),
    ("f32", 64, 8, True), ("f32", 64, 9, False), ("f32", 128, 4, True), ("f32", 128, 5, False)])
def test_room_for_logits_only_where_they_are_kept(B, dt, dim, group, keeps):  # noqa: F811
    """One tile of query heads a kv head: 16 for 16- and 8-bit pools; 8 or 4
    for fp32 ones of 64 or 128."""
    import types
    kind = {"bf16": B.PE_KV_BF16, "e4m3": B.PE_KV_E4M3, "f32": B.PE_KV_F32}[dt]
    pool = types.SimpleNamespace(dtype=kind, head_dim=dim, n_kv_heads=2)
    assert B._cache_logits_width(pool, 2 * group, 100) == (100 if keeps else 0)


@pytest.mark.parametrize("shared", ["k", "v", "scores"])
def test_evict_layers_that_share_a_pool(B, shared):  # noqa: F811
    """In place, two layers over the same memory would move it at once."""
    from tests.test_cache_abi_cpu import _pool
    apart = [dict(k=BASE * (3 * i + 1), v=BASE * (3 * i + 2), scores=BASE * (3 * i + 3))
             for i in range(3)]
    apart[2][shared] = apart[0][shared]
    assert _evict(B, [_pool(B, **x) for x in apart], dict(n=3)) == 1
